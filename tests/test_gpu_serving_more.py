"""The serving operators under the calls a program may make of them: random shapes, captured
graphs, several streams, empty steps, non-finite bounds, and the index-checking build."""
import importlib.util
import os
import random
import subprocess
import sys

import pytest
import torch

from tests import gpu_util, paged_util as pu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _attn(s, o, lse, ws, causal=True, sel=None, stream=None):
    m = gpu_util.ea()
    a = (s.dq, s.dkc, s.dvc, s.dtable, s.dcu, s.dseq)
    if sel is None:
        m.attn_fwd_paged(*a, o, lse, causal, s.scale, ws, stream=stream)
    else:
        m.attn_sparse_paged(*a, sel, o, lse, s.scale, ws, stream=stream)


def _upload(s):
    s.dq, s.dkc, s.dvc = s.q.cuda(), s.kc.cuda(), s.vc.cuda()
    s.dtable, s.dcu, s.dseq = s.table.cuda(), s.cu.cuda(), s.seq.cuda()
    return s


def _out(s):
    return (torch.full((s.T, s.Hq, s.d), -77, dtype=torch.bfloat16, device="cuda"),
            torch.full((s.T, s.Hq), -77, dtype=torch.float32, device="cuda"))


def _ws(d):
    return torch.empty(gpu_util.ea().attn_fwd_paged_workspace_bytes(d), dtype=torch.uint8,
                       device="cuda")


@pytest.mark.parametrize("seed", range(24))
def test_random_steps(seed):
    """Mixed batches (prompts, chunks, single tokens, nothing) of random heads and pages."""
    r = random.Random(seed)
    Hkv = r.choice([1, 2, 3])
    Hq = Hkv * r.choice([1, 2, 4, 5, 8, 17, 33])
    d, ps = r.choice([64, 128]), r.choice([16, 32, 64, 128, 256])
    B = r.randrange(1, 9)
    kind = r.choice(["decode", "drafts", "mixed"])
    new = [1 if kind == "decode" else r.randrange(0, 9) if kind == "drafts"
           else r.choice([0, 1, 1, 40, 130, 257]) for _ in range(B)]
    if sum(new) == 0:
        new[0] = 1
    ctx = [r.choice([0, 1, 15, 127, 128, 129, 500, 1700]) for _ in range(B)]
    s = _upload(pu.make_step(new, ctx, Hq, Hkv, d, ps, seed=seed, pad=r.choice([0, 3])))
    o, lse = _out(s)
    causal = r.random() < 0.7
    _attn(s, o, lse, _ws(d), causal)
    assert gpu_util.ea().attn_status() == 0
    pu.check_attn(s, o.cpu(), lse.cpu(), pu.ref_attn(s, causal), f"seed {seed}")
    K = r.choice([1, 3, 8])
    sel = torch.full((s.T, Hkv, K), -1, dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    for b in range(B):
        pages = max(1, -(-s.lens[b] // ps))
        for i in range(new[b]):
            for h in range(Hkv):
                pick = torch.randperm(pages, generator=g)[:r.randrange(0, K + 1)]
                sel[int(s.cu[b]) + i, h, :len(pick)] = pick.int()
    o, lse = _out(s)
    _attn(s, o, lse, _ws(d), sel=sel.cuda())
    assert gpu_util.ea().attn_status() == 0
    pu.check_attn(s, o.cpu(), lse.cpu(), pu.ref_attn(s, sel=sel), f"sparse seed {seed}")


def test_steps_without_tokens():
    """All sequences empty, or nothing but padding rows: outputs stay as they were."""
    m = gpu_util.ea()
    s = _upload(pu.make_step([0, 0], [40, 0], 4, 2, 64, 16, seed=1, pad=3))
    o, lse = _out(s)
    _attn(s, o, lse, _ws(64))
    sel = torch.full((3, 2, 4), -7, dtype=torch.int32, device="cuda")
    kb = pu.page_bounds(torch.nan_to_num(s.kc)).cuda()
    ws = torch.empty(m.attn_page_select_workspace_bytes(3, 2, s.max_pages), dtype=torch.uint8,
                     device="cuda")
    m.attn_page_select(s.dq, kb, s.dtable, s.dcu, s.dseq, sel, 16, 0, 1, ws)
    assert m.attn_status() == 0
    assert (o == -77).all() and (lse == -77).all() and (sel == -7).all()


def test_many_rows_of_slots():
    """More rows than one CTA, or eight, take at a time."""
    m = gpu_util.ea()
    ps, ctx, new = 16, [5, 0, 100, 33], [4000, 9000, 1, 2000]
    max_pages = 600
    need = [-(-(c + n) // ps) for c, n in zip(ctx, new)]
    num_pages = sum(need) + 5
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(3)).tolist()
    table = [[perm.pop() if i < -(-c // ps) else -5 for i in range(max_pages)] for c in ctx]
    T = sum(new) + 100
    want = pu.ref_tables(ctx, new, perm, 0, table, T, ps, num_pages)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tab, head, seq, cu = i32(table), i32([0]), i32([0] * 4), i32([0] * 5)
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    m.attn_page_tables(i32(ctx), i32(new), i32(perm), head, head, tab, seq, cu, slots, ps, num_pages)
    assert m.attn_status() == 0 and want[-1]
    assert tab.tolist() == want[0] and seq.tolist() == want[1] and cu.tolist() == want[2]
    assert slots.tolist() == want[3] and head.item() == want[4]


def test_captured_graphs_and_streams_side_by_side():
    """Two captured steps with workspaces of their own, replayed at the same time on two streams,
    a few times over, while inputs change between the replays."""
    m = gpu_util.ea()
    steps, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i, (new, ctx, Hq, Hkv, d, ps) in enumerate([([1] * 6, [900, 5, 77, 2000, 128, 640], 8, 2, 128, 64),
                                                    ([140, 3], [300, 1000], 6, 2, 64, 32)]):
        s = _upload(pu.make_step(new, ctx, Hq, Hkv, d, ps, seed=40 + i, pad=2))
        s.out, s.ws = _out(s), _ws(d)
        kb = pu.page_bounds(torch.nan_to_num(s.kc))
        s.kb = kb
        s.dkb = kb.cuda()
        s.sel = torch.full((s.T, Hkv, 5), -7, dtype=torch.int32, device="cuda")
        s.ws2 = torch.empty(m.attn_page_select_workspace_bytes(s.T, Hkv, s.max_pages),
                            dtype=torch.uint8, device="cuda")
        s.out2 = _out(s)
        torch.cuda.synchronize()

        def step(s=s):
            _attn(s, *s.out, s.ws)
            m.attn_page_select(s.dq, s.dkb, s.dtable, s.dcu, s.dseq, s.sel, s.ps, 1, 2, s.ws2)
            _attn(s, *s.out2, s.ws, sel=s.sel)

        with torch.cuda.stream(streams[i]):
            step()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=streams[i]):
                step()
        steps.append(s)
        graphs.append(g)
    for round_ in range(3):
        for s in steps:
            s.q = torch.randn(s.q.shape, generator=torch.Generator().manual_seed(round_)).bfloat16()
            s.dq.copy_(s.q)
            for x in (*s.out, *s.out2):
                x.fill_(-77)
            s.sel.fill_(-7)
        torch.cuda.synchronize()
        for _ in range(5):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        assert m.attn_status() == 0
        for s in steps:
            pu.check_attn(s, s.out[0].cpu(), s.out[1].cpu(), pu.ref_attn(s), "replayed")
            want = pu.ref_select(s, s.kb, 5, 1, 2)
            assert torch.equal(s.sel.cpu(), want)
            pu.check_attn(s, s.out2[0].cpu(), s.out2[1].cpu(), pu.ref_attn(s, sel=want), "replayed")


def test_two_calls_at_once_without_graphs():
    s = [_upload(pu.make_step(n, c, 8, 2, 128, 32, seed=i))
         for i, (n, c) in enumerate([([1, 1], [3000, 900]), ([200], [500]), ([4, 4, 4], [50, 60, 3000])])]
    out, ws = [_out(x) for x in s], [_ws(128) for _ in s]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, o, w, st in zip(s, out, ws, streams):
            _attn(x, *o, w, stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert gpu_util.ea().attn_status() == 0
    for x, o in zip(s, out):
        pu.check_attn(x, o[0].cpu(), o[1].cpu(), pu.ref_attn(x), "side by side")


def test_nan_keys_stay_within_their_rows():
    """A NaN key makes NaN of the rows that see it, and its page is one that select chooses."""
    m = gpu_util.ea()
    for new in ([1, 1], [3, 200]):
        s = pu.make_step(new, [700, 60], 4, 2, 128, 32, seed=9)
        clean = pu.ref_attn(s)
        bad_page = s.table[0, 3].item()
        s.kc[bad_page, 1, 5, 0] = float("nan")          # K/V head 1 of sequence 0
        o, lse = _out(_upload(s))
        _attn(s, o, lse, _ws(128))
        assert m.attn_status() == 0
        o, lse = o.cpu(), lse.cpu()
        hit = torch.zeros(o.shape[:2], dtype=torch.bool)
        hit[:new[0], 2:] = True
        assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
        good = ~hit
        assert ((o[good].double() - clean[0][good]).abs() <= clean[2][good]).all()
        assert ((lse[good].double() - clean[1][good]).abs() <= clean[3][good]).all()
        kb = pu.page_bounds(torch.where(torch.isnan(s.kc), 0, s.kc))
        kb[bad_page, 1, :, 0] = float("nan")
        sel = torch.full((s.T, 2, 3), -7, dtype=torch.int32, device="cuda")
        ws = torch.empty(m.attn_page_select_workspace_bytes(s.T, 2, s.max_pages), dtype=torch.uint8,
                         device="cuda")
        m.attn_page_select(s.dq, kb.cuda(), s.dtable, s.dcu, s.dseq, sel, 32, 0, 1, ws)
        assert m.attn_status() == 0
        assert (sel[:new[0], 1] == 3).any(-1).all()


@pytest.mark.parametrize("new,ctx,Hq,Hkv,d,ps,K,first,last", [
    ([40, 30], [900, 2000], 8, 1, 64, 16, 20, 0, 2), ([19, 15, 19], [4255, 1918, 2622], 8, 1, 64, 128, 15, 0, 2),
    ([70], [1100], 32, 1, 64, 16, 30, 0, 0), ([3] * 30, [200] * 30, 4, 4, 128, 16, 5, 1, 1),
    ([150], [20], 5, 5, 64, 16, 6, 0, 1), ([65, 1, 64], [700, 30, 0], 16, 1, 128, 32, 9, 0, 1),
    ([9], [5000], 33, 1, 64, 16, 60, 2, 2), ([2, 2, 2], [600, 700, 1100], 64, 1, 64, 16, 11, 0, 0),
])
def test_select_of_many_rows(new, ctx, Hq, Hkv, d, ps, K, first, last):
    """Several rounds of rows against one tile of pages, several sequences in a tile of rows."""
    m = gpu_util.ea()
    s = _upload(pu.make_step(new, ctx, Hq, Hkv, d, ps, seed=K, pad=1, poison=False))
    kb = pu.page_bounds(s.kc)
    sel = torch.full((s.T, Hkv, K), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(m.attn_page_select_workspace_bytes(s.T, Hkv, s.max_pages), dtype=torch.uint8,
                     device="cuda")
    m.attn_page_select(s.dq, kb.cuda(), s.dtable, s.dcu, s.dseq, sel, ps, first, last, ws)
    assert m.attn_status() == 0
    assert torch.equal(sel.cpu(), pu.ref_select(s, kb, K, first, last))


@pytest.mark.parametrize("d,Hq,T", [(64, 1, 1), (128, 4, 1), (128, 1, 40)])
@pytest.mark.parametrize("small", ["q", "bounds", "both"])
def test_select_of_very_small_numbers(d, Hq, T, small):
    """Squares of q or of the bounds that are 0 in 32 bits: the choice is still the exact one. Pages 1
    and 3 score 1 + 2^-26 and 1 in units of the largest product, which 32-bit sums do not tell apart."""
    m = gpu_util.ea()
    s = _upload(pu.make_step([T], [16 * 6], Hq, 1, d, 16, seed=1, poison=False))
    sq, sb = {"q": (-80, 10), "bounds": (0, -80), "both": (-70, -40)}[small]
    q = torch.full((T, Hq, d), 2.0 ** sq).bfloat16()
    kb = torch.zeros((s.num_pages, 1, 2, d))
    for lp, low in ((1, 0.0), (3, 2.0 ** -26)):
        kb[s.table[0, lp].long(), 0, :, 0] = 2.0 ** sb
        kb[s.table[0, lp].long(), 0, :, 1] = 2.0 ** sb * low
    kb = kb.bfloat16()
    s.q = q
    sel = torch.full((T, 1, 1), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(m.attn_page_select_workspace_bytes(T, 1, s.max_pages), dtype=torch.uint8,
                     device="cuda")
    m.attn_page_select(q.cuda(), kb.cuda(), s.dtable, s.dcu, s.dseq, sel, 16, 0, 0, ws)
    assert m.attn_status() == 0
    want = pu.ref_select(s, kb, 1, 0, 0)
    assert (want == 3).all()
    assert torch.equal(sel.cpu(), want)


def test_long_batches_of_sequences():
    """More sequences than a CTA has threads."""
    new = [1 if i % 3 else 0 for i in range(1300)]
    s = _upload(pu.make_step(new, [i % 50 for i in range(1300)], 2, 1, 64, 16, seed=2, extra_pages=1))
    o, lse = _out(s)
    _attn(s, o, lse, _ws(64))
    assert gpu_util.ea().attn_status() == 0
    pu.check_attn(s, o.cpu(), lse.cpu(), pu.ref_attn(s), "1300 sequences")


def test_serving_under_the_index_checking_build():
    spec = importlib.util.spec_from_file_location(
        "exact_attn_cuda_build", os.path.join(ROOT, "exact_io_aware_70_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    env = dict(os.environ, EXACT_ATTN_LIB=build.build(debug=True))
    out = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m",
                          "gpu", "tests/test_gpu_serving.py"], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=1800)
    assert out.returncode == 0, out.stdout[-4000:] + out.stderr[-2000:]
    assert " passed" in out.stdout
