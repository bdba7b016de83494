"""Calls of the serving operators at the edges of what their documentation allows."""
from concurrent.futures import ThreadPoolExecutor
from types import SimpleNamespace

import pytest
import torch

from tests import gpu_util, paged_util as pu

pytestmark = pytest.mark.gpu


def _select(s, kb, K, ps, first=0, last=0):
    m = gpu_util.ea()
    sel = torch.full((s.T, s.Hkv, K), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(m.attn_page_select_workspace_bytes(s.T, s.Hkv, s.max_pages),
                     dtype=torch.uint8, device="cuda")
    m.attn_page_select(s.q.cuda(), kb.cuda(), s.table.cuda(), s.cu.cuda(), s.seq.cuda(), sel, ps,
                       first, last, ws)
    return sel.cpu(), m.attn_status()


@pytest.mark.parametrize("T,Hq,ctx", [(1, 1, 300), (1, 4, 1500), (70, 4, 300), (3, 4, 9000)])
@pytest.mark.parametrize("zero", ["q", "bounds"])
def test_select_nan_page_among_zero_scores(T, Hq, ctx, zero):
    """All scores are 0 (of q, or of the bounds) but one page's, which is NaN: that page ranks above
    the others, which follow from the lowest up."""
    s = pu.make_step([T], [ctx], Hq, 1, 128, 16, seed=3, poison=False)
    kb = pu.page_bounds(s.kc)
    if zero == "q":
        s.q = torch.zeros_like(s.q)
    else:
        kb = torch.zeros_like(kb)
    kb[s.table[0, 11].long(), 0, :, 5] = float("nan")
    sel, status = _select(s, kb, 3, 16)
    assert status == 0
    assert (sel == torch.tensor([0, 1, 11], dtype=torch.int32)).all()


@pytest.mark.parametrize("T,ctx", [(1, 300), (1, 3000), (20, 300)])
def test_select_infinite_bounds_on_the_side_not_taken(T, ctx):
    """An infinite bound counts only where q's sign takes it: the choice is still the definition's."""
    s = pu.make_step([T], [ctx], 2, 1, 64, 16, seed=4, poison=False)
    s.q[:, :, 7] = s.q[:, :, 7].abs() + 1
    s.q[:, :, 9] = -s.q[:, :, 9].abs() - 1
    kb = pu.page_bounds(s.kc)
    for i in (2, 5, 6):
        kb[s.table[0, i].long(), 0, 0, 7] = -float("inf")
        kb[s.table[0, i].long(), 0, 1, 9] = float("inf")
    sel, status = _select(s, kb, 4, 16)
    assert status == 0
    assert torch.equal(sel, pu.ref_select(s, kb, 4, 0, 0))


@pytest.mark.parametrize("what", ["long", "negative", "past_rows", "descending", "before_rows"])
@pytest.mark.parametrize("new", [1, 40])
def test_select_reports_bad_lengths_and_offsets(what, new):
    """Lengths and offsets out of range are clamped as the attention clamps them, and reported; all
    table entries are good here, so nothing else sets the status."""
    m = gpu_util.ea()
    s = pu.make_step([new] * 3, [100 - new] * 3, 4, 2, 64, 16, seed=new, pad=0, poison=False,
                     extra_pages=0)
    kb = pu.page_bounds(s.kc)
    if what == "long":          # a table of 7 pages holds 112 tokens
        s.seq[1], s.lens[1] = 10 ** 6, 112
    if what == "negative":
        s.seq[1], s.lens[1] = -3, 0
    if what == "past_rows":
        s.cu[3] = 10 ** 6
    if what == "before_rows":
        s.cu[0] = -2            # the first sequence's rows still end where they did
    if what == "descending":
        s.cu[1] = s.cu[2] + 1
    good = s.cu.clone()
    sel, status = _select(s, kb, 3, 16, 0, 1)
    assert status == m.ATTN_ERR_BAD_INDEX and m.attn_status() == 0
    if what == "descending":    # whose rows these are is not defined
        return
    s.cu = torch.tensor([0, new, 2 * new, 3 * new], dtype=torch.int32)
    assert torch.equal(sel, pu.ref_select(s, kb, 3, 0, 1))
    s.cu = good
    o, lse = (torch.full((s.T, s.Hq, s.d), -77, dtype=torch.bfloat16, device="cuda"),
              torch.full((s.T, s.Hq), -77, dtype=torch.float32, device="cuda"))
    ws = torch.empty(m.attn_fwd_paged_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    m.attn_sparse_paged(s.q.cuda(), s.kc.cuda(), s.vc.cuda(), s.table.cuda(), s.cu.cuda(),
                        s.seq.cuda(), sel.cuda(), o, lse, s.scale, ws)
    assert m.attn_status() == m.ATTN_ERR_BAD_INDEX
    s.cu = torch.tensor([0, new, 2 * new, 3 * new], dtype=torch.int32)
    pu.check_attn(s, o.cpu(), lse.cpu(), pu.ref_attn(s, sel=sel), "the same positions")


@pytest.mark.parametrize("kind", ["flat", "normal", "exponents", "cancel"])
@pytest.mark.parametrize("T,Hq,d", [(1, 4, 128), (3, 1, 64), (70, 4, 128), (40, 8, 64)])
def test_select_scores_are_within_their_error_bound(kind, T, Hq, d):
    """The fp32 scores and the error bounds that a call leaves in its workspace (rows that may take all
    their pages are not ranked further) against scores in 64 bits. A bound is no less than what steps
    of four terms may lose: 2 d / 4 steps cut off 4 + 2 numbers each below 2^-23 of at most |q| |b|;
    the two norms' own sums are off by 2^-15."""
    m = gpu_util.ea()
    s = pu.make_step([T], [1500], Hq, 1, d, 16, seed=T + d, poison=False)
    pages = -(-s.lens[0] // 16)
    g = torch.Generator().manual_seed(7)
    kb = pu.page_bounds(s.kc).double()
    q = s.q.double()
    if kind == "flat":              # equal squares: the bound is as tight as it gets
        q, kb = torch.sign(q) * 1.0078125, torch.sign(kb) * 1.0078125
    if kind == "exponents":
        q = q * 2.0 ** torch.randint(-30, 30, q.shape, generator=g)
        kb = kb * 2.0 ** torch.randint(-30, 30, kb.shape, generator=g)
    if kind == "cancel":            # large terms of both signs, whose sum is small
        q = q.abs()
        kb[..., 0::2], kb[..., 1::2] = kb[..., 0::2].abs() + 100, -kb[..., 1::2].abs() - 100
    s.q, kb = q.bfloat16(), kb.bfloat16()
    q, b = s.q.double(), kb[s.table[0, :pages].long(), 0].double()        # [pages, 2, d]
    want = torch.where(q[:, :, None] >= 0, q[:, :, None] * b[:, 1], q[:, :, None] * b[:, 0]).sum(-1)
    want = want.amax(1)                                                   # [T, pages]
    K = s.max_pages
    ws = torch.zeros(m.attn_page_select_workspace_bytes(T, 1, s.max_pages), dtype=torch.uint8,
                     device="cuda")
    sel = torch.full((T, 1, K), -7, dtype=torch.int32, device="cuda")
    m.attn_page_select(s.q.cuda(), kb.cuda(), s.table.cuda(), s.cu.cuda(), s.seq.cuda(), sel, 16, 0,
                       0, ws)
    assert m.attn_status() == 0
    ws = ws.cpu()
    tiles = -(-s.max_pages // 64)
    at = -(-T * s.max_pages * 8 // 256) * 256
    got = ws[:T * s.max_pages * 8].view(torch.float32).reshape(T, 2 * s.max_pages)[:, :pages].double()
    err = ws[at:at + T * tiles * 4].view(torch.float32).reshape(T, tiles).double()
    pos = s.lens[0] - T + torch.arange(T)
    for tile in range(tiles):
        part = slice(64 * tile, min(64 * tile + 64, pages))
        if part.start >= pages:
            continue
        norm = (q ** 2).sum(-1).sqrt().amax(1) * (b[part] ** 2).sum((1, 2)).sqrt().amax()
        least = (2 * d // 4) * 6 * 2.0 ** -23 * norm * (1 - 2.0 ** -15)
        seen = torch.arange(part.start, part.stop)[None] <= pos[:, None] // 16
        off = torch.where(seen, (got[:, part] - want[:, part]).abs(), 0.0).amax(1)
        assert (off <= err[:, tile]).all(), (off / err[:, tile]).max()
        assert (err[:, tile] >= least).all(), (err[:, tile] / least).min()


def test_tables_largest_number_of_rows():
    """2^30 rows, and sequences that ask for 2^30 tokens each: the first gets them all (two sums of
    2^30 do not fit 32 bits with a sign)."""
    m = gpu_util.ea()
    n, ps, B = 2 ** 30, 1024, 40
    pages = n // ps
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, new = torch.zeros(B, **i32), torch.full((B,), n, **i32)
    new[3] = 7
    head, seq, cu = torch.zeros(1, **i32), torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
    table = torch.full((B, pages), -5, **i32)
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    m.attn_page_tables(ctx, new, torch.arange(pages, **i32), head, head, table, seq, cu, slots, ps,
                       pages)
    assert m.attn_status() == m.ATTN_ERR_BAD_INDEX          # the others' tokens are cut off
    assert seq.tolist() == [n] + [0] * (B - 1) and cu.tolist() == [0] + [n] * B
    assert head.item() == pages
    assert torch.equal(table[0], torch.arange(pages, **i32)) and (table[1:] == -5).all()
    for at in range(0, n, n // 8):
        assert torch.equal(slots[at:at + n // 8], torch.arange(at, at + n // 8, device="cuda"))


def _attn(s, causal=True, sel=None):
    m = gpu_util.ea()
    o = torch.full((s.T, s.Hq, s.d), -77, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.T, s.Hq), -77, dtype=torch.float32, device="cuda")
    ws = torch.empty(m.attn_fwd_paged_workspace_bytes(s.d), dtype=torch.uint8, device="cuda")
    a = (s.q.cuda(), s.kc.cuda(), s.vc.cuda(), s.table.cuda(), s.cu.cuda(), s.seq.cuda())
    if sel is None:
        m.attn_fwd_paged(*a, o, lse, causal, s.scale, ws)
    else:
        m.attn_sparse_paged(*a, sel.cuda(), o, lse, s.scale, ws)
    return o.cpu(), lse.cpu(), m.attn_status()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("N,H,d,ps", [(1, 3, 64, 16), (700, 4, 128, 64), (1025, 2, 64, 32)])
def test_prompt_agrees_with_the_dense_forward(N, H, d, ps, causal):
    """A whole prompt, nothing cached before: attn_fwd and attn_fwd_paged are both within the bounds
    of the 64-bit definition, and so within twice those of each other."""
    m = gpu_util.ea()
    s = pu.make_step([N], [0], H, H, d, ps, seed=N + d)
    o, lse, status = _attn(s, causal)
    assert status == 0
    ref = pu.ref_attn(s, causal)
    pu.check_attn(s, o, lse, ref, "paged")
    k, v, _ = pu.seq_kv(s, 0)
    q = s.q.transpose(0, 1)[None].contiguous().cuda()
    od = torch.empty_like(q)
    ld = torch.empty((1, H, N), dtype=torch.float32, device="cuda")
    m.attn_fwd(q, k.bfloat16()[None].contiguous().cuda(), v.bfloat16()[None].contiguous().cuda(), od,
               ld, causal, s.scale)
    assert m.attn_status() == 0
    od, ld = od[0].transpose(0, 1).cpu(), ld[0].T.cpu()
    pu.check_attn(s, od, ld, ref, "dense")
    assert ((o.double() - od.double()).abs() <= 2 * ref[2]).all()
    assert ((lse.double() - ld.double()).abs() <= 2 * ref[3]).all()


def test_append_bounds_beyond_31_bits():
    """The last slot of a cache of more than 2^31 elements: both bounds are those of the whole page,
    and no other page's change."""
    m = gpu_util.ea()
    ps, Hkv, d = 1024, 8, 128
    pages = 2 ** 31 // (ps * Hkv * d) + 3
    kc, vc = (torch.empty((pages, Hkv, ps, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc[-1] = torch.randn((Hkv, ps, d), device="cuda").bfloat16()
    kb = torch.full((pages, Hkv, 2, d), 3.0, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.randn((1, Hkv, d), device="cuda").bfloat16() for _ in range(2))
    m.attn_paged_append(k, v, torch.tensor([pages * ps - 1], device="cuda"), kc, vc, kb)
    assert m.attn_status() == 0
    assert torch.equal(kc[-1, :, -1], k[0]) and torch.equal(vc[-1, :, -1], v[0])
    assert torch.equal(kb[-1, :, 0], kc[-1].amin(1)) and torch.equal(kb[-1, :, 1], kc[-1].amax(1))
    assert (kb[:-1] == 3).all()


@pytest.mark.parametrize("B,Hkv,new", [(3, 1, 1), (3, 2, 5), (40, 1, 1)])
def test_choice_right_behind_the_tables(B, Hkv, new):
    """A captured step whose page choice follows the kernel that writes its lengths, offsets and tables:
    replay after replay the choice goes by that replay's, although it looks rows up early."""
    m = gpu_util.ea()
    ps, d, K, max_pages, replays = 16, 64, 4, 24, 60
    num_pages = B * max_pages + 7
    g = torch.Generator().manual_seed(B + new)
    free = torch.randperm(num_pages, generator=g).tolist()
    kb = torch.randn((num_pages, Hkv, 2, d), generator=g)
    kb = torch.stack([kb.amin(2), kb.amax(2)], 2).bfloat16()
    q = torch.randn((B * new, 2 * Hkv, d), generator=g).bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    start = [7 * b % 30 for b in range(B)]
    table = [[-1] * max_pages for _ in range(B)]
    for b in range(B):
        for i in range(-(-start[b] // ps)):
            table[b][i] = free.pop()
    lens, dnew = torch.tensor(start, **i32), torch.full((B,), new, **i32)
    dtab, dfree, head = torch.tensor(table, **i32), torch.tensor(free, **i32), torch.zeros(1, **i32)
    cu, slots = torch.zeros(B + 1, **i32), torch.zeros(B * new, dtype=torch.int64, device="cuda")
    dq, dkb = q.cuda(), kb.cuda()
    sel = torch.full((B * new, Hkv, K), -7, **i32)
    ws = torch.empty(m.attn_page_select_workspace_bytes(B * new, Hkv, max_pages), dtype=torch.uint8,
                     device="cuda")
    seen = torch.full((replays, B * new, Hkv, K), -9, **i32)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            m.attn_page_tables(lens, dnew, dfree, head, head, dtab, lens, cu, slots, ps, num_pages)
            m.attn_page_select(dq, dkb, dtab, cu, lens, sel, ps, 1, 1, ws)
        for i in range(replays):
            graph.replay()
            seen[i].copy_(sel)
        assert m.attn_status() == 0
    seen = seen.cpu()
    at, taken = list(start), 0
    for i in range(replays):
        table, at, wcu, _, taken, fine = pu.ref_tables(at, [new] * B, free, taken, table, B * new, ps,
                                                       num_pages)
        assert fine
        s = SimpleNamespace(T=B * new, Hq=2 * Hkv, Hkv=Hkv, B=B, new=[new] * B, lens=at, ps=ps, q=q,
                            cu=torch.tensor(wcu), table=torch.tensor(table), num_pages=num_pages)
        assert torch.equal(seen[i], pu.ref_select(s, kb, K, 1, 1)), f"replay {i}"


@pytest.mark.parametrize("ps,K,Hq", [(16, 480, 4), (64, 480, 1), (128, 480, 8), (256, 240, 2),
                                     (1024, 60, 4)])
def test_sparse_longest_lists(ps, K, Hq):
    """As many pages in a row's list as the call takes, all of them there, in any order."""
    m = gpu_util.ea()
    s = pu.make_step([1, 2], [(K + 3) * ps - 5, 40], Hq, 1, 64, ps, seed=K + ps)
    g = torch.Generator().manual_seed(ps)
    sel = torch.full((3, 1, K), -1, dtype=torch.int32)
    sel[0, 0] = torch.randperm(K + 3, generator=g)[:K].int()
    sel[1, 0, K - 1], sel[2, 0, 0] = 0, 0
    o, lse, status = _attn(s, sel=sel)
    assert status == 0
    pu.check_attn(s, o, lse, pu.ref_attn(s, sel=sel), "long lists")
    with pytest.raises(m.AttnError):
        _attn(s, sel=torch.full((3, 1, K + 1), -1, dtype=torch.int32))


def test_select_largest_table():
    """16384 pages, the most that the choice takes."""
    s = pu.make_step([2], [16384 * 16 - 2], 2, 1, 64, 16, seed=8, poison=False, extra_pages=0)
    assert s.max_pages == 16384
    kb = pu.page_bounds(s.kc)
    sel, status = _select(s, kb, 40, 16, 1, 2)
    assert status == 0 and torch.equal(sel, pu.ref_select(s, kb, 40, 1, 2))
    s.table, s.max_pages = torch.cat([s.table, s.table[:, :1]], 1), 16385
    with pytest.raises(gpu_util.ea().AttnError):
        _select(s, kb, 40, 16, 1, 2)


@pytest.mark.parametrize("new,ctx", [([1, 1, 1], [700, 15, 16]), ([4, 0, 3], [300, 9, 2000]),
                                     ([1, 2], [12000, 9000])])
def test_mostly_padding_rows(new, ctx):
    """A step in a buffer made for far more rows than it has."""
    s = pu.make_step(new, ctx, 8, 2, 128, 32, seed=3, pad=3000)
    o, lse, status = _attn(s)
    assert status == 0
    pu.check_attn(s, o, lse, pu.ref_attn(s), "padded")
    kb = pu.page_bounds(torch.nan_to_num(s.kc))
    sel, status = _select(s, kb, 5, 32, 1, 1)
    assert status == 0 and torch.equal(sel, pu.ref_select(s, kb, 5, 1, 1))
    o, lse, status = _attn(s, sel=sel)
    assert status == 0
    pu.check_attn(s, o, lse, pu.ref_attn(s, sel=sel), "padded, chosen pages")


def test_captured_behind_a_join():
    """A captured step that follows work on two streams, a copy and a fill (the launches overlap only
    what they may)."""
    m = gpu_util.ea()
    s = pu.make_step([1, 30], [900, 77], 8, 2, 64, 16, seed=6, pad=1)
    kb = pu.page_bounds(torch.nan_to_num(s.kc))
    i32 = dict(dtype=torch.int32, device="cuda")
    src = (s.q.cuda(), s.kc.cuda(), s.vc.cuda())
    q, kc, vc = (torch.zeros_like(x) for x in src)
    table, cu, seq, dkb = s.table.cuda(), s.cu.cuda(), s.seq.cuda(), kb.cuda()
    o, o2 = (torch.zeros((s.T, 8, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse, lse2 = (torch.zeros((s.T, 8), dtype=torch.float32, device="cuda") for _ in range(2))
    sel = torch.zeros((s.T, 2, 6), **i32)
    ws = torch.empty(m.attn_fwd_paged_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(m.attn_page_select_workspace_bytes(s.T, 2, s.max_pages), dtype=torch.uint8,
                      device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            kc.copy_(src[1])
            vc.copy_(src[2])
        q.copy_(src[0])
        for x in (o, o2, lse, lse2):
            x.fill_(-77)
        sel.fill_(-7)
        main.wait_stream(side)
        m.attn_fwd_paged(q, kc, vc, table, cu, seq, o, lse, True, s.scale, ws)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            m.attn_page_select(q, dkb, table, cu, seq, sel, 16, 1, 1, ws2)
        main.wait_stream(side)
        m.attn_sparse_paged(q, kc, vc, table, cu, seq, sel, o2, lse2, s.scale, ws)
        kc.zero_()
        q.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert m.attn_status() == 0
    pu.check_attn(s, o.cpu(), lse.cpu(), pu.ref_attn(s), "joined")
    want = pu.ref_select(s, kb, 6, 1, 1)
    assert torch.equal(sel.cpu(), want)
    pu.check_attn(s, o2.cpu(), lse2.cpu(), pu.ref_attn(s, sel=want), "joined, chosen pages")


def test_calls_from_several_threads():
    """Host threads that call at the same time, each on a stream and a workspace of its own; the call
    is the first that a thread makes of CUDA at all."""
    m = gpu_util.ea()
    steps = [pu.make_step([1, 5, 40][i % 3:][:2] + [1], [300, 70, 900][:len([1, 5, 40][i % 3:][:2]) + 1],
                          4, 2, 64, 16, seed=i) for i in range(6)]
    data = [tuple(x.cuda() for x in (s.q, s.kc, s.vc, s.table, s.cu, s.seq)) for s in steps]
    outs = [(torch.full((s.T, 4, 64), -77, dtype=torch.bfloat16, device="cuda"),
             torch.full((s.T, 4), -77, dtype=torch.float32, device="cuda"),
             torch.empty(m.attn_fwd_paged_workspace_bytes(64), dtype=torch.uint8, device="cuda"))
            for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()

    def work(i):
        o, lse, ws = outs[i]
        for _ in range(20):
            m.attn_fwd_paged(*data[i], o, lse, True, steps[i].scale, ws,
                             stream=streams[i].cuda_stream)

    with ThreadPoolExecutor(len(steps)) as pool:
        list(pool.map(work, range(len(steps))))
    torch.cuda.synchronize()
    assert m.attn_status() == 0
    for s, (o, lse, _) in zip(steps, outs):
        pu.check_attn(s, o.cpu(), lse.cpu(), pu.ref_attn(s), "threads")


@pytest.mark.parametrize("what", ["fwd_paged", "sparse", "select", "append", "tables", "fwd", "bwd"])
def test_first_call_of_a_thread(what):
    """Every kind of call as the first that a host thread makes of CUDA."""
    m = gpu_util.ea()
    s = pu.make_step([3, 1], [60, 5], 2, 2, 64, 16, seed=2)
    i32 = dict(dtype=torch.int32, device="cuda")
    q, kc, vc, table, cu, seq = (x.cuda() for x in (s.q, s.kc, s.vc, s.table, s.cu, s.seq))
    o, lse = torch.empty_like(q), torch.empty((4, 2), dtype=torch.float32, device="cuda")
    sel = torch.zeros((4, 2, 3), **i32)
    kb = pu.page_bounds(torch.nan_to_num(s.kc)).cuda()
    ws, ws2 = (torch.empty(n, dtype=torch.uint8, device="cuda")
               for n in (m.attn_fwd_paged_workspace_bytes(64),
                         m.attn_page_select_workspace_bytes(4, 2, s.max_pages)))
    slots, head = torch.arange(4, device="cuda"), torch.zeros(1, **i32)
    ones, free, offsets = torch.ones(2, **i32), torch.arange(9, **i32), torch.zeros(3, **i32)
    dense = [torch.randn((1, 2, 40, 64), device="cuda").bfloat16() for _ in range(8)]
    dl = torch.zeros((1, 2, 40), dtype=torch.float32, device="cuda")
    wb = torch.empty(m.attn_bwd_workspace_bytes(1, 2, 40, 64), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    call = {
        "fwd_paged": lambda: m.attn_fwd_paged(q, kc, vc, table, cu, seq, o, lse, True, s.scale, ws,
                                              stream=stream),
        "sparse": lambda: m.attn_sparse_paged(q, kc, vc, table, cu, seq, sel, o, lse, s.scale, ws,
                                              stream=stream),
        "select": lambda: m.attn_page_select(q, kb, table, cu, seq, sel, 16, 0, 1, ws2, stream=stream),
        "append": lambda: m.attn_paged_append(q, q, slots, kc, vc, kb, stream=stream),
        "tables": lambda: m.attn_page_tables(seq, ones, free, head, head, table, seq, offsets, slots,
                                             16, s.num_pages, stream=stream),
        "fwd": lambda: m.attn_fwd(*dense[:4], dl, True, s.scale, stream=stream),
        "bwd": lambda: m.attn_bwd(*dense[:5], dl, *dense[5:], True, s.scale, wb, stream=stream),
    }[what]
    with ThreadPoolExecutor(1) as pool:
        pool.submit(call).result()
    assert m.attn_status() == 0


FORMS = [([1, 1], 4), ([5, 2], 8), ([3, 90], 4), ([300], 2), ([2], 40)]   # 16, 32 columns, 128-row tiles


@pytest.mark.parametrize("new,G", FORMS)
@pytest.mark.parametrize("sparse", [False, True])
def test_queries_that_are_not_finite_stay_in_their_rows(new, G, sparse):
    """NaN and infinite query rows make NaN of their own outputs alone; those of padding rows of none."""
    s = pu.make_step(new, [700, 40][:len(new)], 2 * G, 2, 64, 16, seed=G, pad=3)
    sel = None
    if sparse:
        sel = torch.arange(6, dtype=torch.int32).expand(s.T, 2, 6).clone()
        for b in range(s.B):
            rows = slice(int(s.cu[b]), int(s.cu[b + 1]))
            sel[rows][sel[rows] * 16 >= s.lens[b]] = -1
    ref = pu.ref_attn(s, sel=sel)
    end = int(s.cu[-1])
    s.q[end:] = float("nan")
    s.q[end + 1] = float("inf")
    bad = torch.zeros((s.T, 2 * G), dtype=torch.bool)
    for t, h, x in ((0, 0, float("nan")), (end - 1, 2 * G - 1, float("inf"))):
        s.q[t, h, 3] = x
        bad[t, h] = True
    o, lse, status = _attn(s, sel=sel)
    assert status == 0
    assert (o[end:] == -77).all() and (lse[end:] == -77).all()
    assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
    good = ~bad
    good[end:] = False
    assert ((o[good].double() - ref[0][good]).abs() <= ref[2][good]).all()
    assert ((lse[good].double() - ref[1][good]).abs() <= ref[3][good]).all()


@pytest.mark.parametrize("new,G", FORMS)
def test_keys_of_minus_infinity_weigh_nothing(new, G):
    """Scores of -infinity among finite ones: as if those keys were not there. The first keys of a
    sequence and the last whole tile before a row's own position, so that a tile can be all of them."""
    s = pu.make_step(new, [700, 40][:len(new)], 2 * G, 2, 64, 16, seed=G + 1)
    s.q[:, :, 0] = s.q[:, :, 0].abs() + 0.5
    keep = [torch.ones(ln, dtype=torch.bool) for ln in s.lens]
    keep[0][:140] = False
    keep[0][256:512] = False
    clean = [pu.seq_kv(s, b)[0] for b in range(s.B)]
    for j in torch.nonzero(~keep[0])[:, 0].tolist():
        s.kc[s.table[0, j // 16], :, j % 16, 0] = -float("inf")
    o, lse, status = _attn(s)
    assert status == 0
    for b in range(s.B):
        n, ln = s.new[b], s.lens[b]
        v = pu.seq_kv(s, b)[1]
        rows = slice(int(s.cu[b]), int(s.cu[b]) + n)
        seen = (torch.arange(ln)[None] <= (ln - n + torch.arange(n))[:, None]) & keep[b]
        for h in range(2 * G):
            q, k, vv = s.q[rows, h].double(), clean[b][h // G], v[h // G]
            score = torch.where(seen, q @ k.T * s.scale, -torch.inf)
            want = torch.logsumexp(score, 1)
            p = torch.exp(score - want[:, None])
            # (the bounds of ref_attn)
            e = torch.where(seen, q.abs() @ k.abs().T, 0.0).amax(1) * s.scale * 2 * 64 * 2.0 ** -24
            tol = 2.0 ** -8 * (p @ vv).abs() + (2.0 ** -8 + 2 * e + 2.0 ** -18)[:, None] * (p @ vv.abs())
            assert ((o[rows, h].double() - p @ vv).abs() <= tol).all()
            assert ((lse[rows, h].double() - want).abs() <= e + 2.0 ** -18 * (1 + want.abs())).all()


@pytest.mark.parametrize("at", [0, 127, 128, 2999])
def test_select_checks_every_sequence_of_a_long_batch(at):
    """3000 sequences, of which one has a length out of range, and only a few rows among them."""
    m = gpu_util.ea()
    new = [1 if b % 500 == 0 else 0 for b in range(3000)]
    s = pu.make_step(new, [b % 40 for b in range(3000)], 2, 1, 64, 16, seed=1, poison=False)
    kb = pu.page_bounds(s.kc)
    want = pu.ref_select(s, kb, 2, 0, 1)
    sel, status = _select(s, kb, 2, 16, 0, 1)
    assert status == 0 and torch.equal(sel, want)
    s.seq[at] = -1
    sel, status = _select(s, kb, 2, 16, 0, 1)
    assert status == m.ATTN_ERR_BAD_INDEX
    rows = [i for i, b in enumerate(range(0, 3000, 500)) if b != at]
    assert torch.equal(sel[rows], want[rows])
