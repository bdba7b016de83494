"""The serving operators on a paged cache, on the B200, against their plain 64-bit definitions."""
import pytest
import torch

from tests import gpu_util, paged_util as pu

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run_attn(s, causal=True, sel=None, ws=None):
    m = gpu_util.ea()
    o = torch.full((s.T, s.Hq, s.d), -77, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.T, s.Hq), -77, dtype=torch.float32, device="cuda")
    if ws is None:
        ws = torch.full((m.attn_fwd_paged_workspace_bytes(s.d),), 0xFF, dtype=torch.uint8,
                        device="cuda")
    q = s.q.cuda() if s.q.is_contiguous() else \
        s.q.as_strided((s.T, s.q.stride(0) // s.d, s.d), (s.q.stride(0), s.d, 1),
                       0).cuda()[:, 1:s.Hq + 1]
    assert q.stride(0) == s.q.stride(0)
    a = (q, s.kc.cuda(), s.vc.cuda(), s.table.cuda(), s.cu.cuda(), s.seq.cuda())
    if sel is None:
        m.attn_fwd_paged(*a, o, lse, causal, s.scale, ws)
    else:
        m.attn_sparse_paged(*a, sel.cuda(), o, lse, s.scale, ws)
    return o.cpu(), lse.cpu(), m.attn_status()


# ------------------------------------------------------------------- tables --
@pytest.mark.parametrize("B,ps,T_pad,head", [(1, 16, 0, 0), (3, 64, 5, 2), (40, 16, 1100, 7),
                                             (1030, 32, 3, 1), (2500, 128, 0, 0)])
def test_tables_match_definition(B, ps, T_pad, head):
    m = gpu_util.ea()
    g = torch.Generator().manual_seed(B + ps)
    ctx = torch.randint(0, 5 * ps, (B,), generator=g).tolist()
    new = torch.randint(0, 3 * ps if B < 100 else 4, (B,), generator=g).tolist()
    ctx[0], new[0] = ps, 1                     # a full page, then one token
    if B > 2:
        ctx[1], new[1], ctx[2], new[2] = 0, 0, 0, 2 * ps
    max_pages = 9
    num_pages = sum(-(-(c + n) // ps) for c, n in zip(ctx, new)) + head + 4
    perm = torch.randperm(num_pages, generator=g).tolist()
    table = [[perm.pop() if i < -(-c // ps) else -5 for i in range(max_pages)] for c in ctx]
    free = [-3] * head + perm
    T = max(1, sum(new) + T_pad)
    want = pu.ref_tables(ctx, new, free, head, table, T, ps, num_pages)
    assert want[-1]
    tab, fh, ho = _i32(table), _i32([head]), _i32([0])
    seq, cu = _i32([0] * B), _i32([0] * (B + 1))
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    m.attn_page_tables(_i32(ctx), _i32(new), _i32(free), fh, ho, tab, seq, cu, slots, ps, num_pages)
    assert m.attn_status() == 0
    assert tab.tolist() == want[0] and seq.tolist() == want[1] and cu.tolist() == want[2]
    assert slots.tolist() == want[3] and ho.item() == want[4]


def test_tables_in_place_and_captured():
    """Lengths and head updated in place; a captured step replayed goes on from the last one."""
    m = gpu_util.ea()
    ps, B, max_pages, F = 16, 5, 8, 64
    ctx, new = [0, 15, 16, 31, 7], [3, 1, 2, 0, 16]
    free = list(range(F - 1, -1, -1))
    table = [[-1] * max_pages for _ in range(B)]
    for b, c in enumerate(ctx):
        for i in range(-(-c // ps)):
            table[b][i] = 40 + 3 * b + i
    T = sum(new) + 2
    dctx, dnew, dfree, dhead, dtab = _i32(ctx), _i32(new), _i32(free), _i32([0]), _i32(table)
    cu = _i32([0] * (B + 1))
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")

    def step():
        m.attn_page_tables(dctx, dnew, dfree, dhead, dhead, dtab, dctx, cu, slots, ps, F)

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step()
    head = 0
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        table, ctx, wcu, wslots, head, fine = pu.ref_tables(ctx, new, free, head, table, T, ps, F)
        assert fine
        assert dtab.tolist() == table and dctx.tolist() == ctx and dhead.item() == head
        assert cu.tolist() == wcu and slots.tolist() == wslots
    assert m.attn_status() == 0


@pytest.mark.parametrize("what", ["free_list_short", "rows_short", "negative", "too_long", "bad_page",
                                  "bad_head"])
def test_tables_bad_values_are_reported(what):
    m = gpu_util.ea()
    ps, num_pages, max_pages = 16, 50, 4
    ctx, new = [10, 0, 20, 33], [20, 17, 5, 20]
    free, head, T = list(range(20, 50)), 0, 70
    if what == "free_list_short":
        free = free[:3]
    if what == "rows_short":
        T = 40
    if what == "negative":
        ctx[1], new[2] = -4, -1
    if what == "too_long":
        new[1] = 2 ** 31 - 1
    if what == "bad_page":
        free[1] = num_pages
    if what == "bad_head":
        head = 99
    table = [[5 * b + i if i < -(-max(c, 0) // ps) else -9 for i in range(max_pages)]
             for b, c in enumerate(ctx)]
    want = pu.ref_tables(ctx, new, free, head, table, T, ps, num_pages)
    assert not want[-1]
    tab, ho = _i32(table), _i32([0])
    seq, cu = _i32([0] * 4), _i32([0] * 5)
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    m.attn_page_tables(_i32(ctx), _i32(new), _i32(free), _i32([head]), ho, tab, seq, cu, slots, ps,
                       num_pages)
    assert m.attn_status() == m.ATTN_ERR_BAD_INDEX
    assert tab.tolist() == want[0] and seq.tolist() == want[1] and cu.tolist() == want[2]
    assert slots.tolist() == want[3] and ho.item() == want[4]


# ------------------------------------------------------------------- append --
@pytest.mark.parametrize("new,ctx,Hkv,d,ps,pad,strided", [
    ([1], [0], 1, 64, 16, 0, False), ([1, 1, 1], [15, 16, 40], 3, 128, 16, 2, True),
    ([5, 0, 40, 1], [62, 3, 0, 127], 2, 64, 64, 3, True), ([300], [77], 2, 128, 128, 0, False),
    ([700, 350], [10, 511], 32, 128, 512, 5, True), ([900, 130], [1, 6], 40, 64, 16, 0, False),
])
def test_append_matches_definition(new, ctx, Hkv, d, ps, pad, strided):
    m = gpu_util.ea()
    s = pu.make_step(new, ctx, Hkv, Hkv, d, ps, seed=sum(new) + ps, pad=pad)
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn((s.T, 2 * Hkv if strided else Hkv, d), generator=g).bfloat16()
            for _ in range(2))
    slots, wk, wv = [], s.kc.clone(), s.vc.clone()
    wb = torch.full((s.num_pages, Hkv, 2, d), 3.0).bfloat16()
    k_rows, v_rows = (k[:, Hkv:], v[:, Hkv:]) if strided else (k, v)
    for b in range(s.B):
        for j in range(ctx[b], ctx[b] + new[b]):
            slots.append(int(s.table[b, j // ps]) * ps + j % ps)
    for t, x in enumerate(slots):
        wk[x // ps, :, x % ps], wv[x // ps, :, x % ps] = k_rows[t], v_rows[t]
    last = {}
    for x in slots:
        last[x // ps] = x % ps
    for page, e in last.items():
        rows = wk[page, :, :e + 1].float()
        wb[page, :, 0], wb[page, :, 1] = rows.amin(1).bfloat16(), rows.amax(1).bfloat16()
    slots = torch.tensor(slots + [-1] * pad, device="cuda")
    kc, vc = s.kc.cuda(), s.vc.cuda()
    kb = torch.full((s.num_pages, Hkv, 2, d), 3.0).bfloat16().cuda()
    kd, vd = k.cuda(), v.cuda()
    if strided:
        kd, vd = kd[:, Hkv:], vd[:, Hkv:]
    m.attn_paged_append(kd, vd, slots, kc, vc, kb)
    assert m.attn_status() == 0
    bits = lambda x: x.cpu().view(torch.int16)  # noqa: E731  (NaN slots compare too)
    assert torch.equal(bits(kc), wk.view(torch.int16)) and torch.equal(bits(vc), wv.view(torch.int16))
    assert torch.equal(kb.cpu(), wb)
    kc2, vc2 = s.kc.cuda(), s.vc.cuda()          # without bounds: the same caches
    m.attn_paged_append(kd, vd, slots, kc2, vc2)
    assert m.attn_status() == 0
    assert torch.equal(bits(kc2), bits(kc)) and torch.equal(bits(vc2), bits(vc))


def test_append_skips_bad_slots_and_carries_nan_into_bounds():
    m = gpu_util.ea()
    ps, Hkv, d, pages = 16, 2, 64, 4
    k = torch.randn((5, Hkv, d), device="cuda").bfloat16()
    k[1, 0, 7] = float("nan")
    kc, vc = (torch.zeros((pages, Hkv, ps, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kb = torch.zeros((pages, Hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([16, 17, pages * ps, -8, 2 ** 40], device="cuda")
    m.attn_paged_append(k, k, slots, kc, vc, kb)
    assert m.attn_status() == m.ATTN_ERR_BAD_INDEX
    want = torch.zeros_like(kc)
    want[1, :, 0], want[1, :, 1] = k[0], k[1]
    assert torch.equal(kc.view(torch.int16), want.view(torch.int16))
    assert torch.isnan(kb[1, 0, :, 7]).all() and not torch.isnan(kb[1, 1]).any()
    ok = torch.ones(d, dtype=torch.bool)
    ok[7] = False
    assert torch.equal(kb[1, 0, 0][ok], torch.minimum(k[0, 0], k[1, 0])[ok])
    assert torch.all(kb[[0, 2, 3]] == 0)


# ---------------------------------------------------------------- attention --
ATTN = [  # new, ctx, Hq, Hkv, d, ps, pad, strided
    ([1], [0], 1, 1, 64, 16, 0, False),
    ([1], [127], 4, 1, 128, 64, 0, False),
    ([1, 1, 1], [128, 129, 700], 8, 2, 128, 16, 2, True),
    ([1, 0, 1], [5000, 4, 33], 32, 8, 128, 256, 1, True),
    ([1, 1], [3, 2049], 12, 12, 64, 1024, 0, False),
    ([3, 1, 6, 2], [100, 254, 0, 511], 28, 4, 128, 16, 3, True),
    ([9], [1500], 6, 2, 64, 32, 0, False),
    ([40, 17], [0, 130], 3, 1, 128, 128, 0, True),
    ([128], [0], 2, 2, 64, 64, 0, False),
    ([129, 127], [1, 128], 2, 1, 128, 64, 9, False),
    ([300, 1, 77], [333, 1000, 0], 8, 2, 128, 32, 0, True),
    ([700], [50], 5, 5, 64, 16, 0, False),
    ([257], [3000], 24, 8, 64, 512, 0, True),
    ([2, 5], [70, 1], 128, 1, 128, 16, 0, False),
    ([3], [200], 100, 1, 64, 64, 1, False),
    ([1] * 200, list(range(0, 1000, 5)), 4, 2, 64, 16, 0, False),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,Hq,Hkv,d,ps,pad,strided", ATTN)
def test_fwd_matches_definition(new, ctx, Hq, Hkv, d, ps, pad, strided, causal):
    s = pu.make_step(new, ctx, Hq, Hkv, d, ps, seed=sum(new) + sum(ctx), pad=pad, strided=strided)
    if not causal:   # every cached V is visible to every row: none may be left out
        assert not torch.isnan(pu.seq_kv(s, 0)[1]).any()
    o, lse, st = _run_attn(s, causal)
    assert st == 0
    pu.check_attn(s, o, lse, pu.ref_attn(s, causal), "fwd")


def test_fwd_rows_that_see_no_key():
    """More new tokens than cached keys: the first rows sit before the sequence (causal); and a
    sequence of length 0."""
    s = pu.make_step([200, 3, 5], [0, 0, 0], 4, 2, 128, 16, seed=3, len_override=[60, 0, 5])
    for causal in (True, False):
        o, lse, st = _run_attn(s, causal)
        assert st == 0
        pu.check_attn(s, o, lse, pu.ref_attn(s, causal), "no key")


@pytest.mark.parametrize("new", [1, 150])
def test_fwd_large_scores(new):
    """Scores up to several hundred, rising along the sequence (the reference maximum moves)."""
    s = pu.make_step([new], [600], 4, 2, 128, 32, seed=5)
    for i in range(-(-s.lens[0] // s.ps)):
        s.kc[s.table[0, i]] *= 0.5 * i
    o, lse, st = _run_attn(s)
    assert st == 0
    pu.check_attn(s, o, lse, pu.ref_attn(s), "large scores")


@pytest.mark.parametrize("new,ps", [([1, 2, 130], 16), ([70, 1, 3], 256)])
def test_fwd_bad_table_entries_are_skipped(new, ps):
    m = gpu_util.ea()
    s = pu.make_step(new, [400, 1000, 300], 8, 2, 128, ps, seed=8)
    s.table[1, 1], s.table[1, 2], s.table[2, 0] = -1, 2 ** 31 - 1, s.num_pages
    o, lse, st = _run_attn(s)
    assert st == m.ATTN_ERR_BAD_INDEX and m.attn_status() == 0
    pu.check_attn(s, o, lse, pu.ref_attn(s), "bad pages")


def test_fwd_bad_lengths_and_offsets_are_clamped():
    m = gpu_util.ea()
    s = pu.make_step([4, 4, 4], [40, 40, 40], 4, 2, 64, 16, seed=2, pad=2)
    want = pu.ref_attn(s)
    good = s.seq.clone(), s.cu.clone()
    s.seq[1] = 10 ** 6
    o, lse, st = _run_attn(s)
    assert st == m.ATTN_ERR_BAD_INDEX
    rows = list(range(4)) + list(range(8, 12))       # the other sequences are exact
    assert ((o[rows].double() - want[0][rows]).abs() <= want[2][rows]).all()
    s.seq, s.cu = good[0], torch.tensor([0, 4, 8, 10 ** 6], dtype=torch.int32)
    o, lse, st = _run_attn(s)
    assert st == m.ATTN_ERR_BAD_INDEX
    assert ((o[:8].double() - want[0][:8]).abs() <= want[2][:8]).all()
    s.cu = torch.tensor([-5, 4, 2, 12], dtype=torch.int32)
    _, _, st = _run_attn(s)
    assert st == m.ATTN_ERR_BAD_INDEX


def test_fwd_is_deterministic_and_needs_no_clean_workspace():
    m = gpu_util.ea()
    s = pu.make_step([1, 300, 5], [9000, 800, 2000], 8, 2, 128, 64, seed=4)
    ws = torch.zeros(m.attn_fwd_paged_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    a = _run_attn(s, ws=ws)
    b = _run_attn(s, ws=ws)
    c = _run_attn(s)
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1]) and x[2] == 0


def test_fwd_agrees_with_decode_paged_and_attn_fwd():
    """The paths that were there, on the inputs they share with the new one."""
    m = gpu_util.ea()
    s = pu.make_step([1, 1], [700, 30], 4, 4, 128, 64, seed=6)
    o, lse, st = _run_attn(s)
    od = torch.empty((2, 4, 1, 128), dtype=torch.bfloat16, device="cuda")
    ld = torch.empty((2, 4, 1), dtype=torch.float32, device="cuda")
    ws = torch.empty(m.attn_decode_workspace_bytes(2, 4, 128, 4), dtype=torch.uint8, device="cuda")
    m.attn_decode_paged(s.q.cuda()[:, :, None].contiguous(), s.kc.cuda(), s.vc.cuda(),
                        s.table.cuda(), s.seq.cuda(), od, ld, s.scale, 4, ws)
    assert st == 0 and m.attn_status() == 0
    ref = pu.ref_attn(s)
    pu.check_attn(s, o, lse, ref)
    assert ((od[:, :, 0].cpu().double() - ref[0]).abs() <= ref[2]).all()
    assert ((ld[:, :, 0].cpu() - lse).abs() <= 2e-5 * (1 + lse.abs())).all()


def test_fwd_long_offsets():
    """A cache whose last page lies beyond 2^31 elements."""
    m = gpu_util.ea()
    ps, Hkv, d = 1024, 8, 128
    pages = (2 ** 31) // (ps * Hkv * d) + 3
    kc = torch.empty((pages, Hkv, ps, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    s = pu.make_step([2], [1800], Hkv, Hkv, d, ps, seed=12)
    far = torch.tensor([pages - 1, pages - 2])
    for i in range(2):
        kc[far[i]], vc[far[i]] = s.kc[s.table[0, i]].cuda(), s.vc[s.table[0, i]].cuda()
    o = torch.full((2, Hkv, d), -77, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, Hkv), -77, dtype=torch.float32, device="cuda")
    ws = torch.empty(m.attn_fwd_paged_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    table = torch.full((1, s.max_pages), -1, dtype=torch.int32)
    table[0, :2] = far
    m.attn_fwd_paged(s.q.cuda(), kc, vc, table.cuda(), s.cu.cuda(), s.seq.cuda(), o, lse, True,
                     s.scale, ws)
    assert m.attn_status() == 0
    pu.check_attn(s, o.cpu(), lse.cpu(), pu.ref_attn(s), "far pages")
    k = torch.randn((1, Hkv, d), device="cuda").bfloat16()
    kb = torch.zeros((pages, Hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    m.attn_paged_append(k, k, torch.tensor([pages * ps - 1], device="cuda"), kc, vc, kb)
    assert m.attn_status() == 0
    assert torch.equal(kc[-1, :, -1], k[0]) and torch.equal(vc[-1, :, -1], k[0])
    assert torch.equal(kb[-1, :, 0], kc[-1].amin(1)) or torch.isnan(kc[-1].float()).any()


# ------------------------------------------------------- select and sparse --
@pytest.mark.parametrize("new,ctx,Hq,Hkv,d,ps,K,first,last", [
    ([1], [0], 1, 1, 64, 16, 1, 0, 0),
    ([1, 1], [500, 90], 8, 2, 128, 16, 6, 1, 2),
    ([5, 0, 33], [200, 7, 0], 6, 2, 64, 16, 4, 0, 1),
    ([2], [5000], 28, 4, 128, 16, 40, 2, 3),
    ([1], [20000], 4, 1, 64, 16, 100, 0, 1),
    ([3], [300], 40, 1, 64, 32, 20, 1, 1),
    ([3, 20], [1500, 40], 100, 1, 128, 16, 20, 1, 0),
    ([1], [70000], 2, 2, 64, 16, 50, 1, 1),
    ([17, 1, 9], [1100, 1023, 2000], 16, 2, 128, 16, 30, 0, 1),
])
def test_select_matches_definition(new, ctx, Hq, Hkv, d, ps, K, first, last):
    m = gpu_util.ea()
    s = pu.make_step(new, ctx, Hq, Hkv, d, ps, seed=K + ps, pad=2, poison=False)
    kb = pu.page_bounds(s.kc)
    kb[5 % s.num_pages] = kb[0]                     # equal scores
    sel = torch.full((s.T, Hkv, K), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(m.attn_page_select_workspace_bytes(s.T, Hkv, s.max_pages), dtype=torch.uint8,
                     device="cuda")
    m.attn_page_select(s.q.cuda(), kb.cuda(), s.table.cuda(), s.cu.cuda(), s.seq.cuda(), sel, ps,
                       first, last, ws)
    assert m.attn_status() == 0
    assert torch.equal(sel.cpu(), pu.ref_select(s, kb, K, first, last))


def test_select_many_equal_scores_and_bad_pages():
    m = gpu_util.ea()
    s = pu.make_step([3], [1600], 4, 2, 64, 16, seed=1, poison=False)
    kb = pu.page_bounds(s.kc)
    kb[:] = kb[1]
    kb[s.table[0, 60]] += 4                        # one above all others, one below
    kb[s.table[0, 3]] -= 4
    s.table[0, 7], s.table[0, 9] = -1, s.num_pages
    sel = torch.full((3, 2, 9), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(m.attn_page_select_workspace_bytes(3, 2, s.max_pages), dtype=torch.uint8,
                     device="cuda")
    m.attn_page_select(s.q.cuda(), kb.cuda(), s.table.cuda(), s.cu.cuda(), s.seq.cuda(), sel, 16,
                       0, 1, ws)
    assert m.attn_status() == m.ATTN_ERR_BAD_INDEX
    assert torch.equal(sel.cpu(), pu.ref_select(s, kb, 9, 0, 1))


@pytest.mark.parametrize("ps,ctx", [(16, 1500), (16, 30000)])
def test_select_near_scores(ps, ctx):
    """Pages whose scores differ by less than 32-bit sums can tell, and rows of zeros."""
    m = gpu_util.ea()
    s = pu.make_step([2, 1], [ctx, 40], 4, 1, 128, ps, seed=5, poison=False)
    s.q[2] = 0
    kb = pu.page_bounds(s.kc)
    base = kb[s.table[0, 0].long()].clone()
    for i in range(ctx // ps):
        row = base.clone()
        row[0, 1] = base[0, 1] * 2.0 ** -(i % 5)          # the largest key of one channel shrinks,
        row[0, 1, 2:] = base[0, 1, 2:]                      # in the first two channels alone
        row[0, 1, 0] = 2.0 ** -20 * (1 + (i * 7919) % 97)   # and by next to nothing in one
        kb[s.table[0, i].long()] = row
    sel = torch.full((3, 1, 9), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(m.attn_page_select_workspace_bytes(3, 1, s.max_pages), dtype=torch.uint8,
                     device="cuda")
    m.attn_page_select(s.q.cuda(), kb.cuda(), s.table.cuda(), s.cu.cuda(), s.seq.cuda(), sel, ps,
                       1, 1, ws)
    assert m.attn_status() == 0
    assert torch.equal(sel.cpu(), pu.ref_select(s, kb, 9, 1, 1))


@pytest.mark.parametrize("new,ctx,Hq,Hkv,d,ps,K", [
    ([1], [0], 1, 1, 64, 16, 3), ([1, 1, 1], [5000, 900, 77], 32, 8, 128, 64, 12),
    ([4, 0, 30], [300, 2, 0], 6, 2, 64, 16, 7), ([3], [2000], 28, 4, 128, 256, 5),
    ([2], [6000], 4, 2, 64, 1024, 3), ([20], [200], 12, 12, 128, 32, 4),
    ([2, 1], [900, 30], 128, 1, 64, 128, 5),
])
def test_sparse_matches_definition(new, ctx, Hq, Hkv, d, ps, K):
    s = pu.make_step(new, ctx, Hq, Hkv, d, ps, seed=K + ps, pad=3, strided=Hq > 4)
    g = torch.Generator().manual_seed(K)
    sel = torch.full((s.T, Hkv, K), -1, dtype=torch.int32)
    for b in range(s.B):
        pages = max(1, -(-s.lens[b] // ps))
        for i in range(new[b]):
            for h in range(Hkv):
                n = int(torch.randint(0, min(K, pages) + 1, (1,), generator=g))
                at = torch.randperm(K, generator=g)[:n]
                sel[int(s.cu[b]) + i, h, at] = torch.randperm(pages, generator=g)[:n].int()
    o, lse, st = _run_attn(s, sel=sel)
    assert st == 0
    pu.check_attn(s, o, lse, pu.ref_attn(s, sel=sel), "sparse")


def test_sparse_repeated_and_out_of_range_entries():
    """A page listed twice counts twice; entries past the sequence are skipped and reported."""
    m = gpu_util.ea()
    s = pu.make_step([2, 1], [300, 40], 4, 2, 128, 16, seed=21)
    sel = torch.tensor([3, 3, 0, -1], dtype=torch.int32).expand(3, 2, 4).clone()
    sel[1] = torch.tensor([18, 5, 18, 2], dtype=torch.int32)
    sel[2] = torch.tensor([1, 1, 1, 0], dtype=torch.int32)
    o, lse, st = _run_attn(s, sel=sel)
    assert st == 0
    pu.check_attn(s, o, lse, pu.ref_attn(s, sel=sel), "repeated")
    sel[2] = torch.tensor([1, 2 ** 31 - 1, -9, 3], dtype=torch.int32)
    o, lse, st = _run_attn(s, sel=sel)
    assert st == m.ATTN_ERR_BAD_INDEX
    pu.check_attn(s, o, lse, pu.ref_attn(s, sel=sel), "out of range")


def test_sparse_over_all_pages_is_the_causal_forward():
    s = pu.make_step([5, 1], [500, 70], 8, 2, 128, 32, seed=31)
    sel = torch.arange(s.max_pages, dtype=torch.int32).expand(s.T, 2, s.max_pages).clone()
    for b in range(2):
        for i in range(s.new[b]):
            row = int(s.cu[b]) + i
            sel[row][sel[row] * s.ps >= s.lens[b]] = -1
    o, lse, st = _run_attn(s, sel=sel)
    assert st == 0
    pu.check_attn(s, o, lse, pu.ref_attn(s), "all pages")


# ------------------------------------------------------------- all together --
def test_serving_steps_together():
    """Three steps of three sequences (prompts, a second chunk, one token each): tables, append,
    attention, and page choice with attention over the chosen pages; every step on another stream
    than the tensors were made on."""
    m = gpu_util.ea()
    Hq, Hkv, d, ps, B, max_pages, F = 8, 2, 128, 16, 3, 24, 80
    g = torch.Generator().manual_seed(77)
    free = torch.randperm(F, generator=g).int().cuda()
    head, lens = _i32([0]), _i32([0] * B)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    nan = float("nan")
    kc, vc = (torch.full((F, Hkv, ps, d), nan, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    kb = torch.zeros((F, Hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(m.attn_fwd_paged_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    past_k = [torch.zeros((0, Hkv, d), dtype=torch.bfloat16) for _ in range(B)]
    past_v = [torch.zeros((0, Hkv, d), dtype=torch.bfloat16) for _ in range(B)]
    stream = torch.cuda.Stream()
    for new in ([100, 7, 33], [50, 0, 141], [1, 1, 1]):
        T = sum(new) + 4
        qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=g).bfloat16()
        dev = qkv.cuda()
        q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
        dnew, cu = _i32(new), _i32([0] * (B + 1))
        slots = torch.zeros(T, dtype=torch.int64, device="cuda")
        K = 5
        sel = torch.full((T, Hkv, K), -7, dtype=torch.int32, device="cuda")
        o, o2 = (torch.full((T, Hq, d), -77, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lse, lse2 = (torch.full((T, Hq), -77, dtype=torch.float32, device="cuda") for _ in range(2))
        ws2 = torch.empty(m.attn_page_select_workspace_bytes(T, Hkv, max_pages), dtype=torch.uint8,
                          device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            m.attn_page_tables(lens, dnew, free, head, head, table, lens, cu, slots, ps, F)
            m.attn_paged_append(k, v, slots, kc, vc, kb)
            m.attn_fwd_paged(q, kc, vc, table, cu, lens, o, lse, True, d ** -0.5, ws)
            m.attn_page_select(q, kb, table, cu, lens, sel, ps, 1, 2, ws2)
            m.attn_sparse_paged(q, kc, vc, table, cu, lens, sel, o2, lse2, d ** -0.5, ws)
            assert m.attn_status() == 0
        # the definition, on the keys and values as they came
        at = 0
        for b in range(B):
            past_k[b] = torch.cat([past_k[b], qkv[at:at + new[b], Hq:Hq + Hkv]])
            past_v[b] = torch.cat([past_v[b], qkv[at:at + new[b], Hq + Hkv:]])
            at += new[b]
        s = pu.make_step(new, [len(p) - n for p, n in zip(past_k, new)], Hq, Hkv, d, ps, seed=0,
                         pad=4, poison=False)
        for b in range(B):
            for i in range(-(-len(past_k[b]) // ps)):
                part = past_k[b][i * ps:(i + 1) * ps]
                s.kc[s.table[b, i], :, :len(part)] = part.transpose(0, 1)
                s.vc[s.table[b, i], :, :len(part)] = past_v[b][i * ps:(i + 1) * ps].transpose(0, 1)
                # bounds of the tokens that are there
                s.kc[s.table[b, i], :, len(part):] = part[-1][:, None]
        s.q = qkv[:, :Hq]
        s.scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
        pu.check_attn(s, o.cpu(), lse.cpu(), pu.ref_attn(s), "step")
        want = pu.ref_select(s, pu.page_bounds(s.kc), K, 1, 2)
        assert torch.equal(sel.cpu(), want)
        pu.check_attn(s, o2.cpu(), lse2.cpu(), pu.ref_attn(s, sel=want), "sparse step")
