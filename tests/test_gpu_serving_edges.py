"""Calls of the serving operators at the edges of what their documentation allows."""
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
