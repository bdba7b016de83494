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
