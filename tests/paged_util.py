"""Inputs and plain 64-bit definitions of the serving operators on a paged cache."""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np
import torch

NAN = float("nan")


def make_step(new, ctx, Hq, Hkv, d, ps, seed, pad=0, poison=True, strided=False, extra_pages=2,
              len_override=None):
    """A step of len(new) sequences over a paged cache, on the CPU. Every slot that holds no token
    of a sequence is NaN (poison), every unused table entry far out of range."""
    g = torch.Generator().manual_seed(seed)
    B = len(new)
    lens = [n + c for n, c in zip(new, ctx)] if len_override is None else list(len_override)
    max_pages = max(1, max(-(-x // ps) for x in lens)) + extra_pages
    held = [-(-x // ps) for x in lens]
    num_pages = sum(held) + 3
    perm = torch.randperm(num_pages, generator=g).tolist()
    table = torch.full((B, max_pages), 2 ** 30 + 7, dtype=torch.int32)
    kc = torch.randn((num_pages, Hkv, ps, d), generator=g).bfloat16()
    vc = torch.randn((num_pages, Hkv, ps, d), generator=g).bfloat16()
    live = torch.zeros((num_pages, ps), dtype=torch.bool)
    at = 0
    for b in range(B):
        for i in range(held[b]):
            table[b, i] = perm[at]
            live[perm[at], :max(0, min(ps, lens[b] - i * ps))] = True
            at += 1
    if poison:
        dead = ~live[:, None, :, None].expand_as(kc)
        kc = torch.where(dead, torch.tensor(NAN, dtype=torch.bfloat16), kc)
        vc = torch.where(dead, torch.tensor(NAN, dtype=torch.bfloat16), vc)
    T = sum(new) + pad
    if strided:
        q = torch.randn((T, Hq + 2 * Hkv + 1, d), generator=g).bfloat16()[:, 1:Hq + 1]
    else:
        q = torch.randn((T, Hq, d), generator=g).bfloat16()
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    return SimpleNamespace(q=q, kc=kc, vc=vc, table=table, cu=cu,
                           seq=torch.tensor(lens, dtype=torch.int32), new=list(new), lens=lens,
                           B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, ps=ps, scale=float(np.float32(d ** -0.5)),
                           num_pages=num_pages, max_pages=max_pages)


def seq_kv(s, b):
    """Sequence b's K and V, [Hkv, len, d] fp64, and which keys can be read."""
    ln = s.lens[b]
    pages = s.table[b, :-(-ln // s.ps)].long()
    ok = (pages >= 0) & (pages < s.num_pages)
    idx = torch.where(ok, pages, 0)
    k = s.kc[idx].permute(1, 0, 2, 3).reshape(s.Hkv, -1, s.d)[:, :ln].double()
    v = s.vc[idx].permute(1, 0, 2, 3).reshape(s.Hkv, -1, s.d)[:, :ln].double()
    return k, v, ok.repeat_interleave(s.ps)[:ln]


def ref_attn(s, causal=True, sel=None):
    """O, LSE in 64 bits and the bounds of their errors, for rows of sequences (others: NaN).

    The kernel rounds twice to bf16: each p (off by 2^-8 of itself at most, so O by 2^-8 of
    sum p |v| / l) and O (2^-8 |O|). Scores are fp32 sums of d exact products, which moves a
    score by at most 2 d 2^-24 sum |q k| scale =: e, p by that share of itself, and the rest (the
    exponential, sums over keys, the joining of parts) is fp32 too: 2^-18 covers it.
      |dO| <= 2^-8 |O| + (2^-8 + 2 e + 2^-18) sum p |v| / l,  |dLSE| <= e + 2^-18 (1 + |LSE|)"""
    T, G = s.T, s.Hq // s.Hkv
    o = torch.full((T, s.Hq, s.d), NAN, dtype=torch.float64)
    lse = torch.full((T, s.Hq), NAN, dtype=torch.float64)
    o_tol, l_tol = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(s.B):
        n, ln = s.new[b], s.lens[b]
        if n == 0:
            continue
        k, v, ok = seq_kv(s, b)
        rows = slice(int(s.cu[b]), int(s.cu[b]) + n)
        pos = ln - n + torch.arange(n)
        seen = ok[None].expand(n, ln)
        if causal or sel is not None:
            seen = seen & (torch.arange(ln)[None] <= pos[:, None])
        for h in range(s.Hq):
            weight = seen.double()
            if sel is not None:      # how often a row lists each key's page
                times = torch.zeros((n, s.max_pages + 1), dtype=torch.float64)
                pick = sel[rows, h // G].long()
                pick = torch.where((pick < 0) | (pick * s.ps >= max(ln, 1)), s.max_pages, pick)
                times.scatter_add_(1, pick, torch.ones_like(pick, dtype=torch.float64))
                weight = weight * times[:, :-1].repeat_interleave(s.ps, 1)[:, :ln]
            kk, vv = k[h // G], v[h // G]
            kk = torch.where(ok[:, None], kk, 0.0)
            vv = torch.where(ok[:, None], vv, 0.0)
            qq = s.q[rows, h].double()
            score = qq @ kk.T * s.scale
            score = torch.where(weight > 0, score + torch.log(weight), -torch.inf)
            L = torch.logsumexp(score, 1) if ln else torch.full((n,), -torch.inf, dtype=torch.float64)
            p = torch.exp(score - torch.where(L.isinf(), 0.0, L)[:, None])
            o[rows, h] = p @ vv
            lse[rows, h] = L
            e = torch.where(weight > 0, qq.abs() @ kk.abs().T, 0.0).amax(1) if ln else torch.zeros(n)
            e = e.double() * s.scale * 2 * s.d * 2.0 ** -24
            o_tol[rows, h] = 2.0 ** -8 * o[rows, h].abs() + \
                (2.0 ** -8 + 2 * e + 2.0 ** -18)[:, None] * (p @ vv.abs())
            l_tol[rows, h] = e + 2.0 ** -18 * (1 + torch.where(L.isinf(), 0.0, L).abs())
    return o, lse, o_tol, l_tol


def check_attn(s, o, lse, ref, what=""):
    """o, lse (CPU) against ref_attn's; rows of no sequence still hold the -77 they began with."""
    ro, rl, o_tol, l_tol = ref
    end = int(s.cu[-1])
    assert torch.all(o[end:] == -77) and torch.all(lse[end:] == -77), f"{what}: rows past the last"
    o, lse, ro, rl = o[:end].double(), lse[:end].double(), ro[:end], rl[:end]
    empty = rl == -torch.inf
    assert torch.equal(lse == -torch.inf, empty), f"{what}: rows that see no key"
    assert torch.all(o[empty] == 0), f"{what}: rows that see no key are 0"
    assert torch.isfinite(o).all(), f"{what}: O not finite"
    do = (o - ro).abs() - o_tol[:end]
    assert do.max().item() <= 0 if do.numel() else True, f"{what}: O over its bound by {do.max()}"
    dl = torch.where(empty, 0.0, (lse - torch.where(empty, 0.0, rl)).abs() - l_tol[:end])
    assert dl.max().item() <= 0 if dl.numel() else True, f"{what}: LSE over its bound by {dl.max()}"


def ref_tables(ctx, new, free, head, table, T, ps, num_pages):
    """The step's bookkeeping, token by token. Returns table, seq, cu, slots, head, whether all
    was in order."""
    table = [list(r) for r in table]
    cap = len(table[0]) * ps
    slots, cu, seq, fine = [], [0], [], True
    if not 0 <= head <= len(free):
        fine, head = False, len(free)
    for b, (c, n) in enumerate(zip(ctx, new)):
        if c < 0 or n < 0 or c + n > cap:
            fine, n, c = False, 0, min(max(c, 0), cap)
        if n > T - len(slots):
            fine, n = False, T - len(slots)
        for j in range(c, c + n):
            page = j // ps
            if j % ps == 0:
                table[b][page] = free[head] if head < len(free) else -1
                if not 0 <= table[b][page] < num_pages:
                    table[b][page] = -1
                head = min(head + 1, len(free))
            e = table[b][page]
            good = 0 <= e < num_pages
            fine = fine and good
            slots.append(e * ps + j % ps if good else -1)
        seq.append(c + n)
        cu.append(len(slots))
    return table, seq, cu, slots + [-1] * (T - len(slots)), head, fine


def ref_select(s, bounds, K, first, last):
    """sel [T, Hkv, K] from the definition in 64 bits (rows of no sequence: -7)."""
    G = s.Hq // s.Hkv
    out = torch.full((s.T, s.Hkv, K), -7, dtype=torch.int32)
    for b in range(s.B):
        for i in range(s.new[b]):
            t = int(s.cu[b]) + i
            pos = s.lens[b] - s.new[b] + i
            count = pos // s.ps + 1 if pos >= 0 else 0
            for h in range(s.Hkv):
                ranked = []
                for j in range(count):
                    page = int(s.table[b, j])
                    if not 0 <= page < s.num_pages:
                        continue
                    if j < first or j >= count - last:
                        ranked.append((-float("inf"), j))
                        continue
                    lo, hi = bounds[page, h].double()
                    q = s.q[t, h * G:(h + 1) * G].double()
                    ranked.append((-float(torch.where(q >= 0, q * hi, q * lo).sum(1).max()), j))
                chosen = sorted(j for _, j in sorted(ranked)[:K])
                out[t, h] = torch.tensor(chosen + [-1] * (K - len(chosen)), dtype=torch.int32)
    return out


def page_bounds(kc):
    f = kc.float()
    return torch.stack([f.amin(2), f.amax(2)], 2).bfloat16()
