"""Workloads of the paged serving operators, for measuring them against their plain definitions.

Five operators that a serving program runs one after another on a paged K/V cache:
  tables  attn_page_tables   block tables, sequence lengths, row offsets and slots of a step's tokens
  append  attn_paged_append  the step's K and V written into the cache, with each page's key bounds
  fwd     attn_fwd_paged     attention of each sequence's new tokens over its cached keys
  select  attn_page_select   the pages each query reads, by an upper bound of its scores in a page
  sparse  attn_sparse_paged  attention of each query over its selected pages

Layouts: caches [num_pages, Hkv, page_size, d], bounds [num_pages, Hkv, 2, d] (least, then largest
key of each channel), q [T, Hq, d] of all sequences' new tokens one after another (rows cu[b] to
cu[b + 1] are sequence b's), block table [B, max_pages].
"""
import math
from types import SimpleNamespace

import torch

own = False

INF = float("inf")


# ---------------------------------------------------------------- the cases --
def listed():
    return [
        # one step of 16 sequences that generate at up to 32768 tokens: latency counts
        dict(name="tables_decode", op="tables", B=16, new=1, ctx=32767, mix=1, ps=64, pad=0),
        # admission of many prompts at once, ragged, in a padded token buffer
        dict(name="tables_prompts", op="tables", B=500, new=150, ctx=900, mix=7, ps=16, pad=331),
        # the same step's K and V: 16 tokens, most of them inside a partly filled page
        dict(name="append_decode", op="append", B=16, new=1, ctx=2047, mix=3, Hkv=8, d=128, ps=64,
             pad=0, fused=True),
        # prompts of up to 4096 tokens written as they come out of the fused projection
        dict(name="append_prompts", op="append", B=5, new=4096, ctx=500, mix=5, Hkv=32, d=128,
             ps=32, pad=77, fused=True),
        # a generating step over a 32K-token cache, grouped query heads
        dict(name="fwd_decode_32k", op="fwd", B=16, new=1, ctx=32767, mix=0, Hq=32, Hkv=8, d=128,
             ps=64, pad=0, fused=True),
        # a few drafted tokens per sequence to check, short ragged caches, padded batch
        dict(name="fwd_drafts", op="fwd", B=7, new=6, ctx=3001, mix=2, Hq=28, Hkv=4, d=128, ps=16,
             pad=5, fused=True),
        # a chunk of two long prompts behind their earlier chunks
        dict(name="fwd_chunk_16k", op="fwd", B=2, new=2048, ctx=14336, mix=9, Hq=32, Hkv=8, d=128,
             ps=64, pad=0, fused=True),
        # whole prompts at the GPT-2 head layout, nothing cached before
        dict(name="fwd_prompts_1k", op="fwd", B=8, new=1024, ctx=0, mix=4, Hq=12, Hkv=12, d=64,
             ps=32, pad=0, fused=False),
        # the page choice of a generating step at 32K: 512 pages, 32 of them read
        dict(name="select_decode_32k", op="select", B=16, new=1, ctx=32767, mix=0, Hq=32, Hkv=8,
             d=128, ps=64, K=32, first=1, last=2, pad=0),
        # the page choice of every token of a chunk
        dict(name="select_chunk_16k", op="select", B=2, new=700, ctx=15000, mix=3, Hq=32, Hkv=8,
             d=128, ps=64, K=16, first=1, last=2, pad=3),
        # attention of that generating step over its 32 pages
        dict(name="sparse_decode_32k", op="sparse", B=16, new=1, ctx=32767, mix=0, Hq=32, Hkv=8,
             d=128, ps=64, K=32, pad=0),
        # and of a chunk's tokens, each over its own 16 pages
        dict(name="sparse_chunk_16k", op="sparse", B=2, new=700, ctx=15000, mix=3, Hq=32, Hkv=8,
             d=128, ps=64, K=16, pad=3),
    ]


def _log(rng, low, top):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(top)))))


def draw(rng):
    op = rng.choice(["tables", "append", "fwd", "fwd", "select", "sparse"])
    ps = rng.choice([16, 32, 64, 128, 256])
    mix = rng.randrange(1, 1000)
    Hq, Hkv = rng.choice([(32, 8), (32, 32), (12, 12), (28, 4), (8, 1), (24, 8), (16, 2)])
    d = rng.choice([64, 128])
    pad = rng.choice([0, 0, 1, 9, 64])
    if op == "tables":
        return dict(op=op, B=_log(rng, 1, 600), new=_log(rng, 1, 120), ctx=_log(rng, 1, 4000),
                    mix=mix, ps=ps, pad=pad)
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, new=_log(rng, 1, 16384 // B), ctx=_log(rng, 1, 1000), mix=mix,
                    Hkv=Hkv, d=d, ps=ps, pad=pad, fused=rng.random() < 0.5)
    if op == "fwd":
        B = _log(rng, 1, 16)
        new = _log(rng, 1, 1024)
        top = min(131072 // B, (1 << 30) // (B * Hq * new))   # tokens a sequence holds, at most
        ctx = _log(rng, 1, max(2, min(32000, top - new)))
        return dict(op=op, B=B, new=new, ctx=ctx, mix=mix, Hq=Hq, Hkv=Hkv, d=d, ps=ps, pad=pad,
                    fused=rng.random() < 0.5)
    new = rng.choice([1, 1, _log(rng, 2, max(3, min(200, 1600 // Hkv)))])
    B = _log(rng, 1, 16) if new == 1 else rng.randrange(1, 4)
    ctx = _log(rng, 8 * ps, 30000 if new == 1 else 8000)
    K = _log(rng, 4, max(5, min(2048 // ps, ctx // ps - 2)))
    if op == "select":
        return dict(op=op, B=B, new=new, ctx=ctx, mix=mix, Hq=Hq, Hkv=Hkv, d=d, ps=ps, K=K,
                    first=rng.randrange(0, 2), last=rng.randrange(1, 3), pad=pad)
    return dict(op=op, B=B, new=new, ctx=ctx, mix=mix, Hq=Hq, Hkv=Hkv, d=d, ps=ps, K=K, pad=pad)


def _ragged(top, low, count, mix):
    """`count` lengths from low to top, the first of them top; mix = 0: all of them top."""
    if mix == 0 or top <= low:
        return [top] * count
    x = [((i * 2654435761 + mix * 40503 + 12345) >> 7) % (top - low + 1) for i in range(count)]
    return [top] + [low + v for v in x[1:]]


def _lens(c):
    new = _ragged(c["new"], min(c["new"], max(1, c["new"] // 4)), c["B"], c["mix"])
    ctx = _ragged(c["ctx"], c["ctx"] // 8, c["B"], c["mix"] * 3)
    return new, ctx


def _pages(n, ps):
    return -(-n // ps)


# ------------------------------------------------------------------ the work --
def work(c):
    new, ctx = _lens(c)
    ps = c["ps"]
    T = sum(new)
    if c["op"] == "tables":
        alloc = sum(_pages(x + n, ps) - _pages(x, ps) for n, x in zip(new, ctx))
        # ctx, new, lengths, offsets; free pages read and entries written; a slot per row
        return dict(bytes=4 * (4 * c["B"] + 1) + 8 * alloc + 8 * (T + c["pad"]), flops=0)
    Hkv, d = c["Hkv"], c["d"]
    if c["op"] == "append":
        touched = sum(_pages(x + n, ps) - x // ps for n, x in zip(new, ctx))
        # K and V in and out, the earlier keys of each sequence's first page, the bounds
        before = sum(x % ps for x in ctx)
        return dict(bytes=8 * T * Hkv * d + 8 * (T + c["pad"]) + 2 * Hkv * d * before +
                    4 * touched * Hkv * d, flops=0)
    Hq = c["Hq"]
    if c["op"] == "fwd":
        seen = sum(n * x + n * (n + 1) // 2 for n, x in zip(new, ctx))   # (row, key) pairs
        keys = sum(n + x for n, x in zip(new, ctx))
        return dict(bytes=4 * T * Hq * d + 4 * T * Hq + 4 * keys * Hkv * d, flops=4 * seen * Hq * d)
    vis = [[(x + i) // ps + 1 for i in range(n)] for n, x in zip(new, ctx)]   # pages a row sees
    if c["op"] == "select":
        return dict(bytes=2 * T * Hq * d + sum(4 * v[-1] * Hkv * d for v in vis) +
                    4 * T * Hkv * c["K"], flops=2 * sum(map(sum, vis)) * Hq * d)
    pairs = sum(min(k, c["K"]) * ps for v in vis for k in v)
    # each sequence's pages at most once, and no more of them than its rows list
    keys = sum(ps * min(v[-1], sum(min(k, c["K"]) for k in v)) for v in vis)
    return dict(bytes=4 * T * Hq * d + 4 * T * Hq + 4 * T * Hkv * c["K"] + 4 * keys * Hkv * d,
                flops=4 * pairs * Hq * d)


# ---------------------------------------------------------------- the inputs --
def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"
    new, ctx = _lens(c)
    B, ps, pad = c["B"], c["ps"], c["pad"]
    s = SimpleNamespace(**{k: v for k, v in c.items() if k != "name"})
    s.T = sum(new) + pad
    s.nmax = max(new)
    s.npg = max(_pages(n + x, ps) for n, x in zip(new, ctx))   # logical pages the longest one holds
    s.max_pages = s.npg + 1
    i32 = dict(dtype=torch.int32, device=dev)
    s.new_lens = torch.tensor(new, **i32)
    s.ctx_lens = torch.tensor(ctx, **i32)
    s.seq = s.ctx_lens + s.new_lens
    s.cu = torch.zeros(B + 1, **i32)
    s.cu[1:] = torch.cumsum(s.new_lens, 0)
    # pages in a random physical order; entries past a sequence's pages are -1
    held = (s.seq.long() + ps - 1) // ps
    total = sum(_pages(n + x, ps) for n, x in zip(new, ctx))
    s.num_pages = total + B + 61
    perm = torch.randperm(s.num_pages, generator=g, device=dev)
    lp = torch.arange(s.max_pages, device=dev)[None]
    at = (torch.cumsum(held, 0) - held)[:, None] + lp
    s.table = torch.where(lp < held[:, None], perm[at.clamp(max=s.num_pages - 1)], -1).int()
    s.ws = None
    if s.op == "tables":
        before = (s.ctx_lens.long() + ps - 1) // ps
        s.old_table = torch.where(lp < before[:, None], s.table, -1).int()
        s.free_pages = torch.cat([torch.full((5,), -1, **i32), perm[torch.randperm(
            s.num_pages, generator=g, device=dev)].int()])
        s.free_head = torch.tensor([5], **i32)
        s.free_out = torch.zeros(1, **i32)
        s.seq_out = torch.zeros(B, **i32)
        s.cu_out = torch.zeros(B + 1, **i32)
        s.slots = torch.zeros(s.T, dtype=torch.int64, device=dev)
        return s

    Hkv, d = c["Hkv"], c["d"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    # keys differ in size from channel to channel
    spread = torch.exp(0.3 * torch.randn((Hkv, 1, d), generator=g, device=dev)).bfloat16()
    s.kc = randn(s.num_pages, Hkv, ps, d)
    s.kc.mul_(spread)
    s.scale = float(torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32))
    if s.op == "append":
        s.vc = randn(s.num_pages, Hkv, ps, d)
        s.bounds = torch.zeros((s.num_pages, Hkv, 2, d), dtype=torch.bfloat16, device=dev)
        if c["fused"]:   # views of one projection's output, as many query heads beside them
            qkv = randn(s.T, 3 * Hkv, d)
            s.k, s.v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
        else:
            s.k, s.v = randn(s.T, Hkv, d), randn(s.T, Hkv, d)
        t, b, i = _rows(s)
        pos = s.ctx_lens[b].long() + i
        # (a padding row's place can lie past the table: it gets no slot)
        slot = s.table[b, (pos // ps).clamp(max=s.max_pages - 1)].long() * ps + pos % ps
        s.slots = torch.where(t < s.cu[-1], slot, -1)
        return s

    Hq = c["Hq"]
    s.q = randn(s.T, Hq + 2 * Hkv, d)[:, :Hq] if c.get("fused") else randn(s.T, Hq, d)
    if s.op == "select":
        f = s.kc.float()
        s.bounds = torch.stack([f.amin(2), f.amax(2)], 2).bfloat16()
        s.kc = None
        s.sel = torch.full((s.T, Hkv, c["K"]), -1, **i32)
        return s
    s.vc = randn(s.num_pages, Hkv, ps, d)
    s.o = torch.zeros((s.T, Hq, d), dtype=torch.bfloat16, device=dev)
    s.lse = torch.zeros((s.T, Hq), dtype=torch.float32, device=dev)
    if s.op == "sparse":
        # ascending pages among those a row sees, its own page always, then -1
        t, b, i = _rows(s)
        vis = (s.ctx_lens[b].long() + i) // ps + 1
        r = torch.rand((s.T, Hkv, s.npg), generator=g, device=dev)
        j = torch.arange(s.npg, device=dev)
        r = torch.where(j < vis[:, None, None], r, 2.0)
        r = torch.where(j == vis[:, None, None] - 1, -1.0, r)
        got, pick = torch.sort(r, dim=-1)
        pick = torch.where(got < 1.5, pick, s.npg)[..., :c["K"]].sort(-1).values
        pick = torch.nn.functional.pad(pick, (0, c["K"] - pick.shape[-1]), value=s.npg)
        s.sel = torch.where(pick < s.npg, pick, -1).int()
    return s


def _rows(s):
    """Every row, the sequence it belongs to and its place in it."""
    t = torch.arange(s.T, device=s.cu.device)
    b = torch.searchsorted(s.cu[1:].contiguous(), t.int(), right=True).clamp(max=s.B - 1)
    return t, b, t - s.cu[b]


# ------------------------------------------------------------- plain forms --
def _plain_tables(s):
    ps = s.ps
    ctx, new = s.ctx_lens.long(), s.new_lens.long()
    cap = s.max_pages * ps
    good = (ctx >= 0) & (new >= 0) & (ctx + new <= cap)
    new = torch.where(good, new, 0)
    ctx = ctx.clamp(0, cap)
    new = torch.minimum((s.T - (torch.cumsum(new, 0) - new)).clamp(min=0), new)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=new.device), torch.cumsum(new, 0)])
    seq = ctx + new
    first, end = (ctx + ps - 1) // ps, (seq + ps - 1) // ps
    need = end - first
    lp = torch.arange(s.max_pages, device=new.device)[None]
    src = s.free_head + (torch.cumsum(need, 0) - need)[:, None] + lp - first[:, None]
    count = s.free_pages.numel()
    entry = torch.where(src < count, s.free_pages[src.clamp(0, count - 1)], -1)
    table = torch.where((lp >= first[:, None]) & (lp < end[:, None]), entry, s.old_table)
    t = torch.arange(s.T, device=new.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=s.B - 1)
    pos = ctx[b] + t - cu[b]
    page = table[b, (pos // ps).clamp(max=s.max_pages - 1)].long()
    slot = torch.where((t < cu[-1]) & (page >= 0), page * ps + pos % ps, -1)
    head = (s.free_head + need.sum()).clamp(max=count)
    return table.int(), seq.int(), cu.int(), slot, head.int()


def _plain_append(s):
    ps = s.ps
    keep = torch.nonzero(s.slots >= 0)[:, 0]
    slot = s.slots[keep]
    page, off = slot // ps, slot % ps
    s.kc[page, :, off] = s.k[keep]
    s.vc[page, :, off] = s.v[keep]
    fill = torch.zeros(s.num_pages, dtype=torch.int64, device=slot.device)
    fill = fill.scatter_reduce(0, page, off + 1, "amax")
    there = (torch.arange(ps, device=slot.device) < fill[:, None])[:, None, :, None]
    f = s.kc.float()
    new = torch.stack([torch.where(there, f, INF).amin(2), torch.where(there, f, -INF).amax(2)], 2)
    s.bounds.copy_(torch.where((fill > 0)[:, None, None, None], new.bfloat16(), s.bounds))
    return s.kc, s.vc, s.bounds


def _softmax_v(score, mask, v):
    """Softmax of the masked scores times v, and the log of the sums; rows with no key: 0, -inf."""
    score = torch.where(mask, score, -INF)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -INF, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return o, (m + torch.log(total))[..., 0]


def _plain_fwd(s):
    ps, G = s.ps, s.Hq // s.Hkv
    S = s.npg * ps
    pages = s.table[:, :s.npg].long().clamp(0, s.num_pages - 1)
    k = s.kc[pages].permute(0, 2, 1, 3, 4).reshape(s.B, s.Hkv, S, s.d).float()
    v = s.vc[pages].permute(0, 2, 1, 3, 4).reshape(s.B, s.Hkv, S, s.d).float()
    i = torch.arange(s.nmax, device=s.q.device)
    q = s.q[(s.cu[:-1, None] + i).clamp(max=s.T - 1).long()].float()   # [B, nmax, Hq, d]
    q = q.reshape(s.B, s.nmax, s.Hkv, G, s.d).permute(0, 2, 3, 1, 4).reshape(
        s.B, s.Hkv, G * s.nmax, s.d)
    j = torch.arange(S, device=s.q.device)
    seen = j <= (s.seq - s.new_lens)[:, None, None] + i[:, None]       # [B, nmax, S]
    seen = seen & (j < s.seq[:, None, None])
    mask = seen[:, None, None].expand(s.B, s.Hkv, G, s.nmax, S).reshape(
        s.B, s.Hkv, G * s.nmax, S)
    score = torch.matmul(q, k.transpose(-1, -2)) * s.scale
    o, lse = _softmax_v(score, mask, torch.where((j < s.seq[:, None])[:, None, :, None], v, 0.0))
    o = o.reshape(s.B, s.Hq, s.nmax, s.d)
    lse = lse.reshape(s.B, s.Hq, s.nmax)
    t, b, at = _rows(s)
    at = at.long().clamp(max=s.nmax - 1)
    live = t < s.cu[-1]
    return (torch.where(live[:, None, None], o[b, :, at].bfloat16(), s.o),
            torch.where(live[:, None], lse[b, :, at], s.lse))


def _plain_select(s):
    # in 64 bits: two pages' scores can be closer than 32 bits tell
    ps, G = s.ps, s.Hq // s.Hkv
    lo_hi = s.bounds[s.table[:, :s.npg].long().clamp(0, s.num_pages - 1)].double()
    lo, hi = lo_hi.permute(3, 0, 2, 1, 4)                               # [B, Hkv, npg, d] each
    i = torch.arange(s.nmax, device=s.q.device)
    q = s.q[(s.cu[:-1, None] + i).clamp(max=s.T - 1).long()].double()
    q = q.reshape(s.B, s.nmax, s.Hkv, G, s.d).permute(0, 2, 3, 1, 4).reshape(
        s.B, s.Hkv, G * s.nmax, s.d)
    score = torch.matmul(q.clamp(min=0), hi.transpose(-1, -2)) + torch.matmul(
        q.clamp(max=0), lo.transpose(-1, -2))
    score = score.reshape(s.B, s.Hkv, G, s.nmax, s.npg).amax(2)
    j = torch.arange(s.npg, device=s.q.device)
    vis = ((s.seq - s.new_lens)[:, None, None, None] + i[:, None]) // ps + 1   # [B, 1, nmax, 1]
    score = torch.where((j < s.first) | (j >= vis - s.last), INF, score)
    score = torch.where(j < vis, score, -INF)
    got, pick = torch.sort(score, dim=-1, descending=True, stable=True)
    pick = torch.where(got > -INF, pick, s.npg)[..., :s.K].sort(-1).values
    pick = torch.nn.functional.pad(pick, (0, s.K - pick.shape[-1]), value=s.npg)
    pick = torch.where(pick < s.npg, pick, -1).int()
    t, b, at = _rows(s)
    return torch.where((t < s.cu[-1])[:, None, None],
                       pick[b, :, at.long().clamp(max=s.nmax - 1)], s.sel)


def _plain_sparse(s):
    ps, G = s.ps, s.Hq // s.Hkv
    t, b, at = _rows(s)
    sel = s.sel.long()
    phys = s.table[b[:, None, None], sel.clamp(min=0)].long().clamp(min=0)
    h = torch.arange(s.Hkv, device=s.q.device)[:, None]
    k = s.kc[phys, h].reshape(s.T, s.Hkv, s.K * ps, s.d).float()
    v = s.vc[phys, h].reshape(s.T, s.Hkv, s.K * ps, s.d).float()
    where = (sel[..., None] * ps + torch.arange(ps, device=s.q.device)).reshape(s.T, s.Hkv, -1)
    pos = (s.seq - s.new_lens)[b] + at
    seen = (where >= 0) & (where <= pos[:, None, None])
    score = torch.matmul(s.q.float().reshape(s.T, s.Hkv, G, s.d), k.transpose(-1, -2)) * s.scale
    o, lse = _softmax_v(score, seen[:, :, None], torch.where(seen[..., None], v, 0.0))
    live = t < s.cu[-1]
    return (torch.where(live[:, None, None], o.reshape(s.T, s.Hq, s.d).bfloat16(), s.o),
            torch.where(live[:, None], lse.reshape(s.T, s.Hq), s.lse))


# -------------------------------------------------------------- one pass --
def run(s):
    if own:
        return _own(s)
    return dict(tables=_plain_tables, append=_plain_append, fwd=_plain_fwd, select=_plain_select,
                sparse=_plain_sparse)[s.op](s)


def _own(s):
    import exact_io_aware_70_b200 as ea
    if s.op == "tables":
        ea.attn_page_tables(s.ctx_lens, s.new_lens, s.free_pages, s.free_head, s.free_out,
                            s.old_table, s.seq_out, s.cu_out, s.slots, s.ps, s.num_pages)
        return s.old_table, s.seq_out, s.cu_out, s.slots, s.free_out
    if s.op == "append":
        ea.attn_paged_append(s.k, s.v, s.slots, s.kc, s.vc, s.bounds)
        return s.kc, s.vc, s.bounds
    if s.op == "fwd":
        if s.ws is None:
            s.ws = torch.empty(ea.attn_fwd_paged_workspace_bytes(s.d), dtype=torch.uint8,
                               device="cuda")
        ea.attn_fwd_paged(s.q, s.kc, s.vc, s.table, s.cu, s.seq, s.o, s.lse, True, s.scale, s.ws)
        return s.o, s.lse
    if s.op == "select":
        if s.ws is None:
            s.ws = torch.empty(ea.attn_page_select_workspace_bytes(s.T, s.Hkv, s.max_pages),
                               dtype=torch.uint8, device="cuda")
        ea.attn_page_select(s.q, s.bounds, s.table, s.cu, s.seq, s.sel, s.ps, s.first, s.last,
                            s.ws)
        return s.sel
    if s.ws is None:
        s.ws = torch.empty(ea.attn_fwd_paged_workspace_bytes(s.d), dtype=torch.uint8,
                           device="cuda")
    ea.attn_sparse_paged(s.q, s.kc, s.vc, s.table, s.cu, s.seq, s.sel, s.o, s.lse, s.scale, s.ws)
    return s.o, s.lse


# ------------------------------------------------- the definition in 64 bits --
def exact(c, seed):
    """What run() returns, from the definitions, one sequence after another in 64 bits."""
    s = prepare(c, seed)
    new, ctx = _lens(c)
    ps = c["ps"]
    if c["op"] == "tables":
        table = s.old_table.cpu().tolist()
        free = s.free_pages.tolist()
        head, slots, cu = 5, [], [0]
        for b, (n, x) in enumerate(zip(new, ctx)):
            for j in range(x, x + n):
                if j % ps == 0:
                    table[b][j // ps] = free[head]
                    head += 1
                slots.append(table[b][j // ps] * ps + j % ps)
            cu.append(len(slots))
        slots += [-1] * c["pad"]
        return (torch.tensor(table, dtype=torch.int32),
                torch.tensor([n + x for n, x in zip(new, ctx)], dtype=torch.int32),
                torch.tensor(cu, dtype=torch.int32), torch.tensor(slots),
                torch.tensor([head], dtype=torch.int32))
    if c["op"] == "append":
        kc, vc, bounds = s.kc.double(), s.vc.double(), s.bounds.double()
        row = 0
        for b, (n, x) in enumerate(zip(new, ctx)):
            for first in range(x // ps, _pages(x + n, ps)):
                page = int(s.table[b, first])
                j0, j1 = max(x, first * ps), min(x + n, first * ps + ps)
                r = slice(row + j0 - x, row + j1 - x)
                kc[page, :, j0 - first * ps:j1 - first * ps] = s.k[r].double().transpose(0, 1)
                vc[page, :, j0 - first * ps:j1 - first * ps] = s.v[r].double().transpose(0, 1)
                there = kc[page, :, :j1 - first * ps]
                bounds[page, :, 0], bounds[page, :, 1] = there.amin(1), there.amax(1)
            row += n
        return kc, vc, bounds
    G = c["Hq"] // c["Hkv"]
    if c["op"] == "select":
        out = s.sel.clone()
        for b, (n, x) in enumerate(zip(new, ctx)):
            pages = s.table[b, :_pages(n + x, ps)].long()
            vis = (x + torch.arange(n, device="cuda")) // ps + 1
            j = torch.arange(len(pages), device="cuda")
            for h in range(c["Hkv"]):
                bound = s.bounds[pages, h].double()                      # [pages, 2, d]
                best = torch.full((n, len(pages)), -INF, dtype=torch.float64, device="cuda")
                for a in range(G):
                    q = s.q[int(s.cu[b]):int(s.cu[b]) + n, h * G + a].double()
                    for r in range(0, n, 256):
                        part = torch.where(q[r:r + 256, None] >= 0, q[r:r + 256, None] * bound[:, 1],
                                           q[r:r + 256, None] * bound[:, 0]).sum(-1)
                        best[r:r + 256] = torch.maximum(best[r:r + 256], part)
                best[(j < c["first"]) | (j >= vis[:, None] - c["last"])] = INF
                best[j >= vis[:, None]] = -INF
                rank = torch.argsort(-best, dim=1, stable=True)
                chosen = torch.zeros_like(best, dtype=torch.bool)
                chosen.scatter_(1, rank[:, :c["K"]], True)
                chosen &= j < vis[:, None]
                order = torch.where(chosen, j, len(pages)).sort(1).values[:, :c["K"]]
                row = torch.full((n, c["K"]), -1, dtype=torch.int32, device="cuda")
                row[:, :order.shape[1]] = torch.where(order < len(pages), order, -1).int()
                out[int(s.cu[b]):int(s.cu[b]) + n, h] = row
        return out
    o, lse = s.o.double(), s.lse.double()
    for b, (n, x) in enumerate(zip(new, ctx)):
        rows = slice(int(s.cu[b]), int(s.cu[b]) + n)
        pages = s.table[b, :_pages(n + x, ps)].long()
        j = torch.arange(len(pages) * ps, device="cuda")
        pos = x + torch.arange(n, device="cuda")
        for h in range(c["Hkv"]):
            k = s.kc[pages, h].reshape(-1, c["d"]).double()
            v = s.vc[pages, h].reshape(-1, c["d"]).double()
            seen = (j <= pos[:, None]) & (j < n + x)
            if c["op"] == "sparse":   # no page is listed twice
                listed_ = torch.zeros((n, len(pages) + 1), dtype=torch.bool, device="cuda")
                pick = s.sel[rows, h].long()
                listed_.scatter_(1, torch.where(pick < 0, len(pages), pick), True)
                seen = seen & listed_[:, :-1].repeat_interleave(ps, 1)
            v[n + x:] = 0
            for a in range(h * G, h * G + G):
                score = (s.q[rows, a].double() @ k.T) * s.scale
                score.masked_fill_(~seen, -INF)
                lse[rows, a] = torch.logsumexp(score, 1)
                o[rows, a] = torch.exp(score - lse[rows, a, None]) @ v
    return o, lse
