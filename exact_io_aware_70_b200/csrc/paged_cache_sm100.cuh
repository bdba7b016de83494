// paged_cache_sm100.cuh -- what surrounds attention over a paged K/V cache:
// block tables and slots of a step's tokens, the write of their K and V with
// each page's key bounds, and the choice of the pages a query reads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "decode_sm100.cuh"
#include "ptx_sm100.cuh"

namespace eattn {

// ----------------------------------------------------- a step's sequences --
struct PagedSeq {
    int tok, n, len;   // first row, new tokens, cached keys; all clamped to the tensors
    bool bad;
};

// Sequence b of a call with parameters p (offsets, lengths and the sizes that bound them).
template <class Params>
__device__ __forceinline__ PagedSeq paged_seq(const Params& p, int b) {
    PagedSeq s;
    const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), l = __ldg(p.seq_lens + b);
    const int cap = p.max_pages << p.page_shift;
    s.tok = min(max(c0, 0), p.T);
    s.n = min(max(c1, s.tok), p.T) - s.tok;
    s.len = min(max(l, 0), cap);
    s.bad = s.tok != c0 || s.tok + s.n != c1 || s.len != l;
    return s;
}

// ---------------------------------------------------------- block tables --
// Sequence b holds ctx[b] tokens and gets new[b] more. With cu the exclusive
// prefix sum of new and P that of the pages each one lacks,
//   lacks[b] = ceil((ctx + new) / ps) - ceil(ctx / ps),
// the i-th page it lacks is free_pages[head + P[b] + i], and its k-th new
// token is row cu[b] + k of the step, at slot page * ps + (ctx + k) % ps.
//
// The work is small (a few words per token), so what counts is the number of
// launches and of dependent steps: one cluster of CTAs does it all. Every CTA
// scans the lengths for itself into shared memory (no exchange between CTAs,
// the lengths come from L2) and then takes its share of the rows, finding a
// row's sequence by bisection. The cluster barrier lies between the last read
// of the lengths and of the free list's head and the first write of lengths,
// offsets and head, so those may be updated in place, and a captured graph can
// run step after step.
constexpr int kTablesThreads = 1024;
constexpr int kTablesMaxSeqs = 8192;    // three words of shared memory each

struct TablesParams {
    const int* ctx_lens;     // [B]
    const int* new_lens;     // [B]
    const int* free_pages;   // [F]
    const int* free_head;    // [1]
    int* free_head_out;      // [1], may be free_head
    int* block_table;        // [B, max_pages]
    int* seq_lens;           // [B], may be ctx_lens
    int* cu_q;               // [B + 1]
    long long* slot_map;     // [T]
    int B, T, F, page_shift, max_pages, num_pages;
};

// Inclusive sums of a and b over the block; `tot`: the block's totals.
__device__ __forceinline__ void block_scan(int& v, int& tot, int* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
    }
    __syncthreads();   // the last scan's reads of red are done
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int x = lane < warps ? red[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += u;
    }
    tot = __shfl_sync(0xffffffffu, x, 31);
    const int before = __shfl_sync(0xffffffffu, x, (warp + 31) & 31);
    if (warp > 0) v += before;
}

// a + b, at most `top`, for a and b in [0, top]: in 32 bits without a sign, as two row counts of
// 2^30 (the largest T) add up to 2^31.
__device__ __forceinline__ int sum_to(int a, int b, int top) {
    return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)top);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kTablesThreads) attn_page_tables_kernel(const TablesParams p) {
    extern __shared__ int s_tab[];
    int* s_cu = s_tab;                // [B + 1]
    int* s_ctx = s_cu + p.B + 1;      // [B]
    int* s_page = s_ctx + p.B;        // [B]: pages taken by the sequences before
    __shared__ int red[32];
    const int tid = threadIdx.x;
    const uint32_t rank = cluster_rank();
    const int ps = 1 << p.page_shift;
    const int cap = p.max_pages << p.page_shift;
    const int raw_head = *p.free_head;
    const bool head_ok = raw_head >= 0 && raw_head <= p.F;
    const int head = head_ok ? raw_head : p.F;   // an invalid head: nothing to give
    unsigned bad = head_ok ? 0 : kDevErrBadIndex;
    int rows = 0, pages = 0;          // sums over the sequences before this round
    for (int b0 = 0; b0 < p.B; b0 += kTablesThreads) {
        const int b = b0 + tid;
        int ctx = 0, add = 0;
        if (b < p.B) {
            ctx = p.ctx_lens[b];
            add = p.new_lens[b];
            if (ctx < 0 || add < 0 || (long long)ctx + add > cap) {
                bad = kDevErrBadIndex;
                ctx = min(max(ctx, 0), cap);
                add = 0;
            }
        }
        // sums saturate at T: rows past the buffer are cut off, tokens with them
        int end = min(add, p.T), tot;
        {
            const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, end, off);
                if (lane >= off) end = sum_to(end, u, p.T);
            }
            __syncthreads();
            if (lane == 31) red[warp] = end;
            __syncthreads();
            int x = red[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x = sum_to(x, u, p.T);
            }
            tot = __shfl_sync(0xffffffffu, x, 31);
            const int before = __shfl_sync(0xffffffffu, x, (warp + 31) & 31);
            if (warp > 0) end = sum_to(end, before, p.T);
        }
        end = sum_to(end, rows, p.T);
        // where this sequence's rows begin: the end of the one before
        __syncthreads();
        if (b < p.B) s_cu[b + 1] = end;
        if (b0 == 0 && tid == 0) s_cu[0] = 0;
        __syncthreads();
        const int start = b < p.B ? s_cu[b] : 0;
        const int got = b < p.B ? end - start : 0;
        if (got < add) bad = kDevErrBadIndex;
        const int need = ((ctx + got + ps - 1) >> p.page_shift) - ((ctx + ps - 1) >> p.page_shift);
        int v = need, ptot;
        block_scan(v, ptot, red);
        if (b < p.B) {
            s_ctx[b] = ctx;
            s_page[b] = pages + v - need;
        }
        rows = sum_to(rows, tot, p.T);
        pages += ptot;
    }
    if (bad) atomicOr(&g_attn_status, bad);
    cluster_sync_all();   // every CTA has read the lengths and the head (and its own scan is done)
    if (rank == 0) {
        for (int b = tid; b < p.B; b += kTablesThreads) {
            p.seq_lens[b] = s_ctx[b] + s_cu[b + 1] - s_cu[b];
            p.cu_q[b] = s_cu[b];
        }
        if (tid == 0) {
            p.cu_q[p.B] = rows;
            *p.free_head_out = (int)min((long long)head + pages, (long long)p.F);
        }
    }
    bad = 0;
    // (four rows in turn per thread, with their page numbers read together, was slower: 11.2
    // against 10.0 us on 47,000 rows of 500 sequences)
    const int step = gridDim.x * kTablesThreads;
    for (int t = rank * kTablesThreads + tid; t < p.T; t += step) {
        long long slot = -1;
        if (t < rows) {
            int lo = 0, hi = p.B;     // the last b with s_cu[b] <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int ctx = s_ctx[lo], pos = ctx + t - s_cu[lo];
            const int lp = pos >> p.page_shift, first = (ctx + ps - 1) >> p.page_shift;
            int* entry = p.block_table + (size_t)lo * p.max_pages + lp;
            if (dcheck(lp < p.max_pages)) {
                int page;
                if (lp >= first) {    // a page this step takes; its first token enters it
                    const long long i = (long long)head + s_page[lo] + lp - first;
                    page = i < p.F ? __ldg(p.free_pages + i) : -1;
                    if (page < 0 || page >= p.num_pages) page = -1;
                    if ((pos & (ps - 1)) == 0) *entry = page;
                } else {
                    page = *entry;
                    if (page >= p.num_pages) page = -1;
                }
                if (page < 0) bad = kDevErrBadIndex;
                else slot = ((long long)page << p.page_shift) + (pos & (ps - 1));
            }
        }
        p.slot_map[t] = slot;
    }
    if (bad) atomicOr(&g_attn_status, bad);
}

// ---------------------------------------------------------------- append --
// K and V rows copied to their slots, and the bounds of every page written to:
//   bounds[page][h][0][c] = min, [1][c] = max over the page's slots 0 .. s of
//   K[slot][h][c], s the last slot written (bf16, exact; a NaN key gives NaN).
// A page's tokens are a run of consecutive rows; the run's last row sees to the
// bounds, taking a key from the new rows where they hold it and from the
// cache where an earlier step wrote it. So no CTA waits for another's writes.
// Bytes are all there is to it: 16-byte loads and stores, K and V of a row in
// flight together.
struct AppendParams {
    const uint16_t* k;           // bf16 [T, Hkv, D], kv_stride elements from row to row
    const uint16_t* v;
    const long long* slot_map;   // [T]
    uint16_t* k_cache;           // bf16 [num_pages, Hkv, ps, D]
    uint16_t* v_cache;
    uint16_t* bounds;            // bf16 [num_pages, Hkv, 2, D] or null
    long long kv_stride, num_slots;
    int T, Hkv, page_shift;
};

constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t bf2_min_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Block (x, h): rows [x * ROWS, + ROWS) of head h.
template <int D, int ROWS>
__global__ void __launch_bounds__(kAppendThreads) attn_paged_append_kernel(const AppendParams p) {
    static_assert(ROWS <= 32, "a warp looks at all of a block's rows");
    constexpr int kPieces = D / 8;                        // 16-byte pieces of a row
    constexpr int kSlots = kAppendThreads / kPieces;      // rows per pass
    __shared__ uint4 s_red[2][kAppendThreads / 32][kPieces];
    const int tid = threadIdx.x, piece = tid % kPieces, rs = tid / kPieces;
    const int lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y;
    const int t0 = blockIdx.x * ROWS, t1 = min(t0 + ROWS, p.T);
    const int ps = 1 << p.page_shift;
    const long long head_off = (long long)h * D + piece * 8;
    // element of the cache at slot s, this head and piece
    auto at = [&](long long s) -> size_t {
        return ((((size_t)(s >> p.page_shift) * p.Hkv + h) << p.page_shift) + (s & (ps - 1))) * D +
               piece * 8;
    };
    unsigned bad = 0;
    auto slot_of = [&](int t) -> long long {
        const long long s = __ldg(p.slot_map + t);
        if (s >= p.num_slots) {
            bad = kDevErrBadIndex;
            return -1;
        }
        return s;
    };
    constexpr int kPasses = (ROWS + kSlots - 1) / kSlots;
    {
        uint4 kr[kPasses], vr[kPasses];
        long long sl[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int t = t0 + rs + i * kSlots;
            sl[i] = t < t1 ? slot_of(t) : -1;
            if (sl[i] >= 0) {
                const size_t src = (size_t)t * p.kv_stride + head_off;
                kr[i] = __ldg(reinterpret_cast<const uint4*>(p.k + src));
                vr[i] = __ldg(reinterpret_cast<const uint4*>(p.v + src));
            }
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
            if (sl[i] >= 0 && dcheck(sl[i] < p.num_slots)) {
                *reinterpret_cast<uint4*>(p.k_cache + at(sl[i])) = kr[i];
                *reinterpret_cast<uint4*>(p.v_cache + at(sl[i])) = vr[i];
            }
    }
    if (p.bounds) {
        // the rows that end their page's run (ROWS <= 32: each warp finds all of them)
        unsigned ends;
        {
            const int t = t0 + lane;
            const long long s = t < t1 ? slot_of(t) : -1;
            const long long nx = t + 1 < p.T && t < t1 ? __ldg(p.slot_map + t + 1) : -1;
            ends = __ballot_sync(0xffffffffu, s >= 0 && (nx < 0 || (nx >> p.page_shift) !=
                                                                       (s >> p.page_shift)));
        }
        for (; ends; ends &= ends - 1) {
            // reduce the page's slots 0 .. s % ps
            const int t = t0 + __ffs(ends) - 1;
            const long long s = __ldg(p.slot_map + t);
            const int last = (int)(s & (ps - 1));
            uint4 lo, hi;
            bool any = false;
#pragma unroll 4
            for (int r = rs; r <= last; r += kSlots) {
                const int u = t - (last - r);
                const long long want = s - (last - r);
                const bool fresh = u >= 0 && __ldg(p.slot_map + u) == want;
                const uint4 x = fresh ? __ldg(reinterpret_cast<const uint4*>(
                                            p.k + (size_t)u * p.kv_stride + head_off))
                                      : *reinterpret_cast<const uint4*>(p.k_cache + at(want));
                if (!any) {
                    lo = hi = x;
                    any = true;
                } else {
                    lo.x = bf2_min_nan(lo.x, x.x); lo.y = bf2_min_nan(lo.y, x.y);
                    lo.z = bf2_min_nan(lo.z, x.z); lo.w = bf2_min_nan(lo.w, x.w);
                    hi.x = bf2_max_nan(hi.x, x.x); hi.y = bf2_max_nan(hi.y, x.y);
                    hi.z = bf2_max_nan(hi.z, x.z); hi.w = bf2_max_nan(hi.w, x.w);
                }
            }
            if (!any) {   // the neutral elements: +inf, -inf
                lo = make_uint4(0x7F807F80u, 0x7F807F80u, 0x7F807F80u, 0x7F807F80u);
                hi = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
            }
            auto fold = [](uint4& a, uint4& b, const uint4& x, const uint4& y) {
                a.x = bf2_min_nan(a.x, x.x); a.y = bf2_min_nan(a.y, x.y);
                a.z = bf2_min_nan(a.z, x.z); a.w = bf2_min_nan(a.w, x.w);
                b.x = bf2_max_nan(b.x, y.x); b.y = bf2_max_nan(b.y, y.y);
                b.z = bf2_max_nan(b.z, y.z); b.w = bf2_max_nan(b.w, y.w);
            };
#pragma unroll
            for (int off = 16; off >= kPieces; off >>= 1) {
                uint4 x, y;
                x.x = __shfl_xor_sync(0xffffffffu, lo.x, off);
                x.y = __shfl_xor_sync(0xffffffffu, lo.y, off);
                x.z = __shfl_xor_sync(0xffffffffu, lo.z, off);
                x.w = __shfl_xor_sync(0xffffffffu, lo.w, off);
                y.x = __shfl_xor_sync(0xffffffffu, hi.x, off);
                y.y = __shfl_xor_sync(0xffffffffu, hi.y, off);
                y.z = __shfl_xor_sync(0xffffffffu, hi.z, off);
                y.w = __shfl_xor_sync(0xffffffffu, hi.w, off);
                fold(lo, hi, x, y);
            }
            __syncthreads();   // the last run's reads of s_red are done
            if (lane < kPieces) {
                s_red[0][warp][lane] = lo;
                s_red[1][warp][lane] = hi;
            }
            __syncthreads();
            if (tid < kPieces) {
                lo = s_red[0][0][tid];
                hi = s_red[1][0][tid];
#pragma unroll
                for (int w = 1; w < kAppendThreads / 32; ++w) fold(lo, hi, s_red[0][w][tid], s_red[1][w][tid]);
                uint16_t* dst = p.bounds +
                                ((size_t)(s >> p.page_shift) * p.Hkv + h) * 2 * D + tid * 8;
                *reinterpret_cast<uint4*>(dst) = lo;
                *reinterpret_cast<uint4*>(dst + D) = hi;
            }
        }
    }
    if (bad) atomicOr(&g_attn_status, bad);
}

// ---------------------------------------------------------------- select --
// Every query row t and K/V head hk gets the K pages whose keys can score
// highest. For a page with bounds lo <= k <= hi (channel by channel),
//   q . k <= sum_c (q_c >= 0 ? q_c hi_c : q_c lo_c) = [min(q, 0), max(q, 0)] . [lo, hi],
// and a page's score is the largest such bound over the G query heads that
// share hk: a matrix product with 2 D terms, then a maximum. The choice has to be
// that of exact scores (equal ones from the lowest page up), and 32-bit sums do
// not tell near ones apart, so it is made in two steps:
//   1. attn_page_score_kernel: the product on the tensor cores (bf16 products are
//      exact, sums fp32), with a bound E of its error per row.
//   2. attn_page_topk_kernel: a row's K-th largest score s, found bit by bit. A page
//      above s + 2 E is chosen and one below s - 2 E is not, whatever the rounding;
//      the few between are scored again in fp64 (where the sum of a row's exact products
//      is all but exact) and the best of them fill up the choice.
// Scoring every page in fp64 ran 287 us on 1098 rows x 8 K/V heads x up to 246 pages
// (0.8e9 terms for 32 query heads); this way the choice takes 55.
struct SelectParams {
    const uint16_t* q;          // bf16 [T, Hq, D], q_stride elements from row to row
    const uint16_t* bounds;     // bf16 [num_pages, Hkv, 2, D]
    const int* block_table;     // [B, max_pages]
    const int* cu_q;            // [B + 1]
    const int* seq_lens;        // [B]
    int* sel;                   // [T, Hkv, K]
    unsigned long long* keys;   // [T, Hkv, max_pages]: scores (fp32), then exact keys of a few
    float* err;                 // [T, Hkv, score tiles]: error bounds
    long long q_stride;
    int B, T, Hq, Hkv, G, K, first, last;
    int page_shift, max_pages, num_pages, tiles;
    int tile_tok;               // tokens of a score tile
};

struct SelectRow {
    int b, end;       // sequence (-1: none), the row after its last one
    int pos, pages;   // the row's position, and the pages it sees
};

// The sequence of row t, where its rows end and how many pages the row sees; by a whole warp.
__device__ __forceinline__ SelectRow select_row(const SelectParams& p, int t, int lane) {
    SelectRow r;
    r.b = -1;
    r.pages = r.end = 0;
    // the last b with cu[b] <= t, 32 places at a time
    int lo = 0, n = p.B;          // it is in [lo, lo + n), or t lies before the first row
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool le = lane * step < n && (lane == 0 || __ldg(p.cu_q + at) <= t);
        const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;   // (offsets ascend)
        lo += k * step;
        n = min(step, n - k * step);
    }
    const int c0 = __ldg(p.cu_q + lo), c1 = __ldg(p.cu_q + lo + 1), l = __ldg(p.seq_lens + lo);
    if (t < c0 || t >= c1) return r;   // before the first, past the last, or offsets that do not ascend
    const int len = min(max(l, 0), p.max_pages << p.page_shift);
    r.b = lo;
    r.end = min(c1, p.T);          // (as paged_seq clamps it: the positions agree with the attention's)
    r.pos = len - r.end + t;
    r.pages = r.pos < 0 ? 0 : (r.pos >> p.page_shift) + 1;
    return r;
}

__device__ __forceinline__ unsigned long long order_key(double x) {
    // ascending keys for ascending scores; NaN ranks above all scores
    if (x != x) return ~0ull;
    const unsigned long long u = (unsigned long long)__double_as_longlong(x);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}
// The same in 32 bits. Never 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return ~0u;
    const uint32_t u = __float_as_uint(x);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes from global to shared memory, zeros where !valid (src must be readable memory still).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Block (x, hk): pages [64 (x % tiles), + 64) for the tile_tok tokens from (x / tiles) *
// tile_tok on, one sequence of them after another. ROWS = 64 or 16 rows (token, head of the
// group) at a time against 64 pages, 2 D terms: 64 or 40 KB of shared memory at D = 128. The
// bounds come by asynchronous copies, all of a tile's at once (through registers, eight at a
// time, the choice for 16 tokens of 512 pages took 3.4 us longer). What
// bounds it is the read of q and of the bounds (each tile of pages is read once per ROWS
// rows), so the products are left to mma.sync, which needs no set-up.
constexpr int kScorePages = 64;
// Threads of a block: its time is that of dependent steps (lookup, loads, products, maxima), so
// 64 rows get eight warps (38 us against 45 with four, at 1,098 tokens of 32 heads on 8 and up
// to 246 pages); 16 rows, whose blocks are small, gain nothing by them (29.6 against 30.3 us for
// the whole choice at 16 tokens and 512 pages).
template <int ROWS>
constexpr int kScoreThreads = ROWS == 64 ? 256 : 128;

// Bytes of the first operand, or of the scores that take its place (at D = 64 they are larger).
template <int D, int ROWS>
constexpr int kScoreABytes = (ROWS * (4 * D > 65 * 4 ? 4 * D : 65 * 4) + 127) / 128 * 128;

// Where a sum of squares begins, so that squares too small for 32 bits (and what
// 2^-126 cuts off elsewhere) do not make a bound of 0 for numbers that are not.
__device__ __forceinline__ float least_sum(const uint32_t (&w)[4]) {
    return ((w[0] | w[1] | w[2] | w[3]) & 0x7FFF7FFFu) ? 0x1p-100f : 0.f;
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kScoreThreads<ROWS>) attn_page_score_kernel(const SelectParams p) {
    constexpr int kThreads = kScoreThreads<ROWS>;
    constexpr int kTerms = 2 * D, kRowBytes = 2 * kTerms, kChunks = kRowBytes / 16;
    constexpr int kParts = kThreads / kScorePages;        // threads that look at one page's sum
    extern __shared__ __align__(128) uint8_t s_tiles[];
    uint8_t* sA = s_tiles;                                // [ROWS][2 D] bf16, 16-byte chunks swizzled
    uint8_t* sB = s_tiles + kScoreABytes<D, ROWS>;        // [64 pages][2 D]
    float* sS = reinterpret_cast<float*>(s_tiles);        // [ROWS][65] scores, over A when it is done
    __shared__ float s_sum[ROWS], s_red[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hk = blockIdx.y, tok_tile = blockIdx.x / p.tiles, tile = blockIdx.x - tok_tile * p.tiles;
    const int page0 = tile * kScorePages;
    const int t0 = tok_tile * p.tile_tok, t1 = min(t0 + p.tile_tok, p.T);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the choice waits by itself
    auto at = [](int row, int chunk) { return row * kRowBytes + ((chunk ^ (row & 7)) << 4); };

    for (int t = t0; t < t1;) {
        const SelectRow first = select_row(p, t, lane);
        if (first.b < 0) {
            ++t;
            continue;
        }
        // tokens [t, te) belong to this sequence; the last one sees most pages
        const int te = min(t1, first.end), last_pos = first.pos + te - 1 - t;
        const int pages = last_pos < 0 ? 0 : (last_pos >> p.page_shift) + 1;
        if (page0 >= pages) {
            t = te;
            continue;
        }
        __syncthreads();          // the last round's reads of shared memory are done
        // ---- bounds of the tile's pages, all on their way before the first is waited for
        {
            constexpr int kRowsPerPass = kThreads / kChunks, kPasses = kScorePages / kRowsPerPass;
            const int c = tid % kChunks, r0 = tid / kChunks;
            int page[kPasses];
#pragma unroll
            for (int k = 0; k < kPasses; ++k) {
                const int lp = page0 + r0 + k * kRowsPerPass;
                page[k] = lp < pages ? __ldg(p.block_table + (size_t)first.b * p.max_pages + lp) : -1;
            }
#pragma unroll
            for (int k = 0; k < kPasses; ++k) {
                const bool valid = page[k] >= 0 && page[k] < p.num_pages;
                const size_t row = (size_t)(valid ? page[k] : 0) * p.Hkv + hk;
                cp_async16(smem_addr(sB) + at(r0 + k * kRowsPerPass, c), p.bounds + row * kTerms + 8 * c,
                           valid);
            }
        }
        bool fresh = true;        // until the first round has waited for them

        // ---- its rows, as many tokens at a time as fit ROWS (G > ROWS: one, in rounds)
        const int sub = max(1, ROWS / p.G);
        for (int s0 = t; s0 < te; s0 += sub) {
        const int rows = (min(te, s0 + sub) - s0) * p.G;
        float best = -INFINITY;       // G > ROWS: of this thread's page, over the rounds
        for (int r0 = 0; r0 < rows; r0 += ROWS) {
            constexpr int kHalf = kChunks / 2, kLoads = ROWS * kHalf / kThreads;
            uint4 x[kLoads];       // all in flight before the first is used
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int row = tid / kHalf + k * (kThreads / kHalf);
                x[k] = make_uint4(0, 0, 0, 0);
                if (r0 + row < rows) {
                    const int tk = (r0 + row) / p.G, h = r0 + row - tk * p.G;
                    x[k] = __ldg(reinterpret_cast<const uint4*>(
                                     p.q + (size_t)(s0 + tk) * p.q_stride +
                                     (size_t)(hk * p.G + h) * D) + tid % kHalf);
                }
            }
            __syncthreads();          // (the last reads of A, scores and sums)
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int row = tid / kHalf + k * (kThreads / kHalf), c = tid % kHalf;
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                uint32_t neg[4], pos[4];
                float sum = least_sum(w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = bf16_lo(w[j]), b = bf16_hi(w[j]);
                    sum = fmaf(a, a, fmaf(b, b, sum));
                    // (a NaN goes with the negative part)
                    const uint32_t keep = (a >= 0.f ? 0x0000FFFFu : 0u) | (b >= 0.f ? 0xFFFF0000u : 0u);
                    pos[j] = w[j] & keep;
                    neg[j] = w[j] & ~keep;
                }
                *reinterpret_cast<uint4*>(sA + at(row, c)) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
                *reinterpret_cast<uint4*>(sA + at(row, c + kHalf)) =
                    make_uint4(pos[0], pos[1], pos[2], pos[3]);
                // the row's threads are neighbours in a warp
#pragma unroll
                for (int off = 1; off < kHalf; off <<= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (c == 0) s_sum[row] = sum;
            }
            if (fresh) cp_async_wait_all();
            __syncthreads();
            if (fresh) {
                // largest sum of squares of a page's terms [part, part + 1) * kTerms / kParts, a part
                // and 32 pages per warp: the sum of the parts' largest bounds every page's
                constexpr int kPart = kChunks / kParts;
                const int row = tid % kScorePages, c0 = tid / kScorePages * kPart;
                float sum = 0.f;
#pragma unroll 4
                for (int k = 0; k < kPart; ++k) {
                    const uint4 b = *reinterpret_cast<const uint4*>(sB + at(row, c0 + k));
                    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
                    sum += least_sum(w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sum = fmaf(bf16_lo(w[j]), bf16_lo(w[j]), sum);
                        sum = fmaf(bf16_hi(w[j]), bf16_hi(w[j]), sum);
                    }
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    sum = fmaxf(sum, __shfl_xor_sync(0xffffffffu, sum, off));
                if (lane == 0) s_red[warp] = sum;
                fresh = false;
            }
            // ---- warp w: 16 of the rows against 32 pages (ROWS = 64) or 16 pages
            constexpr int kN = ROWS == 64 ? 2 : 1;    // groups of 16 pages per warp
            const int wr = ROWS == 64 ? 16 * (warp & 3) : 0;
            const int wp = ROWS == 64 ? 32 * (warp >> 2) : 16 * warp;
            float acc[2 * kN][4];
#pragma unroll
            for (int n = 0; n < 2 * kN; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[n][k] = 0.f;
            const uint32_t a0 = smem_addr(sA), b0 = smem_addr(sB);
#pragma unroll 8
            for (int kk = 0; kk < kTerms / 16; ++kk) {
                uint32_t a[4];
                ldmatrix_x4(a0 + at(wr + (lane & 15), 2 * kk + (lane >> 4)), a);
#pragma unroll
                for (int n = 0; n < kN; ++n) {    // two groups of 8 pages each
                    uint32_t b[4];
                    ldmatrix_x4(b0 + at(wp + 16 * n + (lane & 7) + ((lane >> 4) << 3),
                                        2 * kk + ((lane >> 3) & 1)), b);
                    mma_16816(acc[2 * n], a, b[0], b[1]);
                    mma_16816(acc[2 * n + 1], a, b[2], b[3]);
                }
            }
            __syncthreads();                      // A is read
#pragma unroll
            for (int n = 0; n < 2 * kN; ++n) {
                const int row = wr + (lane >> 2), col = wp + 8 * n + 2 * (lane & 3);
                sS[row * 65 + col] = acc[n][0];
                sS[row * 65 + col + 1] = acc[n][1];
                sS[(row + 8) * 65 + col] = acc[n][2];
                sS[(row + 8) * 65 + col + 1] = acc[n][3];
            }
            __syncthreads();
            // ---- the largest over a token's heads
            const int ntok = p.G <= ROWS ? rows / p.G : 1;
            const int heads = min(p.G, rows - r0 < ROWS ? rows - r0 : ROWS);
            const int in = p.G <= ROWS ? p.G : heads;
            for (int i = tid; i < ntok * kScorePages; i += kThreads) {
                const int tk = i / kScorePages, col = i - tk * kScorePages;
                float m = best;
                for (int h = 0; h < in; ++h) {
                    const float x = sS[(tk * p.G + h) * 65 + col];
                    m = (x > m || x != x) && m == m ? x : m;
                }
                if (p.G > ROWS && r0 + ROWS < rows) {
                    best = m;
                } else if (page0 + col < p.max_pages) {
                    const size_t row = (size_t)(s0 + tk) * p.Hkv + hk;
                    if (dcheck(s0 + tk < p.T))
                        reinterpret_cast<float*>(p.keys + row * p.max_pages)[page0 + col] = m;
                }
            }
            // ---- the error of these sums. How a product adds up is not documented; assumed is
            // that it takes steps of w >= 4 terms, each of which cuts its w + 1 numbers (the
            // terms, and the sum so far) and its result off below 2^-23 of the largest at worst:
            // (2 D / w) (w + 2) 2^-23 <= 64 * 6 * 2^-23 < 4.6e-5 times sum |q b| <= |q| |b|.
            // 5e-5 leaves room for the fp32 sums of squares (2^-15 of themselves), the roots and
            // s +- 2 E below (2^-23 |s|). |q| and |b| are both at least 2^-50 (least_sum), which
            // covers what products and sums lose below 2^-126 (2 D * 2^-126 <= 2^-118). 0: all
            // scores are exactly 0
            if (tid < ntok) {
                float sum = 0.f;
                for (int h = 0; h < in; ++h) sum = fmaxf(sum, s_sum[tid * p.G + h]);
                float b = 0.f;
                for (int w = 0; w < kParts; ++w) b += fmaxf(s_red[2 * w], s_red[2 * w + 1]);
                float e = sqrtf(sum) * sqrtf(b) * 5e-5f;
                float* dst = p.err + ((size_t)(s0 + tid) * p.Hkv + hk) * p.tiles + tile;
                if (r0 > 0) e = fmaxf(e, *dst);   // this thread's own, of the first heads
                if (dcheck(s0 + tid < p.T)) *dst = e;
            }
        }
        }
        t = te;
    }
}

// One group of THREADS threads per (t, hk), PER keys in each thread's registers.
template <int D, int THREADS, int PER>
__global__ void __launch_bounds__(THREADS == 32 ? 128 : THREADS)
    attn_page_topk_kernel(const SelectParams p) {
    constexpr int kGroups = THREADS == 32 ? 4 : 1;       // rows per block
    constexpr int kWarps = THREADS / 32;
    // heads whose exact scores are taken together: with few rows their latency sets the time (16
    // tokens of 512 pages: 24.9 us one by one, 24.0 so), with many the registers do
    constexpr int kHeads = THREADS == 128 ? 4 : 1;
    __shared__ int s_cnt[2][kWarps];
    const int tid = threadIdx.x % THREADS, lane = tid & 31, warp = tid >> 5;
    const long long rowi = (long long)blockIdx.x * kGroups + threadIdx.x / THREADS;
    // Launched while the scores are made, by blocks that have waited for all before them: offsets,
    // lengths and tables may be read at once, the scores once those blocks are done.
    const int t = (int)(rowi / p.Hkv), hk = (int)(rowi - (long long)t * p.Hkv);
    SelectRow row;
    row.b = -1;
    row.pages = 0;
    if (t < p.T) row = select_row(p, t, lane);
    const int* table = p.block_table + (size_t)max(row.b, 0) * p.max_pages;
    // thread i holds pages r * THREADS + i
    uint32_t keep = 0, open = 0;                         // bit r: always chosen / to be ranked
    int kept = 0, ranked = 0;
    bool bad = false;
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int lp = r * THREADS + tid;
        if (lp < row.pages) {
            const int page = __ldg(table + lp);
            if (page < 0 || page >= p.num_pages) {
                bad = true;
            } else if (lp < p.first || lp >= row.pages - p.last) {
                keep |= 1u << r;
                ++kept;
            } else {
                open |= 1u << r;
                ++ranked;
            }
        }
    }
    // lengths and offsets out of range: a share of the sequences per block
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < p.B; b += gridDim.x * blockDim.x)
        bad |= paged_seq(p, b).bad;
    if (bad) atomicOr(&g_attn_status, kDevErrBadIndex);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row.b < 0) return;                               // rows of no sequence stay as they were
    int* out = p.sel + rowi * p.K;
    unsigned long long* exact = p.keys + rowi * p.max_pages;
    int flip = 0;
    auto total = [&](int v) -> int {
        v = __reduce_add_sync(0xffffffffu, v);
        if (kWarps == 1) return v;
        if (lane == 0) s_cnt[flip][warp] = v;
        __syncthreads();
        v = 0;
        for (int w = 0; w < kWarps; ++w) v += s_cnt[flip][w];
        flip ^= 1;
        return v;
    };
    auto lowest = [&](uint32_t v) -> uint32_t {
        v = __reduce_min_sync(0xffffffffu, v);
        if (kWarps == 1) return v;
        if (lane == 0) s_cnt[flip][warp] = (int)v;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) v = min(v, (uint32_t)s_cnt[flip][w]);
        flip ^= 1;
        return v;
    };
    // position of this thread among those with `x`, and how many there are
    auto rank = [&](bool x, int& all) -> int {
        const unsigned m = __ballot_sync(0xffffffffu, x);
        int before = __popc(m & ((1u << lane) - 1));
        all = __popc(m);
        if (kWarps > 1) {
            if (lane == 0) s_cnt[flip][warp] = all;
            __syncthreads();
            all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += s_cnt[flip][w];
                all += s_cnt[flip][w];
            }
            flip ^= 1;
        }
        return before;
    };
    uint32_t key[PER];                                   // 0: not to be ranked
#pragma unroll
    for (int r = 0; r < PER; ++r)
        key[r] = (open >> r) & 1
                     ? order_key(reinterpret_cast<const float*>(exact)[r * THREADS + tid]) : 0;
    const int want = p.K - total(kept);                  // to be chosen by their scores
    ranked = total(ranked);
    float err = 0.f;
    for (int i = lane; i * kScorePages < row.pages; i += 32) err = fmaxf(err, p.err[rowi * p.tiles + i]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, off));

    // bit r: chosen for certain / to be ranked by exact keys
    uint32_t sure = keep, maybe = 0;
    int need = 0, unsure = 0;
    if (ranked <= want) {
#pragma unroll
        for (int r = 0; r < PER; ++r) sure |= (key[r] != 0) << r;
    } else if (want > 0) {
        // the want-th largest key: bit by bit, from the first in which two keys differ
        uint32_t most = 0, least = ~0u;
#pragma unroll
        for (int r = 0; r < PER; ++r) {
            most = max(most, key[r]);
            if (key[r]) least = min(least, key[r]);
        }
        least = lowest(least);
        most = ~lowest(~most);
        // A NaN score has no error bound (the bounds' maxima above leave NaN out), and it may be the
        // product's alone: 0 times an infinite bound on the side that q's sign does not take. So
        // with one in the row every page is undecided and the exact scores say what is what.
        if (most == ~0u) err = INFINITY;
        const int bits = 32 - __clz(least ^ most);
        uint32_t kth = bits == 32 ? 0 : (most >> bits) << bits;
        for (int bit = bits - 1; bit >= 0; --bit) {
            const uint32_t cand = kth | (1u << bit);
            int n = 0;
#pragma unroll
            for (int r = 0; r < PER; ++r) n += key[r] >= cand;
            n = total(n);
            if (n >= want) kth = cand;
            if (n == want) {                             // it is the least of these
                uint32_t low = ~0u;
#pragma unroll
                for (int r = 0; r < PER; ++r)
                    if (key[r] >= cand) low = min(low, key[r]);
                kth = lowest(low);
                break;
            }
        }
        const float s = key_value(kth);
        const float above = s + 2.0f * err, below = s - 2.0f * err;
        int n = 0, m = 0;
#pragma unroll
        for (int r = 0; r < PER; ++r) {
            const float v = key_value(key[r]);
            // (comparisons with NaN are false: undecided)
            const bool yes = key[r] != 0 && v > above, no = key[r] == 0 || v < below;
            sure |= (uint32_t)yes << r;
            maybe |= (uint32_t)(!yes && !no) << r;
            n += yes;
            m += !yes && !no;
        }
        need = want - total(n);
        unsure = total(m);
        if (unsure <= need) {
            sure |= maybe;
            maybe = 0;
        }
    }
    // ---- exact keys of the undecided pages, in page order
    unsigned long long kth = 0;
    int ties = 0;
    unsigned picked = 0;          // of up to 32 undecided pages
    if (unsure > need) {
        __syncwarp();
        if (kWarps > 1) __syncthreads();                 // all scores are in registers
        int base = 0;
#pragma unroll 1
        for (int r = 0; r * THREADS < row.pages; ++r) {
            int all;
            const int before = rank((maybe >> r) & 1, all);
            if (all == 0) continue;
            unsigned m = __ballot_sync(0xffffffffu, (maybe >> r) & 1);
            while (m && err == 0.f) {                    // no rounding at all: they are equal
                const int src = __ffs(m) - 1;
                m &= m - 1;
                const int place = base + __shfl_sync(0xffffffffu, before, src);
                if (lane == 0 && dcheck(place < p.max_pages)) exact[place] = 1;
            }
            while (m) {                                  // a warp scores its own pages
                const int src = __ffs(m) - 1;
                m &= m - 1;
                const int lp = r * THREADS + warp * 32 + src;
                const uint16_t* bnd = p.bounds + ((size_t)__ldg(table + lp) * p.Hkv + hk) * 2 * D;
                float lo[D / 32], hi[D / 32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    lo[c] = __uint_as_float((uint32_t)__ldg(bnd + 32 * c + lane) << 16);
                    hi[c] = __uint_as_float((uint32_t)__ldg(bnd + D + 32 * c + lane) << 16);
                }
                double best = -INFINITY;
                bool nan = false;
                for (int g0 = 0; g0 < p.G; g0 += kHeads) {
                    float x[kHeads][D / 32];
                    double sum[kHeads];
#pragma unroll
                    for (int g = 0; g < kHeads; ++g) {
                        // (a head past the last: the last one again)
                        const uint16_t* q = p.q + (size_t)t * p.q_stride +
                                            (size_t)(hk * p.G + min(g0 + g, p.G - 1)) * D;
#pragma unroll
                        for (int c = 0; c < D / 32; ++c)
                            x[g][c] = __uint_as_float((uint32_t)__ldg(q + 32 * c + lane) << 16);
                    }
#pragma unroll
                    for (int g = 0; g < kHeads; ++g) {
                        sum[g] = 0;
#pragma unroll
                        for (int c = 0; c < D / 32; ++c)
                            sum[g] = fma((double)x[g][c], (double)(x[g][c] >= 0.f ? hi[c] : lo[c]),
                                         sum[g]);
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                        for (int g = 0; g < kHeads; ++g)
                            sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], off);
#pragma unroll
                    for (int g = 0; g < kHeads; ++g) {
                        nan = nan || sum[g] != sum[g];
                        best = fmax(best, sum[g]);
                    }
                }
                const int place = base + __shfl_sync(0xffffffffu, before, src);
                if (lane == 0 && dcheck(place < p.max_pages))
                    exact[place] = nan ? ~0ull : order_key(best);
            }
            base += all;
        }
        __syncwarp();
        if (kWarps > 1) __syncthreads();
        if (unsure <= 32) {
            // rank them against each other: lane i holds the i-th
            const unsigned long long mine = lane < unsure ? exact[lane] : 0;
            int ahead = 0;
            for (int i = 0; i < unsure; ++i) {
                const unsigned long long o = __shfl_sync(0xffffffffu, mine, i);
                ahead += o > mine || (o == mine && i < lane);
            }
            picked = __ballot_sync(0xffffffffu, lane < unsure && ahead < need);
        } else {
            // the need-th largest of them
            for (int bit = 63; bit >= 0; --bit) {
                const unsigned long long cand = kth | (1ull << bit);
                int n = 0;
                for (int i = tid; i < unsure; i += THREADS) n += exact[i] >= cand;
                if (total(n) >= need) kth = cand;
            }
            int n = 0;
            for (int i = tid; i < unsure; i += THREADS) n += exact[i] > kth;
            ties = need - total(n);                      // of the equal ones, from the lowest page up
        }
    }
    // ---- the chosen pages in ascending order
    int at = 0, base = 0;
#pragma unroll 1
    for (int r = 0; r * THREADS < row.pages; ++r) {
        bool take = (sure >> r) & 1;
        if (unsure > need) {
            const bool mine = (maybe >> r) & 1;
            int all;
            const int place = base + rank(mine, all);
            base += all;
            if (unsure <= 32) {
                take = take || (mine && ((picked >> place) & 1));
            } else {
                const unsigned long long k = mine ? exact[place] : 0;
                int equal;
                const int eq = rank(mine && k == kth, equal);
                take = take || (mine && (k > kth || (k == kth && eq < ties)));
                ties = max(0, ties - equal);
            }
        }
        int all;
        const int pos = at + rank(take, all);
        if (take && dcheck(pos < p.K)) out[pos] = r * THREADS + tid;
        at += all;
    }
    for (int i = at + tid; i < p.K; i += THREADS) out[i] = -1;
}

}  // namespace eattn
