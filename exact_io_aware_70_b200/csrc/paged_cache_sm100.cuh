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
            // min(. , T) of a sum of values <= T: scan in 64 bits would do the same
            const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, end, off);
                if (lane >= off) end = min(end + u, p.T);
            }
            __syncthreads();
            if (lane == 31) red[warp] = end;
            __syncthreads();
            int x = red[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x = min(x + u, p.T);
            }
            tot = __shfl_sync(0xffffffffu, x, 31);
            const int before = __shfl_sync(0xffffffffu, x, (warp + 31) & 31);
            if (warp > 0) end = min(end + before, p.T);
        }
        end = min(end + rows, p.T);
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
        rows = min(rows + tot, p.T);
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
        for (int t = t0; t < t1; ++t) {
            const long long s = slot_of(t);
            if (s < 0) continue;
            if (t + 1 < p.T) {
                const long long nx = __ldg(p.slot_map + t + 1);
                if (nx >= 0 && (nx >> p.page_shift) == (s >> p.page_shift)) continue;
            }
            // row t ends its page's run: reduce the page's slots 0 .. s % ps
            const int last = (int)(s & (ps - 1));
            uint4 lo, hi;
            bool any = false;
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
//   q . k <= sum_c (q_c >= 0 ? q_c hi_c : q_c lo_c),
// and a page's score is the largest such bound over the G query heads that
// share hk. The products of two bf16 are exact in fp64 and their sum all but
// is, so the choice does not depend on the order of the sum; pages with equal
// scores are taken from the lowest up. Scores go to the workspace as 64-bit
// keys of the same order; a second kernel finds each row's K-th largest key
// bit by bit and writes the pages above it in ascending order.
struct SelectParams {
    const uint16_t* q;          // bf16 [T, Hq, D], q_stride elements from row to row
    const uint16_t* bounds;     // bf16 [num_pages, Hkv, 2, D]
    const int* block_table;     // [B, max_pages]
    const int* cu_q;            // [B + 1]
    const int* seq_lens;        // [B]
    int* sel;                   // [T, Hkv, K]
    unsigned long long* keys;   // [T, Hkv, max_pages]
    long long q_stride;
    int B, T, Hq, Hkv, G, K, first, last;
    int page_shift, max_pages, num_pages;
};

struct SelectRow {
    int b, pages;    // sequence (-1: none), visible pages
};

// The sequence of row t and how many pages the row sees.
__device__ __forceinline__ SelectRow select_row(const SelectParams& p, int t) {
    SelectRow r;
    r.b = -1;
    r.pages = 0;
    if (t < __ldg(p.cu_q) || t >= __ldg(p.cu_q + p.B)) return r;
    int lo = 0, hi = p.B;    // the last b with cu[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu_q + mid) <= t) lo = mid;
        else hi = mid;
    }
    const int c0 = __ldg(p.cu_q + lo), c1 = __ldg(p.cu_q + lo + 1);
    if (t < c0 || t >= c1) return r;   // offsets that do not ascend
    const int cap = p.max_pages << p.page_shift;
    const int l = __ldg(p.seq_lens + lo), len = min(max(l, 0), cap);
    r.b = lo;
    const long long pos = (long long)len - c1 + t;
    r.pages = pos < 0 ? 0 : (int)(pos >> p.page_shift) + 1;
    return r;
}

__device__ __forceinline__ unsigned long long order_key(double x) {
    // ascending keys for ascending scores; NaN ranks above all scores, below the pages always kept
    if (x != x) return ~1ull;
    const unsigned long long u = (unsigned long long)__double_as_longlong(x);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

constexpr int kScoreThreads = 128;

// Block (x, row): pages [x * kScoreThreads, + kScoreThreads) of a (t, hk), one
// page per thread.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) attn_page_score_kernel(const SelectParams p) {
    extern __shared__ double s_q[];   // [G][D]
    const long long rowi = (long long)blockIdx.z * 65535 + blockIdx.y;
    if (rowi >= (long long)p.T * p.Hkv) return;
    const int t = (int)(rowi / p.Hkv), hk = (int)(rowi % p.Hkv);
    const SelectRow row = select_row(p, t);
    const int page0 = blockIdx.x * kScoreThreads;
    if (page0 >= row.pages) return;
    for (int i = threadIdx.x; i < p.G * D; i += kScoreThreads)
        s_q[i] = (double)__uint_as_float(
            (uint32_t)__ldg(p.q + (size_t)t * p.q_stride + (size_t)hk * p.G * D + i) << 16);
    __syncthreads();
    const int lp = page0 + threadIdx.x;
    if (lp >= row.pages) return;
    unsigned long long key = 0;       // a page that cannot be read is never chosen
    const int page = __ldg(p.block_table + (size_t)row.b * p.max_pages + lp);
    if (page < 0 || page >= p.num_pages) {
        atomicOr(&g_attn_status, kDevErrBadIndex);
    } else if (lp < p.first || lp >= row.pages - p.last) {
        key = ~0ull;
    } else {
        const uint4* lo4 = reinterpret_cast<const uint4*>(p.bounds + ((size_t)page * p.Hkv + hk) * 2 * D);
        const uint4* hi4 = lo4 + D / 8;
        double best = -INFINITY;
        bool nan = false;
        for (int g0 = 0; g0 < p.G; g0 += 4) {
            double acc[4] = {0, 0, 0, 0};
            for (int c = 0; c < D / 8; ++c) {
                const uint4 l = __ldg(lo4 + c), h = __ldg(hi4 + c);
                const uint32_t lw[4] = {l.x, l.y, l.z, l.w}, hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const double l0 = bf16_lo(lw[i]), l1 = bf16_hi(lw[i]);
                    const double h0 = bf16_lo(hw[i]), h1 = bf16_hi(hw[i]);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const double* q = s_q + min(g0 + g, p.G - 1) * D + 8 * c + 2 * i;
                        acc[g] = fma(q[0], q[0] >= 0 ? h0 : l0, acc[g]);
                        acc[g] = fma(q[1], q[1] >= 0 ? h1 : l1, acc[g]);
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                nan = nan || acc[g] != acc[g];
                best = fmax(best, acc[g]);
            }
        }
        key = nan ? ~1ull : order_key(best);
    }
    p.keys[rowi * p.max_pages + lp] = key;
}

// One group of THREADS threads per (t, hk), PER keys in each thread's registers.
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS == 32 ? 128 : THREADS)
    attn_page_topk_kernel(const SelectParams p) {
    constexpr int kGroups = THREADS == 32 ? 4 : 1;       // rows per block
    constexpr int kWarps = THREADS / 32;
    __shared__ int s_cnt[2][kWarps];
    const int tid = threadIdx.x % THREADS, lane = tid & 31, warp = tid >> 5;
    const long long rowi =
        ((long long)blockIdx.y * gridDim.x + blockIdx.x) * kGroups + threadIdx.x / THREADS;
    if (rowi >= (long long)p.T * p.Hkv) return;
    const int t = (int)(rowi / p.Hkv);
    const SelectRow row = select_row(p, t);
    if (row.b < 0) return;                               // rows of no sequence stay as they were
    int* out = p.sel + rowi * p.K;
    // thread i holds pages r * THREADS + i
    unsigned long long key[PER];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int lp = r * THREADS + tid;
        key[r] = lp < row.pages ? p.keys[rowi * p.max_pages + lp] : 0;
    }
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
    // the K-th largest key (0: fewer than K pages can be read)
    unsigned long long kth = 0;
    int above = -1;
    for (int bit = 63; bit >= 0; --bit) {
        const unsigned long long cand = kth | (1ull << bit);
        int n = 0;
#pragma unroll
        for (int r = 0; r < PER; ++r) n += key[r] >= cand;
        n = total(n);
        if (n >= p.K) kth = cand;
        if (n == p.K) {                                   // exactly these: no need to go on
            above = 0;
            break;
        }
    }
    if (kth == 0) kth = 1;                               // key 0 marks what cannot be chosen
    // how many of the keys equal to the K-th are taken, from the lowest page up
    int gt = 0;
    if (above != 0) {
#pragma unroll
        for (int r = 0; r < PER; ++r) gt += key[r] > kth;
        gt = total(gt);
    }
    int ties = above == 0 ? 0x7fffffff : p.K - gt;
    int at = 0;                                          // pages written so far
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        if (r * THREADS >= row.pages) break;             // the same for the whole group
        const bool eq = above != 0 && key[r] == kth;
        bool take = above == 0 ? key[r] >= kth : key[r] > kth;
        // position among this round's equal keys, then among its chosen ones
        const unsigned lt = (1u << lane) - 1;
        unsigned me = __ballot_sync(0xffffffffu, eq);
        int eq_before = 0, eq_all = __popc(me);
        if (kWarps > 1) {
            if (lane == 0) s_cnt[flip][warp] = eq_all;
            __syncthreads();
            eq_all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) eq_before += s_cnt[flip][w];
                eq_all += s_cnt[flip][w];
            }
            flip ^= 1;
        }
        if (eq && eq_before + __popc(me & lt) < ties) take = true;
        ties = max(0, ties - eq_all);
        const unsigned mt = __ballot_sync(0xffffffffu, take);
        int tk_before = 0, tk_all = __popc(mt);
        if (kWarps > 1) {
            if (lane == 0) s_cnt[flip][warp] = tk_all;
            __syncthreads();
            tk_all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) tk_before += s_cnt[flip][w];
                tk_all += s_cnt[flip][w];
            }
            flip ^= 1;
        }
        const int pos = at + tk_before + __popc(mt & lt);
        if (take && dcheck(pos < p.K)) out[pos] = r * THREADS + tid;
        at += tk_all;
    }
    for (int i = at + tid; i < p.K; i += THREADS) out[i] = -1;
}

}  // namespace eattn
