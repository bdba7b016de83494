// paged_fwd_sm100.cuh -- attention of new tokens over a paged K/V cache.
//
// For every sequence b with n new tokens, of which the last sits at position
// len - 1 of the cache, and for every query head h (K/V head hk = h / G):
//   O_i = sum_j p_ij v_j / l_i,  p_ij = exp(scale q_i . k_j - m_i),  l_i = sum_j p_ij,
//   LSE_i = m_i + ln l_i,
// over the keys j that row i sees: all of the sequence's, or those up to the
// row's own position (causal), or the tokens up to that position in a list of
// pages of the row's own (sparse). Statistics and accumulators are fp32; P is
// rounded to bf16 for the P V product (its rounding errors are independent
// and average out against the output's own rounding, which is as large).
//
// How the work is laid out:
//   * Rows of a tile are (token, head of the group): one Q tile of 128 rows is
//     floor(128 / G) tokens x the G query heads that share a K/V head, so that
//     grouped heads read each K/V tile once and a decoded token fills G rows.
//   * A unit is (sequence, K/V head, up to 256 rows), against all of its keys.
//     With more than 128 rows ("wide") two Q tiles share every K/V tile; with
//     fewer ("narrow": decode, drafts) the two softmax groups take alternate
//     key tiles of the same Q tile, and group 0 joins the two results, reading
//     both accumulators from tensor memory.
//   * All units are laid on one line, each as long as the keys it sees (plus a
//     constant for its start), and every CTA gets an equal stretch of it. Units
//     that a stretch's end cuts leave fp32 partial rows in the workspace (at
//     most two pieces per CTA); a second kernel joins them. The cut needs only
//     the lengths, which every CTA scans itself: the host never learns them and
//     no plan is kept.
//   * Warps 0-3 and 4-7 are the softmax groups of Q tile 0 and 1 (one thread per
//     row), warp 8 loads tiles by TMA, one thread of warp 9 issues the products
//     (S_t = Q_t K^T, then O_t += P_t V with P_t over S_t in tensor memory),
//     warp 10 cleans V tiles (below), warp 11 plans units ahead.
//   * Key tiles are 128 keys: 128 / page_size boxes of a tensor map over the
//     cache, one lane of the producer warp per box. A page-table entry out of
//     range, and everything past the last key, is read from a coordinate
//     outside the map, which fills zeros; a 128-bit mask per tile tells the
//     softmax which keys exist. What a page still holds behind the sequence's
//     last token may be anything (NaN too): its scores are replaced, and its V
//     rows are zeroed in shared memory by a warp of their own before P V.
//
// Few rows per sequence go to paged_rows_sm100.cuh instead. Measured (2 sequences of 2048 and 957
// new tokens behind 14.3K and 11.3K keys, 32 query heads on 8, d = 128): 700 us, 1000 TFLOP/s of
// the visible pairs, in a burst of a dozen launches, 784 us and 893 TFLOP/s under the power limit of
// longer runs. On the dense forward's own shape (32 heads of 128, 8192 tokens, causal) it takes 661
// us (678 sustained), that one 488 (541). What bounds it is the issuing thread, as in the dense
// forward (a product costs it about 0.48 us of queueing for 0.27 us of tensor time), and on short
// prompts (8 of up to 1024 tokens, 12 heads of 64: 50-54 us) the start of units and
// the instruction fetch of code that runs a few times only.
#pragma once

#include <cstdint>

#include "decode_sm100.cuh"
#include "fwd_sm100.cuh"
#include "paged_cache_sm100.cuh"
#include "paged_drain.cuh"
#include "ptx_sm100.cuh"
#include "tmem_wide.cuh"

namespace eattn {

constexpr int kPagedMaxCtas = 160;     // slots of the workspace; the grid is at most this
// In keys: what starting a unit costs; the least stretch worth a CTA of its own; and how near a
// cut may come to a unit's end before it is moved there (a piece costs its CTA a Q load and
// an epilogue, and the merge a pass). Measured: 128 to 640, 256 to 1024 within 2% of each other on
// decode, drafts, chunks and prompts; moved cuts (0 -> 128) 58.9 -> 55.6 us on prompts of up to
// 1024 tokens, 300 and more 4% slower on drafts.
constexpr int kPagedUnitCost = 128, kPagedMinStretch = 512, kPagedSnap = 128;
constexpr int kPagedListMax = 480;     // entries of a sparse row's list of key runs

// One CTA's partial rows of a unit that its stretch covers only in part.
// Slot 2c: a piece that continues a unit begun by an earlier CTA; slot 2c + 1: one that
// begins a unit and does not end it.
struct PagedPiece {
    int valid, last;     // last: the unit's keys end here
    int tok, ntok, hk;   // first row of q, tokens, K/V head
    int pad[3];
};

struct PagedParams {
    uint16_t* o;              // bf16 [T, Hq, D]
    float* lse;               // fp32 [T, Hq]
    const int* block_table;   // [B, max_pages]
    const int* cu_q;          // [B + 1]
    const int* seq_lens;      // [B]
    const int* sel;           // [T, Hkv, K] pages of each row; null: all
    float* part_o;            // fp32 [2 * kPagedMaxCtas][256][D]
    float* part_lse;          // fp32 [2 * kPagedMaxCtas][256]
    PagedPiece* pieces;       // [2 * kPagedMaxCtas]
    int B, T, Hq, Hkv, G, K;
    int tpt, unit_tok;        // tokens of a Q tile and of a unit
    int page_shift, max_pages, num_pages;
    int causal;
    float scale_log2;
};

// N = 0: 128-row Q tiles (this file); N = 16, 32: at most N rows per unit, kept as columns
// (paged_rows_sm100.cuh).
template <int D, int N = 0>
struct PagedTraits {
    static constexpr int kD = D, kN = N;
    static constexpr int kPanels = D / 64;
    static constexpr int kPanelBytes = 128 * 128;
    static constexpr int kTileBytes = kPanels * kPanelBytes;
    // K/V tile pairs in the ring: what shared memory leaves
    static constexpr int kPairs = D == 128 ? (N == 16 ? 3 : 2) : N == 16 ? 6 : N == 32 ? 5 : 4;
    static constexpr int kSlots = 2 * kPairs;
    static constexpr int kUnits = 4;                     // unit records in flight
    // the mask ring is longer than the K/V ring by the tiles that units planned ahead can have
    // without any work for one of the groups (kUnits, one tile each)
    static constexpr int kMasks = 2 * kPairs + 2 * kUnits;
    // N > 0: warp 12 plans and warp 13 loads V (one warp for both takes 1.1 us per key tile to
    // issue its copies: too long where K and V come from L2); else warp 11 plans
    static constexpr int kThreads = N ? 448 : 384;
    static constexpr int kLoaders = N ? 2 : 1;
    static constexpr int kQRows = N ? N : 128;
    static constexpr int kQPanelBytes = kQRows * 128;
    static constexpr int kQBytes = kPanels * kQPanelBytes;    // one Q slot (of two)
    static constexpr int kIssuers = N ? 2 : 1;           // threads that issue products
    static constexpr int kStageWarpBytes = 32 * 64;
    // N = 0: the epilogue's staging blocks; else P of both softmax groups (N x 128 bf16 each)
    static constexpr int kStageBytes = N ? 2 * N * 256 : 8 * kStageWarpBytes;
    static constexpr int kMlBytes = N ? 3 * N * 8 + 2 * 6 * N * 4 : 128 * 8;
    static constexpr int kBars = 2 * kSlots + kPairs + 4 + 4 + 8 + 2 * kUnits + 3 + 2 * kMasks;
    static constexpr int kOffKV = 2 * kQBytes;
    static constexpr int kOffStage = kOffKV + kSlots * kTileBytes;
    static constexpr int kOffList = kOffStage + kStageBytes;
    static constexpr int kOffMl = kOffList + kUnits * kPagedListMax * 8;
    static constexpr int kOffMask = kOffMl + kMlBytes;
    static constexpr int kOffUnits = kOffMask + kMasks * 16;
    static constexpr int kOffBars = kOffUnits + kUnits * 64;
    static constexpr int kOffMisc = kOffBars + kBars * 8;
    static constexpr int kSmemBytes = 1024 + kOffMisc + 64;
    static_assert(kSmemBytes <= 232448, "shared memory per CTA");
    // as in the dense forward: the launch gives every thread 168 registers (the
    // build checks it) and the warpgroups redistribute them
    static constexpr int kLaunchRegs = 168, kSoftmaxRegs = 192, kOtherRegs = 120;
    static_assert(2 * 128 * kSoftmaxRegs + 128 * kOtherRegs <= 384 * kLaunchRegs,
                  "register split exceeds the launch allocation");
    static constexpr uint32_t kColS0 = 0, kColS1 = N ? 64 : 128, kColO0 = N ? 128 : 256,
                              kColO1 = N ? 192 : 384;
};

template <class T>
struct PagedBars {
    uint32_t base;
    __device__ __forceinline__ uint32_t at(int i) const { return base + 8 * i; }
    __device__ __forceinline__ uint32_t kv_full(int i) const { return at(i); }
    __device__ __forceinline__ uint32_t kv_empty(int i) const { return at(T::kSlots + i); }
    __device__ __forceinline__ uint32_t v_raw(int i) const { return at(2 * T::kSlots + i); }
    static constexpr int kA = 2 * T::kSlots + T::kPairs;
    __device__ __forceinline__ uint32_t tail_full(int i) const { return at(kA + i); }
    __device__ __forceinline__ uint32_t tail_empty(int i) const { return at(kA + 2 + i); }
    __device__ __forceinline__ uint32_t q_full(int i) const { return at(kA + 4 + i); }
    __device__ __forceinline__ uint32_t q_empty(int i) const { return at(kA + 6 + i); }
    __device__ __forceinline__ uint32_t s_full(int t) const { return at(kA + 8 + t); }
    __device__ __forceinline__ uint32_t p_full(int t) const { return at(kA + 10 + t); }
    __device__ __forceinline__ uint32_t o_final(int t) const { return at(kA + 12 + t); }
    __device__ __forceinline__ uint32_t o_free(int t) const { return at(kA + 14 + t); }
    __device__ __forceinline__ uint32_t unit_full(int i) const { return at(kA + 16 + i); }
    __device__ __forceinline__ uint32_t unit_empty(int i) const {
        return at(kA + 16 + T::kUnits + i);
    }
    // the joining group's (m, l) of the other one's rows are there
    __device__ __forceinline__ uint32_t ml_full(int t) const { return at(kA + 16 + 2 * T::kUnits + t); }
    __device__ __forceinline__ uint32_t drain() const { return at(kA + 18 + 2 * T::kUnits); }
    // Key tile x of the CTA: its mask is written and its K slot has been given to it
    // (entry x % kMasks), and the same for its V slot. A parity tells only the
    // last two uses of a slot apart, so a thread that has not itself waited for the
    // slot's previous use waits for these first.
    __device__ __forceinline__ uint32_t mask_full(int i) const {
        return at(kA + 19 + 2 * T::kUnits + i);
    }
    __device__ __forceinline__ uint32_t v_given(int i) const {
        return at(kA + 19 + 2 * T::kUnits + T::kMasks + i);
    }
};

// A unit (or the piece of one) that the CTA works on, handed from the planner
// to the other roles through a ring in shared memory.
struct PagedUnit {
    int kind;        // 0: end of the CTA's work; 1: narrow; 2: wide
    int hk;
    int tok, ntok;   // first row of q, tokens
    int pos0;        // position of the first token in its sequence (may be negative)
    int len;         // keys of the sequence (dense), or a bound that masks nothing (sparse)
    int key0;        // first key of the piece, a multiple of 128
    int n0, n1;      // key tiles of Q tile / softmax group 0 and 1
    int slot;        // -1: whole unit; else the workspace slot of its partial rows
    int qs;          // Q slot of a narrow unit
    int seq, keys;   // sequence and its keys
    int entries;     // sparse: runs in the unit's list
    int pad[2];
};
static_assert(sizeof(PagedUnit) == 64, "unit record");

// Waits of the roles. The part that actually waits is one function for all of them: some
// thirty copies of it, inlined, kept the SM's instruction cache (shared by roles that run
// different code at the same time) from holding their loops. Only the softmax warps of
// the 128-row form, with a row of scores in registers, have it inline (SLIM = false).
__device__ __noinline__ bool paged_wait_slow(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag) {
    return mbar_wait_limit(bar, parity, abort_flag, &g_attn_status, kWaitLimitNs);
}
template <bool SLIM = true>
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity,
                                           volatile int* abort_flag) {
    if constexpr (!SLIM) return mbar_wait(bar, parity, abort_flag, &g_attn_status);
    if (mbar_test(bar, parity)) return true;
    return paged_wait_slow(bar, parity, abort_flag);
}
// by a whole warp; the outcome is the same in all lanes
template <bool SLIM = true>
__device__ __forceinline__ bool paged_warp_wait(uint32_t bar, uint32_t parity,
                                                volatile int* abort_flag) {
    const bool ok = paged_wait<SLIM>(bar, parity, abort_flag);
    return __all_sync(0xffffffffu, ok);
}

// ------------------------------------------------------------- schedule --
// a / b for a >= 0, b > 0; the 64-bit division is long, and rarely needed
__device__ __noinline__ long long div_long(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long div_fast(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return div_long(a, b);
}

// Lengths of a sequence's units on the line: unit q is base + min((q + 1) * U, n) *
// slope long; begin(q) is where unit q starts within one head.
struct PagedLine {
    long long base;
    int U, n, m, slope;
    __device__ __forceinline__ PagedLine(const PagedParams& p, const PagedSeq& s) {
        U = p.unit_tok;
        n = s.n;
        m = (s.n + U - 1) / U;
        slope = (!p.sel && p.causal) ? 1 : 0;
        base = kPagedUnitCost +
               (p.sel ? ((long long)p.K << p.page_shift) : p.causal ? max(s.len - s.n, 0) : s.len);
    }
    __device__ __forceinline__ long long unit(int q) const {
        return base + (slope ? min((long long)(q + 1) * U, (long long)n) : 0);
    }
    __device__ __forceinline__ long long begin(int q) const {
        long long x = base * q;
        if (slope) {
            x += (long long)U * q * (q + 1) / 2;
            if (q == m && q > 0) x -= (long long)m * U - n;
        }
        return x;
    }
};

// This CTA's stretch: the sequence it starts in, the offset in it and the length.
struct PagedStretch {
    long long offset, length;
    int b;
    PagedSeq s;  // of sequence b
    int block;   // sparse: tokens of a block of units (see PagedWalk)
};

// Run by the whole CTA. `red`: THREADS / 32 + 4 words of 64 bits.
template <int THREADS>
__device__ __forceinline__ PagedStretch paged_schedule(const PagedParams& p, long long* red) {
    constexpr int kWarps = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto cost = [&](int b, bool report) -> long long {
        const PagedSeq s = paged_seq(p, b);
        if (report && s.bad) atomicOr(&g_attn_status, kDevErrBadIndex);
        const PagedLine line(p, s);
        return p.Hkv * line.begin(line.m);
    };
    long long mine = 0, first = 0;
    for (int b = tid; b < p.B; b += THREADS) {
        const long long c = cost(b, blockIdx.x == 0);
        if (b == tid) first = c;
        mine += c;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
    if (lane == 0) red[warp] = mine;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += red[w];
    __syncthreads();
    long long chunk = div_fast(total + gridDim.x - 1, gridDim.x);
    if (chunk < kPagedMinStretch) chunk = kPagedMinStretch;
    PagedStretch st;
    st.block = 1;
    if (p.sel) {   // about as many tokens as one stretch holds for all K/V heads
        const long long all_heads =
            (kPagedUnitCost + ((long long)p.K << p.page_shift)) * p.Hkv;
        st.block = (int)min(max(div_fast(chunk + all_heads / 2, all_heads), 1ll), 1ll << 20);
    }
    const long long start = chunk * blockIdx.x;
    st.length = min(chunk, total - start);
    st.offset = 0;
    st.b = 0;
    st.s.tok = st.s.n = st.s.len = 0;
    st.s.bad = false;
    if (st.length <= 0) {   // the same for the whole CTA
        st.length = 0;
        return st;
    }
    long long before = 0;
    for (int b0 = 0; b0 < p.B && before <= start; b0 += THREADS) {
        const int b = b0 + tid;
        const long long v = b < p.B ? (b0 == 0 ? first : cost(b, false)) : 0;
        long long incl = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += u;
        }
        if (lane == 31) red[warp] = incl;
        __syncthreads();
        long long all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) incl += red[w];
            all += red[w];
        }
        incl += before;
        if (start >= incl - v && start < incl) {
            const PagedSeq s = paged_seq(p, b);
            red[kWarps] = b;
            red[kWarps + 1] = start - (incl - v);
            red[kWarps + 2] = s.tok;
            red[kWarps + 3] = ((long long)s.n << 32) | s.len;
        }
        before += all;
        __syncthreads();
    }
    st.b = (int)red[kWarps];
    st.offset = red[kWarps + 1];
    st.s.tok = (int)red[kWarps + 2];
    st.s.n = (int)(red[kWarps + 3] >> 32);
    st.s.len = (int)red[kWarps + 3];
    st.s.bad = false;
    return st;
}

// -------------------------------------------------------------- producer --
__device__ __forceinline__ uint32_t low_bits(int n) {   // n clamped to 0 .. 32
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

struct PagedShared {
    uint8_t* smem;
    volatile int* abort_flag;
    int* tail_info;        // [2]: the pair
    uint32_t* tail_mask;   // [2][4]: its keys
};

// 3-D tile load with an L2 policy, one box per calling lane.
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int x, int y, int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}

// The units of a CTA's stretch in order. Dense: K/V head by head, and a head's
// rows in turn. Sparse: blocks of `block` tokens, head by head within a block:
// as a stretch is about one block long, the CTAs sweep the heads together and L2
// holds the pages of one head at a time.
template <bool SPARSE>
struct PagedWalk {
    PagedSeq s;
    PagedLine line;
    int sb, hk, q, q0, block;
    long long rem, left;     // where in unit q the stretch stands, and what is left of it

    __device__ __forceinline__ PagedWalk(const PagedParams& p, const PagedStretch& st)
        : s(st.s), line(p, s), sb(st.b), hk(0), q(0), q0(0), block(st.block),
          rem(st.offset), left(st.length) {
        if (left <= 0) return;
        if constexpr (SPARSE) {
            const long long i = div_fast(rem, line.base);      // units before this one
            rem -= i * line.base;
            q0 = (int)div_fast(i, (long long)block * p.Hkv) * block;
            const int in = (int)(i - (long long)q0 * p.Hkv), nq = min(block, line.m - q0);
            hk = in / nq;
            q = q0 + in - hk * nq;
        } else {
            const long long head = line.begin(line.m);
            hk = (int)div_fast(rem, head);
            rem -= hk * head;
            // the last unit that begins at or before rem
            int hi = line.m - 1;
            while (q < hi) {
                const int mid = (q + hi + 1) >> 1;
                if (line.begin(mid) <= rem) q = mid;
                else hi = mid - 1;
            }
            rem -= line.begin(q);
        }
        // (the CTA before moves its end by the same rule)
        const long long ulen = line.unit(q);
        if (rem > 0 && rem < kPagedSnap) {
            left += rem;
            rem = 0;
        } else if (rem > 0 && ulen - rem < kPagedSnap) {
            advance(p, ulen - rem);
        }
    }
    // how far into its unit the stretch goes (0: it ends before)
    __device__ __forceinline__ long long end(const PagedParams& p, long long ulen) const {
        const long long e = rem + left;
        return e >= ulen ? ulen : e < kPagedSnap ? 0 : ulen - e < kPagedSnap ? ulen : e;
    }
    // past the part of unit q that [rem, rem + taken) is
    __device__ __forceinline__ void advance(const PagedParams& p, long long taken) {
        left -= taken;
        rem = 0;
        if (left <= 0) return;
        if (++q < (SPARSE ? min(q0 + block, line.m) : line.m)) return;
        if (++hk < p.Hkv) {
            q = q0;
            return;
        }
        hk = 0;
        q0 = q;
        if (q < line.m) return;
        q = q0 = 0;
        do {
            if (++sb >= p.B) {
                left = 0;
                return;
            }
            s = paged_seq(p, sb);
        } while (s.n == 0);
        line = PagedLine(p, s);
    }
};

// The planner warp, all lanes together: the units one after another, up to kUnits
// ahead (planning a unit takes a few microseconds of dependent steps), and for sparse
// rows the lists of their pages.
template <class T, bool SPARSE>
__device__ void paged_planner(const PagedParams& p, const PagedStretch& st, const PagedBars<T>& b,
                              const PagedShared& sh, int lane) {
    PagedUnit* ring = reinterpret_cast<PagedUnit*>(sh.smem + T::kOffUnits);
    const int ps = 1 << p.page_shift;
    const int rshift = min(p.page_shift, 7);      // rows of a box: min(page_size, 128)
    const int R = 1 << rshift;
    int qs = 0;

    if (lane < 2) p.pieces[2 * blockIdx.x + lane].valid = 0;
    __syncwarp();

    PagedWalk<SPARSE> w(p, st);
    for (uint32_t units = 0;; ++units) {
        const int ri = units % T::kUnits;
        PagedUnit u;
        u.kind = 0;
        const bool more = w.left > 0 && w.end(p, w.line.unit(w.q)) > 0;
        // sparse: the row's first 32 entries and their pages, read while the ring is full
        int ahead_e = -1, ahead_page = -1;
        auto visible = [&](int e) {   // (and so in the table)
            return e >= 0 && ((long long)e << p.page_shift) <= w.s.len - w.s.n + w.q;
        };
        auto page_of = [&](int e) { return __ldg(p.block_table + (size_t)w.sb * p.max_pages + e); };
        if (SPARSE && more && lane < p.K) {
            ahead_e = __ldg(p.sel + ((size_t)(w.s.tok + w.q) * p.Hkv + w.hk) * p.K + lane);
            if (visible(ahead_e)) ahead_page = page_of(ahead_e);
        }
        if (units >= (uint32_t)T::kUnits &&
            !paged_warp_wait(b.unit_empty(ri), (units / T::kUnits - 1) & 1, sh.abort_flag))
            return;
        if (more) {
            const long long ulen = w.line.unit(w.q);
            const long long p0 = w.rem, p1 = w.end(p, ulen);
            u.seq = w.sb;
            u.keys = u.len = w.s.len;
            u.hk = w.hk;
            u.tok = w.s.tok + w.q * w.line.U;
            u.ntok = min(w.line.U, w.s.n - w.q * w.line.U);
            u.pos0 = w.s.len - w.s.n + w.q * w.line.U;
            u.kind = u.ntok > p.tpt ? 2 : 1;
            u.qs = 0;
            u.entries = 0;
            int tiles[2];        // key tiles of the whole unit, for each Q tile
            if constexpr (SPARSE) {
                // the row's visible pages as runs of up to R keys: (page, first row, keys)
                int2* list = reinterpret_cast<int2*>(sh.smem + T::kOffList) + ri * kPagedListMax;
                const int* row = p.sel + ((size_t)u.tok * p.Hkv + u.hk) * p.K;
                int next_e = ahead_e;
                for (int k0 = 0; k0 < p.K; k0 += 32) {
                    const int e = next_e;
                    next_e = k0 + 32 + lane < p.K ? __ldg(row + k0 + 32 + lane) : -1;
                    if (e != -1 && (e < 0 || ((long long)e << p.page_shift) >= u.len))
                        atomicOr(&g_attn_status, kDevErrBadIndex);
                    int page = -1, nv = 0;
                    if (visible(e)) {
                        page = k0 == 0 ? ahead_page : page_of(e);
                        if (page < 0 || page >= p.num_pages)
                            atomicOr(&g_attn_status, kDevErrBadIndex);
                        else
                            nv = min(ps, u.pos0 + 1 - (e << p.page_shift));
                    }
                    const int runs = (nv + R - 1) >> rshift;
                    int at = u.entries;
                    if (rshift == p.page_shift) {     // a page is one run
                        const unsigned full = __ballot_sync(0xffffffffu, runs > 0);
                        at += __popc(full & ((1u << lane) - 1));
                        u.entries += __popc(full);
                    } else {
                        int incl = runs;
#pragma unroll
                        for (int off = 1; off < 32; off <<= 1) {
                            const int v = __shfl_up_sync(0xffffffffu, incl, off);
                            if (lane >= off) incl += v;
                        }
                        at += incl - runs;
                        u.entries += __shfl_sync(0xffffffffu, incl, 31);
                    }
                    for (int r = 0; r < runs; ++r)
                        if (dcheck(at + r < kPagedListMax))
                            list[at + r] =
                                make_int2(page, (r << rshift << 8) | min(R, nv - (r << rshift)));
                }
                __syncwarp();
                tiles[0] = (u.entries * R + 127) >> 7;
                tiles[1] = 0;
                u.len = 0x7fffffff;   // the masks say it all
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    int vis = 0;
                    if (u.ntok > t * p.tpt)
                        vis = p.causal ? u.pos0 + min((t + 1) * p.tpt, u.ntok) : u.len;
                    tiles[t] = (max(vis, 0) + 127) >> 7;
                }
            }
            const int all = max(tiles[0], tiles[1]);
            auto tile_at = [&](long long pos) -> int {
                const long long k = (pos - kPagedUnitCost) >> 7;
                return k < 0 ? 0 : k > all ? all : (int)k;
            };
            const int k0 = p0 == 0 ? 0 : tile_at(p0);
            const int N = (p1 == ulen ? all : tile_at(p1)) - k0;
            u.key0 = k0 << 7;
            if (u.kind == 2) {
                u.n0 = min(max(tiles[0] - k0, 0), N);
                u.n1 = min(max(tiles[1] - k0, 0), N);
            } else {
                u.n0 = (N + 1) >> 1;
                u.n1 = N >> 1;
                u.qs = qs;
                if (N > 0) qs ^= 1;
            }
            u.slot = -1;
            if (p0 > 0 || p1 < ulen) {
                u.slot = 2 * blockIdx.x + (p0 > 0 ? 0 : 1);
                if (lane == 0 && dcheck(u.slot < 2 * kPagedMaxCtas)) {
                    PagedPiece* pc = p.pieces + u.slot;
                    pc->last = p1 == ulen ? 1 : 0;
                    pc->tok = u.tok;
                    pc->ntok = u.ntok;
                    pc->hk = u.hk;
                    pc->valid = 1;
                }
            }
            w.advance(p, p1 - p0);
        }
        if (lane == 0) {
            ring[ri] = u;
            mbar_arrive(b.unit_full(ri));
        }
        if (!more) return;
    }
}

// A producer warp, all lanes together: Q and the K/V tiles of the planned units. K and V:
// which of the two it loads (Q and the masks go with K).
template <class T, bool SPARSE, bool K, bool V>
__device__ void paged_producer(const PagedParams& p, const CUtensorMap* tq, const CUtensorMap* tk,
                               const CUtensorMap* tv, const PagedBars<T>& b, const PagedShared& sh,
                               int lane) {
    const uint32_t sQ = smem_addr(sh.smem), sKV = sQ + T::kOffKV;
    const PagedUnit* ring = reinterpret_cast<const PagedUnit*>(sh.smem + T::kOffUnits);
    volatile int* abort_flag = sh.abort_flag;
    const int ps = 1 << p.page_shift;
    const int rshift = min(p.page_shift, 7);      // rows of a box: min(page_size, 128)
    const int R = 1 << rshift;
    const int boxes = 128 >> rshift;              // boxes of a tile and panel
    const int bx = lane & (boxes - 1), panel = lane >> (7 - rshift);
    const bool issues = panel < T::kPanels;
    const uint32_t box_off = panel * T::kPanelBytes + bx * R * 128;
    const int z_out = p.num_pages * p.Hkv;        // outside the map: reads zeros
    // decode reads each K/V byte once (narrow), a chunk's query blocks re-read it (wide)
    const uint64_t pol_first = l2_policy_evict_first(), pol_last = l2_policy_evict_last();

    uint32_t it = 0;                  // key tiles loaded by this CTA
    uint32_t q_used[2] = {0, 0};
    uint32_t tails = 0, raw_par = 0, raw_last = 0;   // (bits by slot pair, see paged_drain)
    bool v_skipped = false;           // gave up before the last counted tile's V copy

    for (uint32_t units = 0;; ++units) {
        const int ri = units % T::kUnits;
        if (!paged_warp_wait(b.unit_full(ri), (units / T::kUnits) & 1, abort_flag)) goto fail;
        {
            const volatile PagedUnit& u = ring[ri];
            const int kind = u.kind;
            if (kind == 0) break;
            const bool wide = kind == 2;
            const int hk = u.hk, tok = u.tok, uqs = u.qs, keys_all = u.keys, first = u.key0 >> 7;
            const int entries = SPARSE ? u.entries : 0;
            const int N = wide ? max(u.n0, u.n1) : u.n0 + u.n1;
            const int* table = p.block_table + (size_t)u.seq * p.max_pages;
            const int2* list = reinterpret_cast<const int2*>(sh.smem + T::kOffList) + ri * kPagedListMax;
            if (K && N > 0) {
                // Q: token-major rows of the group's heads
                for (int t = 0; t < (wide ? 2 : 1); ++t) {
                    const int slot = wide ? t : uqs;
                    if (q_used[slot] > 0 &&
                        !paged_warp_wait(b.q_empty(slot), (q_used[slot] - 1) & 1, abort_flag))
                        goto fail;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(b.q_full(slot),
                                              (uint32_t)(T::kPanels * p.tpt * p.G * 128));
                        for (int pn = 0; pn < T::kPanels; ++pn)
                            tma_load_3d(sQ + slot * T::kQBytes + pn * T::kQPanelBytes, tq,
                                        b.q_full(slot), pn * 64, hk * p.G, tok + t * p.tpt);
                    }
                    ++q_used[slot];
                }
            }
            const uint64_t pol = wide ? pol_last : pol_first;
            // the page, first row and key count of this lane's box of key tile k
            auto look = [&](int k, int& page, int& y, int& keys) {
                if constexpr (SPARSE) {
                    const int e = k * boxes + bx;
                    const int2 x = e < entries ? list[e] : make_int2(-1, 0);
                    page = x.x;
                    y = x.y >> 8;
                    keys = x.y & 255;
                } else {
                    const long long key = (long long)k * 128 + bx * R;
                    const int lp = (int)(key >> p.page_shift);
                    keys = (int)min(max((long long)keys_all - key, 0ll), (long long)R);
                    y = (int)(key & (ps - 1));
                    page = keys > 0 && dcheck(lp < p.max_pages) ? __ldg(table + lp) : -1;
                }
            };
            int page = -1, y = 0, keys = 0;
            if (N > 0) look(first, page, y, keys);
            for (int j = 0; j < N; ++j) {
                int npage = -1, ny = 0, nkeys = 0;
                if (j + 1 < N) look(first + j + 1, npage, ny, nkeys);   // ahead of the waits
                if (keys > 0 && (page < 0 || page >= p.num_pages)) {
                    if (panel == 0) atomicOr(&g_attn_status, kDevErrBadIndex);
                    keys = 0;
                }
                const int z = keys > 0 ? page * p.Hkv + hk : z_out;
                // which of the tile's keys exist, 32 to a word (lanes 0 .. 3)
                const int wi = lane & 3;
                uint32_t word =
                    low_bits(min(__shfl_sync(0xffffffffu, keys, (32 * wi) >> rshift) -
                                     ((32 * wi) & (R - 1)), R));
                {
                    const int hi = __shfl_sync(0xffffffffu, keys, ((32 * wi) >> rshift) + 1);
                    if (R == 16) word |= low_bits(min(hi, 16)) << 16;
                }
                const bool whole = __all_sync(0xffffffffu, word == 0xffffffffu);
                const uint32_t pair = it % T::kPairs, round = it / T::kPairs;
                const uint32_t sk = 2 * pair, sv = 2 * pair + 1;
                if constexpr (K) {
                    if (round > 0 && !paged_warp_wait(b.kv_empty(sk), (round - 1) & 1, abort_flag))
                        goto fail;
                    if (lane < 4)
                        reinterpret_cast<volatile uint32_t*>(
                            sh.smem + T::kOffMask)[(it % T::kMasks) * 4 + lane] = word;
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(b.kv_full(sk), T::kTileBytes);
                        mbar_arrive(b.mask_full(it % T::kMasks));
                    }
                    __syncwarp();
                    if (issues)
                        tma_load_3d_hint(sKV + sk * T::kTileBytes + box_off, tk, b.kv_full(sk),
                                         panel * 64, y, z, pol);
                }
                if constexpr (V) {
                    if (round > 0 && !paged_warp_wait(b.kv_empty(sv), (round - 1) & 1, abort_flag)) {
                        ++it;
                        v_skipped = true;
                        goto fail;
                    }
                    uint32_t vbar = b.kv_full(sv);
                    if (!whole) {   // rows without a key must be zeroed before P V
                        const uint32_t i = tails & 1;
                        if (tails >= 2 &&
                            !paged_warp_wait(b.tail_empty(i), ((tails >> 1) - 1) & 1, abort_flag)) {
                            ++it;
                            v_skipped = true;
                            goto fail;
                        }
                        vbar = b.v_raw(pair);
                        if (lane < 4) reinterpret_cast<volatile uint32_t*>(sh.tail_mask)[4 * i + lane] = word;
                        __syncwarp();
                        if (lane == 0) {
                            reinterpret_cast<volatile int*>(sh.tail_info)[i] = (int)pair;
                            mbar_arrive_expect_tx(vbar, T::kTileBytes);
                            mbar_arrive(b.tail_full(i));
                        }
                        ++tails;
                        raw_par ^= 1u << pair;
                        raw_last |= 1u << pair;
                    } else {
                        if (lane == 0) mbar_arrive_expect_tx(vbar, T::kTileBytes);
                        raw_last &= ~(1u << pair);
                    }
                    if (T::kIssuers > 1 && lane == 0) mbar_arrive(b.v_given(it % T::kMasks));
                    __syncwarp();
                    if (issues)
                        tma_load_3d_hint(sKV + sv * T::kTileBytes + box_off, tv, vbar, panel * 64, y,
                                         z, pol);
                }
                ++it;
                page = npage;
                y = ny;
                keys = nkeys;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(b.unit_empty(ri));   // the list is read
        }
    }
    if (V) {
        const uint32_t i = tails & 1;
        if (tails >= 2 && !paged_warp_wait(b.tail_empty(i), ((tails >> 1) - 1) & 1, abort_flag)) goto fail;
        if (lane == 0) {
            reinterpret_cast<volatile int*>(sh.tail_info)[i] = -1;
            mbar_arrive(b.tail_full(i));
        }
    }
    return;
fail:
    // Give up: wait (bounded, ignoring the abort flag) for the copies still in
    // flight so that none lands in shared memory after the CTA has exited.
    if (lane == 0) {
        volatile int no_abort = 0;
        paged_drain<K, V>(
            it, v_skipped, T::kPairs, raw_par, raw_last,
            [&](uint32_t pair, uint32_t par) { paged_wait(b.kv_full(2 * pair), par, &no_abort); },
            [&](uint32_t pair, bool raw, uint32_t par) {
                paged_wait(raw ? b.v_raw(pair) : b.kv_full(2 * pair + 1), par, &no_abort);
            });
        for (int i = 0; i < 2; ++i)
            if (K && q_used[i] > 0)
                paged_wait(b.q_full(i), (q_used[i] - 1) & 1, &no_abort);
    }
    __syncwarp();
}

// Zeroes the V rows of keys that do not exist (a whole warp).
template <class T>
__device__ void paged_tail(const PagedBars<T>& b, const PagedShared& sh, int lane) {
    const uint32_t sKV = smem_addr(sh.smem) + T::kOffKV;
    uint32_t par = 0;
    for (uint32_t i = 0;; ++i) {
        if (!paged_warp_wait(b.tail_full(i & 1), (i >> 1) & 1, sh.abort_flag)) return;
        const int info = reinterpret_cast<volatile int*>(sh.tail_info)[i & 1];
        if (info < 0) return;
        const uint32_t pair = info;
        if (!paged_warp_wait(b.v_raw(pair), (par >> pair) & 1, sh.abort_flag)) return;
        par ^= 1u << pair;
        const volatile uint32_t* mask = reinterpret_cast<volatile uint32_t*>(sh.tail_mask) + 4 * (i & 1);
        const uint32_t tile = sKV + (2 * pair + 1) * T::kTileBytes;
        for (int r = lane; r < 128; r += 32) {
            if ((mask[r >> 5] >> (r & 31)) & 1) continue;
            for (int pn = 0; pn < T::kPanels; ++pn)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    st_shared_v4(tile + pn * T::kPanelBytes + r * 128 + c * 16, 0, 0, 0, 0);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(b.kv_full(2 * pair + 1));
            mbar_arrive(b.tail_empty(i & 1));
        }
    }
}

// ------------------------------------------------------------ MMA issuer --
// One thread. Per step i and Q tile (or softmax group) t: P_t(i) V, then
// S_t(i + 1), which overwrites P_t(i). A wide unit's step i uses key tile i for
// both t, a narrow one's key tile 2 i + t.
template <int D>
__device__ void paged_mma(uint32_t tbase, const PagedBars<PagedTraits<D>>& b,
                          const PagedShared& sh) {
    using T = PagedTraits<D>;
    using F = FwdTraits<D, false>;
    static_assert(F::kTileBytes == T::kTileBytes && F::kPanelBytes == T::kPanelBytes, "tiles");
    constexpr uint64_t kTileStep = T::kTileBytes >> 4;
    const uint32_t sQ = smem_addr(sh.smem), sKV = sQ + T::kOffKV;
    const uint64_t dq0 = fwd_sdesc<F>(sQ, 16);
    const uint64_t dk0 = fwd_sdesc<F>(sKV, 16);
    const uint64_t dv0 = fwd_sdesc<F>(sKV, T::kPanelBytes);
    volatile int* abort_flag = sh.abort_flag;
    const PagedUnit* ring = reinterpret_cast<const PagedUnit*>(sh.smem + T::kOffUnits);
    uint32_t it = 0, units = 0;
    uint32_t q_used[2] = {0, 0}, o_used[2] = {0, 0}, p_par[2] = {0, 0};
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return paged_wait(bar, parity, abort_flag);
    };
    for (;; ++units) {
        const int ri = units % T::kUnits;
        if (!wait(b.unit_full(ri), (units / T::kUnits) & 1)) goto done;
        const volatile PagedUnit& u = ring[ri];
        const int kind = u.kind;
        const int n[2] = {u.n0, u.n1};
        const int uqs = u.qs;
        mbar_arrive(b.unit_empty(ri));
        if (kind == 0) break;
        const bool wide = kind == 2;
        const int N = wide ? max(n[0], n[1]) : n[0] + n[1];
        if (N == 0) continue;
        const int steps = max(n[0], n[1]);
        for (int t = 0; t < (wide ? 2 : 1); ++t) {
            const int slot = wide ? t : uqs;
            const uint32_t used = slot ? q_used[1] : q_used[0];
            if (!wait(b.q_full(slot), used & 1)) goto done;
            if (slot) ++q_used[1];
            else ++q_used[0];
            if (wide && (t ? n[1] : n[0]) == 0) mma_commit_w(b.q_empty(t), 1);
        }
        // key tile k of the unit sits in pair (it + k) % kPairs. One copy of each product's
        // code serves both t (rolled loops: the roles share the instruction cache).
#pragma unroll 1
        for (int i = -1; i < steps; ++i) {
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                const int nt = t ? n[1] : n[0];
                const uint32_t tS = tbase + (t ? T::kColS1 : T::kColS0);
                // tile 1 of a wide unit finds what tile 0 has waited for
                const bool second = wide && t == 1;
                if (i >= 0 && i < nt) {
                    const uint32_t x = it + (wide ? i : 2 * i + t), sv = 2 * (x % T::kPairs) + 1;
                    if (!(second && i < n[0]) && !wait(b.kv_full(sv), (x / T::kPairs) & 1)) goto done;
                    const uint32_t par = t ? p_par[1] : p_par[0], used = t ? o_used[1] : o_used[0];
                    if (!wait(b.p_full(t), par)) goto done;
                    if (t) p_par[1] ^= 1;
                    else p_par[0] ^= 1;
                    if (i == 0 && used > 0 && !wait(b.o_free(t), (used - 1) & 1)) goto done;
                    tc_fence_after_sync();
                    const uint32_t tO = tbase + (t ? T::kColO1 : T::kColO0);
                    fwd_issue_pv<D, false>(tO, tS, dv0 + sv * kTileStep, i > 0, 0, 1);
                    fwd_issue_pv<D, false>(tO, tS, dv0 + sv * kTileStep, true, 1, 1);
                    if (i == nt - 1) mma_commit_w(b.o_final(t), 1);
                    if (!wide || t == 1 || i >= n[1]) mma_commit_w(b.kv_empty(sv), 1);
                }
                const int i1 = i + 1;
                if (i1 < nt) {
                    const int k = wide ? i1 : 2 * i1 + t;
                    const uint32_t x = it + k, sk = 2 * (x % T::kPairs);
                    if (!(second && i1 < n[0]) && !wait(b.kv_full(sk), (x / T::kPairs) & 1)) goto done;
                    tc_fence_after_sync();
                    fwd_issue_s<D, false>(tS, dq0 + (wide ? t : uqs) * kTileStep, dk0 + sk * kTileStep, 1);
                    mma_commit_w(b.s_full(t), 1);
                    if (!wide || t == 1 || i1 >= n[1]) mma_commit_w(b.kv_empty(sk), 1);
                    // a Q tile's last product lets the producer refill it
                    if (wide ? i1 == nt - 1 : k == N - 1) mma_commit_w(b.q_empty(wide ? t : uqs), 1);
                }
            }
        }
        if (n[0] > 0) ++o_used[0];
        if (n[1] > 0) ++o_used[1];
        it += N;
    }
done: {
    // Every MMA issued so far must finish before tensor memory is released.
    volatile int no_abort = 0;
    mma_commit_w(b.drain(), 1);
    paged_wait(b.drain(), 0, &no_abort);
}
}

// --------------------------------------------------------------- softmax --
// 32 columns of this warp's 32 rows, staged as in fwd_store_chunk so that a
// store instruction writes whole 64-byte pieces of rows; dst[i]: where row
// 8 i + lane / 4 of the warp goes (null: a row without a token).
template <int D>
__device__ __forceinline__ void paged_store_chunk(uint32_t stage, const uint32_t (&w)[16], int lane,
                                                  uint16_t* const (&dst)[4], int c) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k)
        st_shared_v4(stage + stage_slot(lane, k), w[4 * k], w[4 * k + 1], w[4 * k + 2],
                     w[4 * k + 3]);
    __syncwarp();
    uint4 val[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        val[i] = ld_shared_v4(stage + stage_slot(i * 8 + (lane >> 2), lane & 3));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (dst[i]) *reinterpret_cast<uint4*>(dst[i] + c + 8 * (lane & 3)) = val[i];
}

template <int D>
__device__ void paged_softmax(const PagedParams& p, uint32_t tbase,
                              const PagedBars<PagedTraits<D>>& b, const PagedShared& sh, int warp,
                              int lane) {
    using T = PagedTraits<D>;
    const int t = warp >> 2;                 // Q tile, or softmax group of a narrow unit
    const int quarter = warp & 3;            // tensor-memory lanes this warp may access
    const int r = quarter * 32 + lane;       // row of the tile
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const uint32_t tS = tbase + lane_off + (t ? T::kColS1 : T::kColS0);
    const uint32_t tO = tbase + lane_off + (t ? T::kColO1 : T::kColO0);
    const uint32_t tO1 = tbase + lane_off + T::kColO1;
    volatile int* abort_flag = sh.abort_flag;
    const PagedUnit* ring = reinterpret_cast<const PagedUnit*>(sh.smem + T::kOffUnits);
    volatile float2* ml = reinterpret_cast<volatile float2*>(sh.smem + T::kOffMl);
    const uint32_t masks = smem_addr(sh.smem) + T::kOffMask;
    const uint32_t stage = smem_addr(sh.smem) + T::kOffStage + warp * T::kStageWarpBytes;
    const float c2 = p.scale_log2;
    uint32_t it = 0, s_cnt = 0, ml_cnt = 0;
    uint32_t o_par = 0;                      // uses of O by group 0 (bit 0) and 1 (bit 1), mod 2

    // A unit's record is kept (not released) until its end, and read where it is needed: with a
    // row of scores in registers there is no room for its fields.
    for (uint32_t units = 0;; ++units) {
        const int ri = units % T::kUnits;
        if (!paged_warp_wait<false>(b.unit_full(ri), (units / T::kUnits) & 1, abort_flag)) return;
        const volatile PagedUnit& uu = ring[ri];
        if (uu.kind == 0) break;
        const bool wide = uu.kind == 2;
        const int n = t ? uu.n1 : uu.n0;
        // rows [0, rows_of()) of the tile have a token; token_of(): the tile's first one
        auto token_of = [&]() { return wide ? t * p.tpt : 0; };
        auto rows_of = [&]() { return min(max(uu.ntok - token_of(), 0), p.tpt) * p.G; };
        const bool active = quarter * 32 < rows_of();       // any of this warp's rows
        // keys [0, lim) of the piece's are visible to this row
        int lim = uu.len;
        if (p.causal && lim != 0x7fffffff) lim = min(lim, uu.pos0 + token_of() + r / p.G + 1);
        lim -= uu.key0;
        float m_ref = -INFINITY, l = 0.f;

        for (int i = 0; i < n; ++i) {
            const int k = wide ? i : 2 * i + t;
            if (!paged_warp_wait<false>(b.s_full(t), s_cnt & 1, abort_flag)) return;
            ++s_cnt;
            if (!active) {   // no row to work on: P stays what it is (rows are independent)
                __syncwarp();
                if (lane == 0) mbar_arrive(b.p_full(t));
                continue;
            }
            // the mask was written before K was loaded, and its entry is not written again
            // before this tile's P V has freed V's slot
            const uint32_t x = it + k;
            if (!paged_warp_wait<false>(b.mask_full(x % T::kMasks), (x / T::kMasks) & 1, abort_flag)) return;
            const uint32_t mask_at = masks + 16 * (x % T::kMasks);
            bool masked;
            {
                const uint4 mask = ld_shared_v4(mask_at);
                masked = lim - k * 128 < 128 || (mask.x & mask.y & mask.z & mask.w) != 0xffffffffu;
            }
            tc_fence_after_sync();
            uint32_t sr[128];
            tmem_ld128(tS, sr);
            tmem_wait_ld128(sr);
            if (masked) {
                // keys that exist and lie before the row's limit
                const int cl = lim - k * 128;
                const uint4 mask = ld_shared_v4(mask_at);
                const uint32_t seen[4] = {mask.x & low_bits(cl), mask.y & low_bits(cl - 32),
                                          mask.z & low_bits(cl - 64), mask.w & low_bits(cl - 96)};
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (!((seen[c >> 5] >> (c & 31)) & 1)) sr[c] = __float_as_uint(-INFINITY);
            }
            float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
            for (int c = 0; c < 128; c += 8) {
                mx0 = fmax3(mx0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                mx1 = fmax3(mx1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
                mx2 = fmax3(mx2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
                mx3 = fmax3(mx3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
            }
            const float mxs = fmax3(mx0, mx1, fmaxf(mx2, mx3)) * c2;
            // the reference maximum moves only when it has grown by more than 2^8:
            // p and l use the same one, so the quotient is exact
            const bool need = mxs > m_ref + 8.0f;
            const bool any_need = __any_sync(0xffffffffu, need);
            const float m_new = need ? mxs : m_ref;
            const float alpha = need ? fast_exp2(m_ref - m_new) : 1.0f;
            m_ref = m_new;
            const float base = (m_ref == -INFINITY) ? 0.f : m_ref;
            const f32x2_t c2x2 = f2_pack(c2, c2);
            const f32x2_t nbx2 = f2_pack(-base, -base);
            f32x2_t lsum_a = f2_pack(0.f, 0.f), lsum_b = f2_pack(0.f, 0.f);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pk[32];
#pragma unroll
                for (int q = 0; q < 32; ++q) {
                    const int c = 64 * h + 2 * q;
                    const f32x2_t xv = f2_fma(
                        f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), c2x2, nbx2);
                    float x0, x1;
                    f2_unpack(xv, x0, x1);
                    const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
                    pk[q] = pack_bf16x2(e0, e1);
                    if (q & 1)
                        lsum_b = f2_add(lsum_b, f2_pack(e0, e1));
                    else
                        lsum_a = f2_add(lsum_a, f2_pack(e0, e1));
                }
                if (h == 0 && any_need && i > 0) {
                    // the commit that signalled S_t(i) covers P_t(i-1) V
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t orr[32];
                        tmem_ld32(tO + c, orr);
                        tmem_wait_ld(orr);
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            orr[q] = __float_as_uint(__uint_as_float(orr[q]) * alpha);
                        tmem_st32(tO + c, orr);
                    }
                }
                tmem_st32(tS + 32 * h, pk);
            }
            tmem_wait_st();
            softmax_arrive<true>(b.p_full(t), lane);
            float la0, la1, lb0, lb1;
            f2_unpack(lsum_a, la0, la1);
            f2_unpack(lsum_b, lb0, lb1);
            l = l * alpha + ((la0 + la1) + (lb0 + lb1));
        }
        const int n0 = uu.n0, n1 = uu.n1;
        it += wide ? max(n0, n1) : n0 + n1;

        // ---- epilogue
        const bool joins = !wide && n1 > 0;      // group 0 joins both groups' results
        const bool used = n > 0;
        if (used && !paged_warp_wait<false>(b.o_final(t), (o_par >> t) & 1, abort_flag)) return;
        float w0 = 1.f, w1 = 0.f;
        if (joins) {
            if (t == 1) {
                ml[r].x = m_ref;
                ml[r].y = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(b.ml_full(0));
            } else {
                // group 1 has waited for its own o_final by then
                if (!paged_warp_wait<false>(b.ml_full(0), ml_cnt & 1, abort_flag)) return;
                if (!paged_warp_wait<false>(b.o_final(1), o_par >> 1, abort_flag)) return;
                const float m1 = ml[r].x, l1 = ml[r].y;
                const float m = fmaxf(m_ref, m1);
                const float mb = m == -INFINITY ? 0.f : m;
                w0 = fast_exp2(m_ref - mb);
                w1 = fast_exp2(m1 - mb);
                // a NaN or infinite maximum leaves its NaN in l
                l = l * w0 + l1 * w1;
                m_ref = m;
            }
            ++ml_cnt;
        }
        o_par ^= (n0 > 0 ? 1u : 0u) | (n1 > 0 ? 2u : 0u);
        const bool writes = wide || t == 0;      // group 1 of a narrow unit only feeds group 0
        if (writes && active) {
            const int rows = rows_of(), tile_tok = token_of(), slot = uu.slot, hk = uu.hk, tok0 = uu.tok;
            const int my_tok = r / p.G, my_head = r - my_tok * p.G;
            const bool row_valid = r < rows;
            const float inv = l != 0.f ? 1.0f / l : 0.f;
            const float lse = l != 0.f ? (m_ref + log2f(l)) * 0.69314718055994531f : -INFINITY;
            const float f0 = inv * w0, f1 = inv * w1;
            tc_fence_after_sync();
            uint16_t* dst[4];
            float* part = nullptr;
            if (slot < 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rr = quarter * 32 + i * 8 + (lane >> 2);
                    const int tk = rr / p.G;
                    const size_t row =
                        (size_t)(tok0 + tile_tok + tk) * p.Hq + hk * p.G + (rr - tk * p.G);
                    dst[i] = rr < rows && dcheck(row < (size_t)p.T * p.Hq) ? p.o + row * D : nullptr;
                }
                const size_t row = (size_t)(tok0 + tile_tok + my_tok) * p.Hq + hk * p.G + my_head;
                if (row_valid && dcheck(row < (size_t)p.T * p.Hq)) p.lse[row] = lse;
            } else {
                const size_t row = (size_t)slot * 256 + (wide ? t * 128 : 0) + r;
                if (row_valid && dcheck(row < (size_t)512 * kPagedMaxCtas)) {
                    part = p.part_o + row * D;
                    p.part_lse[row] = lse;
                }
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t orr[32];
                if (used) {
                    tmem_ld32(tO + c, orr);
                    tmem_wait_ld(orr);
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        orr[q] = __float_as_uint(__uint_as_float(orr[q]) * f0);
                }
                if (joins) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t o1[16];
                        tmem_ld16(tO1 + c + 16 * h, o1);
                        tmem_wait_ld16(o1);
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            orr[16 * h + q] = __float_as_uint(
                                fmaf(__uint_as_float(o1[q]), f1, __uint_as_float(orr[16 * h + q])));
                    }
                }
                // a row that saw no key is 0 whatever its accumulator holds
                if (!used || l == 0.f) {
#pragma unroll
                    for (int q = 0; q < 32; ++q) orr[q] = 0;
                }
                if (slot < 0) {
                    uint32_t w[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        w[q] = pack_bf16x2(__uint_as_float(orr[2 * q]),
                                           __uint_as_float(orr[2 * q + 1]));
                    paged_store_chunk<D>(stage, w, lane, dst, c);
                } else if (part) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<uint4*>(part + c + 4 * q) = make_uint4(
                            orr[4 * q], orr[4 * q + 1], orr[4 * q + 2], orr[4 * q + 3]);
                }
            }
        }
        if (writes) {
            if (used) softmax_arrive<true>(b.o_free(t), lane);
            if (joins) softmax_arrive<true>(b.o_free(1), lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b.unit_empty(ri));
    }
}

// ---------------------------------------------------------------- kernel --
// One thread initialises the barriers of a CTA.
template <class T>
__device__ __forceinline__ void paged_init(const PagedBars<T>& b, const PagedShared& sh) {
    for (int i = 0; i < T::kSlots; ++i) {
        mbar_init(b.kv_full(i), 1);
        mbar_init(b.kv_empty(i), 1);
    }
    for (int i = 0; i < T::kPairs; ++i) mbar_init(b.v_raw(i), 1);
    for (int i = 0; i < T::kMasks; ++i) {
        mbar_init(b.mask_full(i), 1);
        mbar_init(b.v_given(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(b.tail_full(i), 1);
        mbar_init(b.tail_empty(i), 1);
        mbar_init(b.q_full(i), 1);
        mbar_init(b.q_empty(i), T::kIssuers);
        mbar_init(b.s_full(i), 1);
        mbar_init(b.p_full(i), 4);
        mbar_init(b.o_final(i), 1);
        mbar_init(b.o_free(i), 4);
    }
    for (int i = 0; i < T::kUnits; ++i) {
        mbar_init(b.unit_full(i), 1);
        // read by the issuers, the producers and 8 softmax warps
        mbar_init(b.unit_empty(i), T::kIssuers + T::kLoaders + 8);
    }
    for (int t = 0; t < 2; ++t) mbar_init(b.ml_full(t), 4);
    mbar_init(b.drain(), T::kIssuers);
    *sh.abort_flag = 0;
    fence_mbar_init();
}

template <int D, bool SPARSE>
__global__ void __launch_bounds__(PagedTraits<D>::kThreads, 1)
    attn_paged_sm100_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
    using T = PagedTraits<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    PagedBars<T> b;
    b.base = smem_addr(smem + T::kOffBars);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + T::kOffMisc);
    PagedShared sh;
    sh.smem = smem;
    sh.abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    sh.tail_info = reinterpret_cast<int*>(tmem_holder + 2);
    sh.tail_mask = tmem_holder + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the merge may be set up as soon as SMs have room; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) paged_init<T>(b, sh);
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 9) {
        tmem_alloc(smem_addr(tmem_holder), 512);
        tmem_relinquish();
    }
    // the staging area is free until the first epilogue
    // nothing that an earlier kernel may still write or read was touched so far
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedStretch st =
        paged_schedule<T::kThreads>(p, reinterpret_cast<long long*>(smem + T::kOffStage));
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tbase = *tmem_holder;

    if (warp < 8) {
        regs_increase<T::kSoftmaxRegs>();
        paged_softmax<D>(p, tbase, b, sh, warp, lane);
    } else {
        regs_decrease<T::kOtherRegs>();
        if (warp == 8)
            paged_producer<T, SPARSE, true, true>(p, &tm_q, &tm_k, &tm_v, b, sh, lane);
        else if (warp == 9) {
            if (lane == 0) paged_mma<D>(tbase, b, sh);
        } else if (warp == 10)
            paged_tail<T>(b, sh, lane);
        else
            paged_planner<T, SPARSE>(p, st, b, sh, lane);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 9) {
        __syncwarp();
        tmem_dealloc(tbase, 512);
    }
}

// Joins the partial rows of every unit that was cut: block (c, y) takes rows of the
// unit that CTA c began and did not finish; its other pieces are in the slots
// 2 (c + 1), 2 (c + 2), ... up to the one marked last.
//   M = max_s lse_s;  O = sum_s 2^((lse_s - M) log2 e) O_s / W;  LSE = M + ln W
constexpr int kPagedMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kPagedMergeThreads)
    attn_paged_merge_kernel(const PagedParams p, int ctas) {
    constexpr int kPerRow = D / 4, kRows = kPagedMergeThreads / kPerRow;
    // launched while the attention kernel still runs; nothing of it is read before it is over
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x;
    const PagedPiece first = p.pieces[2 * c + 1];
    if (!first.valid) return;
    // how many pieces the unit has: up to the one marked last
    int pieces = 1;
    for (const int lane = threadIdx.x & 31;; pieces += 32) {
        const int at = c + pieces + lane;
        const bool end = at >= ctas || !p.pieces[2 * at].valid || p.pieces[2 * at].last;
        const unsigned m = __ballot_sync(0xffffffffu, end);
        if (m) {
            const int i = __ffs(m) - 1, last = c + pieces + i;
            pieces += i + (last < ctas && p.pieces[2 * last].valid ? 1 : 0);
            break;
        }
    }
    constexpr float kLog2e = 1.4426950408889634f;
    const int col = threadIdx.x % kPerRow;
    // R: row of the unit's (at most) 256
    for (int R = blockIdx.y * kRows + threadIdx.x / kPerRow; R < 256; R += gridDim.y * kRows) {
        const int t = R >> 7, r = R & 127;
        if (r >= min(max(first.ntok - t * p.tpt, 0), p.tpt) * p.G) continue;
        float M = -INFINITY, W = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        // piece 0 is in slot 2 c + 1, piece i > 0 in slot 2 (c + i); four in flight
        for (int i0 = 0; i0 < pieces; i0 += 4) {
            float ls[4];
            float4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = min(i0 + k, pieces - 1);
                const size_t row = (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * 256 + R;
                ls[k] = p.part_lse[row];
                x[k] = *reinterpret_cast<const float4*>(p.part_o + row * D + 4 * col);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (i0 + k >= pieces) break;
                const float mn = fmaxf(M, ls[k]);
                if (mn != -INFINITY) {
                    // NaN partials stay NaN: fmaxf drops them from the maximum, not from W
                    const float a = fast_exp2((M - mn) * kLog2e), w = fast_exp2((ls[k] - mn) * kLog2e);
                    W = W * a + w;
                    acc.x = acc.x * a + w * x[k].x;
                    acc.y = acc.y * a + w * x[k].y;
                    acc.z = acc.z * a + w * x[k].z;
                    acc.w = acc.w * a + w * x[k].w;
                    M = mn;
                } else if (!(ls[k] == -INFINITY)) {
                    W = ls[k];   // NaN and nothing before it
                }
            }
        }
        const int tk = r / p.G;
        const size_t row =
            (size_t)(first.tok + t * p.tpt + tk) * p.Hq + first.hk * p.G + (r - tk * p.G);
        if (!dcheck(row < (size_t)p.T * p.Hq)) continue;
        const float inv = W != 0.f ? 1.0f / W : 0.f;
        *reinterpret_cast<uint2*>(p.o + row * D + 4 * col) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (col == 0) p.lse[row] = W != 0.f ? M + logf(W) : -INFINITY;
    }
}

}  // namespace eattn
