// paged_rows_sm100.cuh -- attention of few rows over a paged K/V cache: decode,
// drafted tokens, and rows that each read pages of their own.
//
// The same sums as paged_fwd_sm100.cuh, for units of at most N = 16 or 32
// rows (token, head of the group). There, 128 rows of a tile are computed
// whatever the unit has, and the thread of a row takes its 128 scores one after
// another: with 4 rows of 128 in use that thread sets the pace (1.4 us per key
// tile), not memory. Here the tile is turned: keys are the 128 rows of the
// product and the unit's rows its columns,
//   S^T = K Q^T  [128 keys x N],   O^T += V^T P^T  [D x N],
// so 128 threads share each tile's exponentials (N each) and the products take
// N / 128 of the time. What the turn asks for:
//   * maxima run across threads. The reference maximum of a row moves only
//     when a score exceeds it by 2^8 (rare after a unit's first tile), so per
//     tile the four warps of a group only vote (one barrier with an "or"); the
//     reduction and the rescaling of O happen when the vote says so.
//   * sums stay one partial per thread until the unit ends.
//   * P goes to shared memory (bf16, 128-byte swizzle) as the second operand;
//     V, stored [keys][D], is the first operand as it lies (M-major).
// The two softmax groups take alternate key tiles, each with its own issuing
// thread, so neither waits for the other; they take turns at joining their results
// (group 0 when it alone had a tile).
//
// Warps: 0-3 and 4-7 softmax, 8 loads Q and K, 13 V, 9 and 11 issue the products of
// group 0 and 1, 10 cleans V tiles, 12 plans. Measured (CUDA graph): 16 sequences of 32768
// keys, 32 query heads on 8, 327 us = 6.57 TB/s of K/V, the card's copy rate (128-row form:
// 354); 1098 rows over 16 pages of 64 each, 553 us (128-row form: 1449), 8.3 TB/s of K/V tiles
// mostly out of L2: no unit is near its limit there (L2 at 36% of its peak, DRAM 11%, tensor pipe
// 7%), so what bounds it is the loads' latency with three tile pairs in flight and units that
// are 8 tiles long; 7 sequences of up to 6 drafted tokens, 25 us, most of it start-up.
#pragma once

#include <cfloat>

#include "paged_fwd_sm100.cuh"

namespace eattn {

// Named barrier over one softmax group (ids 1 and 2), and the same with an "or".
__device__ __forceinline__ void group_sync(int t) {
    asm volatile("bar.sync %0, 128;" ::"r"(t + 1) : "memory");
}
__device__ __forceinline__ bool group_any(int t, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(t + 1)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// The largest of a warp's 32 values, in every lane (NaN ignored).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Sums of 16 values over a warp: lane l ends with the sum of value l / 2.
__device__ __forceinline__ float warp_sum16(float (&v)[16], int lane) {
#pragma unroll
    for (int half = 8; half >= 1; half >>= 1) {
        const bool hi = (lane & (2 * half)) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = hi ? v[i] : v[i + half], keep = hi ? v[i + half] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * half);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// 8 columns of this warp's 32 tensor-memory lanes; the wait takes in two such loads.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld8(uint32_t (&a)[8], uint32_t (&b)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]),
                   "+r"(a[6]), "+r"(a[7]), "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]),
                   "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
                 :
                 : "memory");
}

// N consecutive columns of this warp's 32 tensor-memory lanes
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 16) {
        tmem_ld16(taddr, r);
        tmem_wait_ld16(r);
    } else {
        tmem_ld32(taddr, r);
        tmem_wait_ld(r);
    }
}
// ------------------------------------------------------------ MMA issuer --
// The thread of group t issues S^T and O^T of key tiles t, t + 2, ... of a unit:
// P(i) V, then S(i + 1). A completed S(i + 1) therefore means that P(i) V is
// complete too.
template <int D, int N>
__device__ void rows_mma(uint32_t tbase, const PagedBars<PagedTraits<D, N>>& b,
                         const PagedShared& sh, int t) {
    using T = PagedTraits<D, N>;
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, N, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(D, N, false) | (1u << 15);   // V^T: M-major
    const uint32_t sQ = smem_addr(sh.smem), sKV = sQ + T::kOffKV;
    const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024);
    const uint64_t dk0 = sdesc_sw128(sKV, 16, 1024);
    const uint64_t dv0 = sdesc_sw128(sKV, T::kPanelBytes, 1024);
    const uint64_t dp = sdesc_sw128(sQ + T::kOffStage + t * N * 256, 16, 1024);
    const uint32_t tS = tbase + (t ? T::kColS1 : T::kColS0);
    const uint32_t tO = tbase + (t ? T::kColO1 : T::kColO0);
    volatile int* abort_flag = sh.abort_flag;
    const PagedUnit* ring = reinterpret_cast<const PagedUnit*>(sh.smem + T::kOffUnits);
    uint32_t it = 0, units = 0, o_used = 0, p_cnt = 0;
    uint32_t q_par[2] = {0, 0};
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return paged_wait(bar, parity, abort_flag);
    };
    for (;; ++units) {
        const int ri = units % T::kUnits;
        if (!wait(b.unit_full(ri), (units / T::kUnits) & 1)) goto done;
        const volatile PagedUnit& u = ring[ri];
        const int kind = u.kind, n = t ? u.n1 : u.n0, all = u.n0 + u.n1, qs = u.qs;
        mbar_arrive(b.unit_empty(ri));
        if (kind == 0) break;
        if (all == 0) continue;
        if (!wait(b.q_full(qs), q_par[qs])) goto done;
        q_par[qs] ^= 1;
        const uint64_t dq = dq0 + qs * (T::kQBytes >> 4);
        auto issue_s = [&](int i) -> bool {
            const uint32_t x = it + 2 * i + t, sk = 2 * (x % T::kPairs);
            // the slot's last use may have been the other group's: first see that it is over
            if (!wait(b.mask_full(x % T::kMasks), (x / T::kMasks) & 1)) return false;
            if (!wait(b.kv_full(sk), (x / T::kPairs) & 1)) return false;
            tc_fence_after_sync();
            const uint64_t dk = dk0 + sk * (T::kTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma_bf16_ss(tS, dk + (((kk / 4) * T::kPanelBytes + (kk % 4) * 32) >> 4),
                            dq + (((kk / 4) * T::kQPanelBytes + (kk % 4) * 32) >> 4), idesc_s,
                            kk > 0 ? 1u : 0u);
            mma_commit(b.s_full(t));
            mma_commit(b.kv_empty(sk));
            if (i == n - 1) mma_commit(b.q_empty(qs));
            return true;
        };
        if (n == 0) {
            mma_commit(b.q_empty(qs));
        } else if (!issue_s(0)) {
            goto done;
        }
        for (int i = 0; i < n; ++i) {
            const uint32_t x = it + 2 * i + t, sv = 2 * (x % T::kPairs) + 1;
            if (!wait(b.v_given(x % T::kMasks), (x / T::kMasks) & 1)) goto done;
            if (!wait(b.kv_full(sv), (x / T::kPairs) & 1)) goto done;
            if (!wait(b.p_full(t), p_cnt & 1)) goto done;
            ++p_cnt;
            if (i == 0 && o_used > 0 && !wait(b.o_free(t), (o_used - 1) & 1)) goto done;
            tc_fence_after_sync();
            const uint64_t dv = dv0 + sv * (T::kTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)      // 16 keys each
                mma_bf16_ss(tO, dv + ((kk * 16 * 128) >> 4),
                            dp + (((kk / 4) * N * 128 + (kk % 4) * 32) >> 4), idesc_o,
                            (i > 0 || kk > 0) ? 1u : 0u);
            mma_commit(b.kv_empty(sv));
            if (i == n - 1) mma_commit(b.o_final(t));
            if (i + 1 < n && !issue_s(i + 1)) goto done;
        }
        if (n > 0) ++o_used;
        it += all;
    }
done: {
    // Every MMA this thread issued must finish before tensor memory is released.
    volatile int no_abort = 0;
    mma_commit(b.drain());
    paged_wait(b.drain(), 0, &no_abort);
}
}

// --------------------------------------------------------------- softmax --
// Thread r of group t is key r of the group's tiles, and then lane r of O^T:
// dimension r (D = 128), or dimension 16 (r / 32) + r % 32 for r % 32 < 16 (D = 64,
// a product of 64 rows fills half of each 32 lanes).
//
// The four warps of a group meet at named barriers, which wait without a limit: so a
// warp whose bounded wait has given up goes on to the next vote, and the whole
// group leaves there together.
template <int D, int N>
__device__ void rows_softmax(const PagedParams& p, uint32_t tbase,
                             const PagedBars<PagedTraits<D, N>>& b, const PagedShared& sh, int warp,
                             int lane) {
    using T = PagedTraits<D, N>;
    const int t = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const uint32_t tS = tbase + lane_off + (t ? T::kColS1 : T::kColS0);
    const uint32_t tO = tbase + lane_off + (t ? T::kColO1 : T::kColO0);
    const uint32_t tOther = tbase + lane_off + (t ? T::kColO0 : T::kColO1);
    volatile int* abort_flag = sh.abort_flag;
    const PagedUnit* ring = reinterpret_cast<const PagedUnit*>(sh.smem + T::kOffUnits);
    const volatile uint32_t* masks =
        reinterpret_cast<const volatile uint32_t*>(sh.smem + T::kOffMask);
    // per row: (m, l) for the joining group, and each group's weights as it joins;
    // per group: the negated reference maximum (the lowest float before the
    // first key: every score is far above it), the factor of a rescaling, a word per warp
    float2* ml = reinterpret_cast<float2*>(sh.smem + T::kOffMl);
    float2* weight = ml + (1 + t) * N;
    float* minus_ref = reinterpret_cast<float*>(sh.smem + T::kOffMl + 3 * N * 8) + t * 6 * N;
    float* alpha = minus_ref + N;
    float* red = alpha + N;
    // where key r of row c goes in P: 128-byte rows of 64 keys, 16-byte pieces swizzled by row
    const uint32_t sP =
        smem_addr(sh.smem) + T::kOffStage + t * N * 256 + (r >> 6) * N * 128 + (r & 7) * 2;
    const uint32_t piece = (r & 63) >> 3;
    constexpr int kChunk = N == 16 ? 8 : 16;    // columns skipped together when no row has them
    const float c2 = p.scale_log2;
    uint32_t it = 0, s_cnt = 0, ml_cnt = 0;
    uint32_t o_used[2] = {0, 0};

    for (uint32_t units = 0;; ++units) {
        const int ri = units % T::kUnits;
        const bool got = paged_warp_wait(b.unit_full(ri), (units / T::kUnits) & 1, abort_flag);
        if (r < N) minus_ref[r] = FLT_MAX;
        if (group_any(t, !got)) return;
        const volatile PagedUnit& uu = ring[ri];
        const int kind = uu.kind, hk = uu.hk, tok0 = uu.tok, ntok = uu.ntok, pos0 = uu.pos0;
        const int len = uu.len, key0 = uu.key0, un[2] = {uu.n0, uu.n1}, slot = uu.slot;
        __syncwarp();
        if (lane == 0) mbar_arrive(b.unit_empty(ri));
        if (kind == 0) break;
        const int n = un[t], rows = ntok * p.G;   // columns [0, rows) are in use
        const bool diag = p.causal && len != 0x7fffffff;
        float l[N];
#pragma unroll
        for (int c = 0; c < N; ++c) l[c] = 0.f;
        for (int i = 0; i < n; ++i) {
            const uint32_t x = it + 2 * i + t;
            bool ok = paged_warp_wait(b.mask_full(x % T::kMasks), (x / T::kMasks) & 1, abort_flag);
            const bool there = (masks[4 * (x % T::kMasks) + quarter] >> lane) & 1;
            // rows [first, N) see this key
            const long long key = (long long)key0 + (2 * i + t) * 128 + r;
            const long long behind = diag ? key - pos0 : 0;   // tokens before the key's own
            const int first = !there ? N : behind <= 0 ? 0 : behind >= N ? N : (int)behind * p.G;
            ok = ok && paged_warp_wait(b.s_full(t), s_cnt & 1, abort_flag);
            ++s_cnt;
            tc_fence_after_sync();
            // exponents of every column in use, and whether one of them is above 2^8
            const bool masked = __any_sync(0xffffffffu, first > 0);
            float arg[N];
            auto exponents = [&]() -> bool {
                float top = -INFINITY;
                uint32_t sr[N];
                tmem_ld_cols<N>(tS, sr);
#pragma unroll
                for (int c0 = 0; c0 < N; c0 += kChunk) {
                    if (c0 < rows) {
#pragma unroll
                        for (int c = c0; c < c0 + kChunk; c += 4) {
                            const float4 m = *reinterpret_cast<const float4*>(minus_ref + c);
                            arg[c] = fmaf(__uint_as_float(sr[c]), c2, m.x);
                            arg[c + 1] = fmaf(__uint_as_float(sr[c + 1]), c2, m.y);
                            arg[c + 2] = fmaf(__uint_as_float(sr[c + 2]), c2, m.z);
                            arg[c + 3] = fmaf(__uint_as_float(sr[c + 3]), c2, m.w);
                        }
                        if (masked) {
#pragma unroll
                            for (int c = c0; c < c0 + kChunk; ++c)
                                if (c < first) arg[c] = -INFINITY;
                        }
#pragma unroll
                        for (int c = c0; c < c0 + kChunk; c += 2)
                            top = fmax3(top, arg[c], arg[c + 1]);
                    }
                }
                return top > 8.0f;
            };
            for (bool again = false;; again = true) {
                const bool over = exponents();
                if (again || !group_any(t, over || !ok)) break;
                if (group_any(t, !ok)) return;
                // the reference of every row moves to its maximum so far
#pragma unroll 1
                for (int c0 = 0; c0 < rows; c0 += 16) {
                    uint32_t sr[16];
                    tmem_ld16(tS + c0, sr);
                    tmem_wait_ld16(sr);
                    float mine = 0.f;
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float v = warp_max(
                            c0 + c >= first ? __uint_as_float(sr[c]) * c2 : -INFINITY);
                        if (lane == c) mine = v;
                    }
                    if (lane < 16) red[quarter * N + c0 + lane] = mine;
                }
                group_sync(t);
                if (r < N) {    // columns without a row too: they share their chunk's vote
                    const float m_old = -minus_ref[r];
                    const float v = fmaxf(fmaxf(red[r], red[N + r]),
                                          fmaxf(red[2 * N + r], red[3 * N + r]));
                    const float m_new = fmaxf(m_old, v);
                    alpha[r] = fast_exp2(m_old - m_new);
                    minus_ref[r] = -m_new;
                }
                group_sync(t);
#pragma unroll
                for (int c0 = 0; c0 < N; c0 += kChunk) {
                    if (c0 < rows) {
#pragma unroll
                        for (int c = c0; c < c0 + kChunk; c += 4) {
                            const float4 a = *reinterpret_cast<const float4*>(alpha + c);
                            l[c] *= a.x;
                            l[c + 1] *= a.y;
                            l[c + 2] *= a.z;
                            l[c + 3] *= a.w;
                        }
                    }
                }
                if (i > 0) {      // S(i) is complete, so P(i-1) V is
#pragma unroll 1
                    for (int c = 0; c < rows; c += 16) {
                        uint32_t orr[16];
                        tmem_ld16(tO + c, orr);
                        tmem_wait_ld16(orr);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            orr[k] = __float_as_uint(__uint_as_float(orr[k]) * alpha[c + k]);
                        tmem_st16(tO + c, orr);
                    }
                    tmem_wait_st();
                }
            }
#pragma unroll
            for (int c0 = 0; c0 < N; c0 += kChunk) {
                if (c0 < rows) {
#pragma unroll
                    for (int c = c0; c < c0 + kChunk; c += 2) {
                        const float e0 = fast_exp2(arg[c]), e1 = fast_exp2(arg[c + 1]);
                        l[c] += e0;
                        l[c + 1] += e1;
                        const uint32_t pk = pack_bf16x2(e0, e1);
                        st_shared_u16(sP + c * 128 + ((piece ^ (c & 7)) << 4), (uint16_t)pk);
                        st_shared_u16(sP + (c + 1) * 128 + ((piece ^ ((c + 1) & 7)) << 4),
                                      (uint16_t)(pk >> 16));
                    }
                }
            }
            fence_async_shared();
            softmax_arrive<true>(b.p_full(t), lane);
        }
        it += un[0] + un[1];

        // ---- sums over the group's keys, then the two groups joined by group 0
        float m = -INFINITY, sum = 0.f;    // of row r, in the threads r < N
        if (n > 0) {
#pragma unroll
            for (int c0 = 0; c0 < N; c0 += 16) {
                if (c0 < rows) {
                    float v[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = l[c0 + c];
                    const float x = warp_sum16(v, lane);
                    if ((lane & 1) == 0) red[quarter * N + c0 + (lane >> 1)] = x;
                }
            }
            const bool ok = paged_warp_wait(b.o_final(t), o_used[t] & 1, abort_flag);
            if (group_any(t, !ok)) return;
            if (r < N && r < rows) {
                m = -minus_ref[r];
                sum = (red[r] + red[N + r]) + (red[2 * N + r] + red[3 * N + r]);
            }
        }
        const bool both = un[1] > 0;
        const int joiner = both ? (int)(units & 1) : 0;
        if (t != joiner) {
            if (both) {
                if (r < N) ml[r] = make_float2(m, sum);
                __syncwarp();
                if (lane == 0) mbar_arrive(b.ml_full(joiner));
            }
        } else {
            if (both) {
                // the other group has waited for its own o_final by then
                const bool ok = paged_warp_wait(b.ml_full(t), ml_cnt & 1, abort_flag) &&
                                paged_warp_wait(b.o_final(t ^ 1), o_used[t ^ 1] & 1, abort_flag);
                if (group_any(t, !ok)) return;
                ++ml_cnt;
            }
            if (r < N && r < rows) {
                float w0 = n > 0 ? 1.f : 0.f, w1 = 0.f;
                if (both) {
                    const float2 o = ml[r];
                    const float mn = fmaxf(m, o.x);
                    w0 = fast_exp2(m - mn);
                    w1 = fast_exp2(o.x - mn);
                    sum = sum * w0 + o.y * w1;
                    m = mn;
                }
                const float inv = sum != 0.f ? 1.0f / sum : 0.f;
                weight[r] = make_float2(w0 * inv, w1 * inv);
                const float lse = sum != 0.f ? (m + log2f(sum)) * 0.69314718055994531f : -INFINITY;
                if (slot < 0) {
                    const int tk = r / p.G;
                    const size_t row = (size_t)(tok0 + tk) * p.Hq + hk * p.G + (r - tk * p.G);
                    if (dcheck(row < (size_t)p.T * p.Hq)) p.lse[row] = lse;
                } else if (dcheck(slot < 2 * kPagedMaxCtas)) {
                    p.part_lse[(size_t)slot * 256 + r] = lse;
                }
            }
            group_sync(t);
            tc_fence_after_sync();
            const int dim = D == 128 ? r : quarter * 16 + lane;
            const bool has_dim = D == 128 || lane < 16;
            const size_t row0 = slot < 0 ? (size_t)tok0 * p.Hq + hk * p.G : (size_t)slot * 256;
            uint16_t* dst = p.o + row0 * D + dim;
            float* part = p.part_o + row0 * D + dim;
            const size_t skip = (size_t)(p.Hq - p.G) * D;    // to the group's heads of the next token
            int head = 0;
#pragma unroll 1
            for (int c0 = 0; c0 < rows; c0 += 8) {
                uint32_t o0[8], o1[8];
                tmem_ld8(tO + c0, o0);
                tmem_ld8(tOther + c0, o1);
                tmem_wait_ld8(o0, o1);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (c0 + c >= rows) break;
                    const float2 w = weight[c0 + c];
                    float v = n > 0 ? __uint_as_float(o0[c]) * w.x : 0.f;
                    if (both) v = fmaf(__uint_as_float(o1[c]), w.y, v);
                    if (slot < 0) {
                        if (has_dim && dcheck(dst < p.o + (size_t)p.T * p.Hq * D))
                            *dst = (uint16_t)pack_bf16x2(v, 0.f);
                        dst += D;
                        if (++head == p.G) {
                            head = 0;
                            dst += skip;
                        }
                    } else {
                        if (has_dim && dcheck(part < p.part_o + (size_t)512 * kPagedMaxCtas * D))
                            *part = v;
                        part += D;
                    }
                }
            }
            group_sync(t);       // the weights are read
            if (n > 0) softmax_arrive<true>(b.o_free(t), lane);
            if (both) softmax_arrive<true>(b.o_free(t ^ 1), lane);
        }
        for (int k = 0; k < 2; ++k)
            if (un[k] > 0) ++o_used[k];
    }
}

// ---------------------------------------------------------------- kernel --
template <int D, int N, bool SPARSE>
__global__ void __launch_bounds__(PagedTraits<D, N>::kThreads, 1)
    attn_paged_rows_sm100_kernel(const __grid_constant__ CUtensorMap tm_q,
                                 const __grid_constant__ CUtensorMap tm_k,
                                 const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
    using T = PagedTraits<D, N>;
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

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge, as there
    if (threadIdx.x == 0) paged_init<T>(b, sh);
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 9) {
        tmem_alloc(smem_addr(tmem_holder), 256);
        tmem_relinquish();
    }
    // Q rows that no copy ever writes are zeros, so their columns stay finite
    for (int i = threadIdx.x; i < 2 * T::kQBytes / 16; i += T::kThreads)
        reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    fence_async_shared();
    // P's area is free until the first tile
    // nothing that an earlier kernel may still write or read was touched so far
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedStretch st =
        paged_schedule<T::kThreads>(p, reinterpret_cast<long long*>(smem + T::kOffStage));
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tbase = *tmem_holder;

    if (warp < 8)
        rows_softmax<D, N>(p, tbase, b, sh, warp, lane);
    else if (warp == 8)
        paged_producer<T, SPARSE, true, false>(p, &tm_q, &tm_k, &tm_v, b, sh, lane);
    else if (warp == 13)
        paged_producer<T, SPARSE, false, true>(p, &tm_q, &tm_k, &tm_v, b, sh, lane);
    else if (warp == 9 || warp == 11) {
        if (lane == 0) rows_mma<D, N>(tbase, b, sh, warp == 9 ? 0 : 1);
    } else if (warp == 10)
        paged_tail<T>(b, sh, lane);
    else
        paged_planner<T, SPARSE>(p, st, b, sh, lane);
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 9) {
        __syncwarp();
        tmem_dealloc(tbase, 256);
    }
}

}  // namespace eattn
