// paged_drain.cuh -- which copies a producer that gives up still has to wait for.
// Plain C++ (no CUDA headers), so that the rule can be checked on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define EATTN_DRAIN_FN __device__ __forceinline__
#else
#define EATTN_DRAIN_FN inline
#endif

namespace eattn {

// A producer has counted `it` key tiles into a ring of `pairs` K/V slot pairs (tile i in pair
// i % pairs); with v_skipped, the last of them got no V copy, because the wait for its V slot or
// for what follows did not end. Whatever is in flight is the last copy of some slot: calls
// k(pair, parity) for the K slots and v(pair, raw, parity) for the V slots, with the parity of the
// barrier phase that the copy completes. A V copy completes kv_full, one phase per tile, or,
// where rows have to be zeroed behind it, v_raw: bit `pair` of raw_last says which of the two the
// slot's last copy does, that of raw_par is the number of v_raw phases so far, modulo 2.
template <bool K, bool V, class WaitK, class WaitV>
EATTN_DRAIN_FN void paged_drain(uint32_t it, bool v_skipped, uint32_t pairs, uint32_t raw_par,
                                uint32_t raw_last, WaitK k, WaitV v) {
    for (uint32_t i = it > pairs ? it - pairs : 0; i < it; ++i) {
        const uint32_t pair = i % pairs;
        uint32_t round = i / pairs;
        if (K) k(pair, round & 1);
        if (!V) continue;
        if (v_skipped && i + 1 == it) {   // the slot still belongs to the tile a round before
            if (round == 0) continue;
            --round;
        }
        const bool raw = (raw_last >> pair) & 1;
        v(pair, raw, raw ? ((raw_par >> pair) & 1) ^ 1 : round & 1);
    }
}

}  // namespace eattn
