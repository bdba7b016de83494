// paged_host.cuh -- host-side choices of the serving entry points, apart from CUDA so that they
// can be checked without it.
#pragma once

namespace eattn {

// CTAs of the block-table cluster: as many as there are rows for, `threads` a CTA. 16 is more
// than the 8 that every context can place (a context with few SMs of a GPC has no room for it),
// so it is taken only where `sixteen_fit`. On 47,000 rows of 500 sequences 16 CTAs take 7.1 us, 8
// took 10.0.
inline int tables_ctas(long long rows, int threads, bool sixteen_fit) {
    if (rows <= threads) return 1;
    if (rows <= 2ll * threads) return 2;
    if (rows <= 8ll * threads || !sixteen_fit) return 8;
    return 16;
}

}  // namespace eattn
