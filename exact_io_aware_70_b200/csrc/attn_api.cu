// attn_api.cu -- the C ABI declared in include/exact_attn.h.
//
// Argument checking, TMA tensor-map encoding and kernel launches. This is the
// only translation unit of the library that includes the kernels (they live
// in the .cuh files below) and defines the device status word, so that word
// has a single definition. The library's other translation unit,
// attn_noalloc.cu, holds the allocation-free decode's scratch array and calls
// only the extern "C" entry points defined here.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "exact_attn.h"

namespace eattn {
// Device status word: kernels OR error bits into it; attn_status() reads and clears it.
__device__ unsigned g_attn_status = 0;
}  // namespace eattn

#include "bwd_sm100.cuh"
#include "decode_sm100.cuh"
#include "fwd_sm100.cuh"
#include "paged_cache_sm100.cuh"
#include "paged_fwd_sm100.cuh"
#include "paged_host.cuh"
#include "paged_rows_sm100.cuh"

using namespace eattn;

namespace eattn {
// Waits on an mbarrier that nothing ever arrives on, through the same bounded
// wait every pipeline kernel uses, so the give-up path can be exercised
// without faulting or hanging the GPU.
__global__ void attn_wait_selftest_kernel(unsigned long long limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&bar), 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) mbar_wait_limit(smem_addr(&bar), 0, &abort_flag, &g_attn_status, limit_ns);
}
}  // namespace eattn

namespace {

constexpr int kAbiVersion = 1;
constexpr float kLog2e = 1.4426950408889634f;
constexpr long long kMaxSeq = 1ll << 30;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Encodes a 3-D tiled map whose rows beyond the tensor read as zero. The driver call needs a
// current context, which a host thread gets with its first runtime call that uses the device:
// where this is the thread's first call of all, the device's context is made current first.
bool encode_tiled(CUtensorMap* map, CUtensorMapDataType type, const void* base,
                  const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                  const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    const cuuint32_t estr[3] = {1, 1, 1};
    auto encode = [&] {
        return enc(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = encode();
    if (r != CUDA_SUCCESS && r != CUDA_ERROR_INVALID_VALUE) {
        int dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encode();
    }
    return r == CUDA_SUCCESS;
}

// Tensor map over a bf16 tensor viewed as [BH][N][D]; box = box_rows rows x 64
// columns, 128-byte swizzle, out-of-range rows read as zero.
bool encode_bf16_map(CUtensorMap* map, const void* base, int BH, int N, int D,
                     int box_rows = 128) {
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base,
                        {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)BH},
                        {(cuuint64_t)D * 2, (cuuint64_t)N * D * 2}, {64, (cuuint32_t)box_rows, 1},
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

// Tensor map over an 8-bit tensor viewed as [BH][N][D] with D = 128 or 64: box =
// 128 rows x D bytes, 128-byte swizzle (64-byte swizzle for D = 64), rows past
// N read as zero.
bool encode_u8_map(CUtensorMap* map, const void* base, int BH, int N, int D) {
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base,
                        {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)BH},
                        {(cuuint64_t)D, (cuuint64_t)N * D}, {(cuuint32_t)D, 128, 1},
                        D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Tensor map over q viewed as [T][Hq][D] with `stride` elements from row to row;
// box = `tokens` rows x the `heads` query heads of a group x 64 columns.
bool encode_q_map(CUtensorMap* map, const void* base, int T, int Hq, int D, long long stride,
                  int heads, int tokens) {
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base,
                        {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T},
                        {(cuuint64_t)D * 2, (cuuint64_t)stride * 2},
                        {64, (cuuint32_t)heads, (cuuint32_t)tokens}, CU_TENSOR_MAP_SWIZZLE_128B);
}

struct DeviceInfo {
    int sms = 0;
    bool paged_attr_set[12] = {};
    bool tables_attr_set = false, tables_sixteen = false;
    bool score_attr_set[4] = {};
    bool fwd_attr_set[8] = {false, false, false, false, false, false, false, false};
    bool bwd_attr_set[4] = {false, false, false, false};
};
DeviceInfo g_dev[64];
std::mutex g_dev_mu;

int current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    return dev;
}

// Unit-queue entry of the next forward launch (round robin): two launches
// share an entry only if kFwdQueueSlots further launches are started while
// the first is still running.
std::atomic<unsigned> g_fwd_queue_rr{0};

// Heads per group of the forward's unit order: as many heads as keep their
// K and V within EATTN_FWD_GROUP_BYTES, so the CTAs in flight find them in
// L2. Measured at 16K (8 MB of K/V per head): 16, 32, 48, 64, 96 and 128 MB
// groups ran 3.63, 3.55-3.59, 3.58, 3.50-3.54, 3.67 and 3.58 ms.
#ifndef EATTN_FWD_GROUP_BYTES
#define EATTN_FWD_GROUP_BYTES (64ll << 20)
#endif
int fwd_group_heads(int BH, int Nkv, int d, int elem_bytes) {
    const long long per_head = 2ll * Nkv * d * elem_bytes;
    long long g = EATTN_FWD_GROUP_BYTES / (per_head > 0 ? per_head : 1);
    if (g < 1) g = 1;
    return g < BH ? (int)g : BH;
}
// Units are dealt dynamically, in head groups, only when the K and V of all
// heads exceed this (the launch's K/V then cannot stay in the 126 MB L2 while
// every head is in flight); below it a static deal of the heaviest-first
// order is used. 0 forces the dynamic queue, a huge value the static deal.
// 1: the static deal also walks the units in head groups (measured slower)
#ifndef EATTN_FWD_STATIC_GROUPS
#define EATTN_FWD_STATIC_GROUPS 0
#endif
#ifndef EATTN_FWD_QUEUE_MIN_BYTES
#define EATTN_FWD_QUEUE_MIN_BYTES (192ll << 20)
#endif

template <int D, bool CAUSAL, bool FP8 = false>
attn_status_t launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CUtensorMap& to, FwdParams p, cudaStream_t stream) {
    using T = FwdTraits<D, FP8>;
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return ATTN_ERR_CUDA;
    auto kern = attn_fwd_sm100_kernel<D, CAUSAL, FP8>;
    int sms;
    {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        DeviceInfo& di = g_dev[dev];
        if (di.sms == 0 &&
            cudaDeviceGetAttribute(&di.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return ATTN_ERR_CUDA;
        const int slot = (FP8 ? 4 : 0) + (D == 128 ? 2 : 0) + (CAUSAL ? 1 : 0);
        if (!di.fwd_attr_set[slot]) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     T::kSmemBytes) != cudaSuccess)
                return ATTN_ERR_CUDA;
            di.fwd_attr_set[slot] = true;
        }
        sms = di.sms;
    }
    const int grid = p.num_units < sms ? p.num_units : sms;
    p.dynamic_units =
        2ll * p.BH * p.Nkv * D * T::kElemBytes > EATTN_FWD_QUEUE_MIN_BYTES ? 1 : 0;
    // EXACT_ATTN_FWD_SCHEDULE=dynamic|static overrides the choice (for tests
    // and measurements; the result is the same either way)
    if (const char* sched = std::getenv("EXACT_ATTN_FWD_SCHEDULE")) {
        if (std::strcmp(sched, "dynamic") == 0) p.dynamic_units = 1;
        if (std::strcmp(sched, "static") == 0) p.dynamic_units = 0;
    }
    p.group_heads = (p.dynamic_units || EATTN_FWD_STATIC_GROUPS)
                        ? fwd_group_heads(p.BH, p.Nkv, D, T::kElemBytes)
                        : p.BH;
    p.queue_slot = (int)(g_fwd_queue_rr.fetch_add(1, std::memory_order_relaxed) % kFwdQueueSlots);
    kern<<<grid, T::kThreads, T::kSmemBytes, stream>>>(tq, tk, tv, to, p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, bool CAUSAL>
attn_status_t launch_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CUtensorMap& tdo, const BwdParams& p, cudaStream_t stream) {
    using T = BwdTraits<D>;
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return ATTN_ERR_CUDA;
    auto kern = attn_bwd_sm100_kernel<D, CAUSAL>;
    {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        DeviceInfo& di = g_dev[dev];
        const int slot = (D == 128 ? 2 : 0) + (CAUSAL ? 1 : 0);
        if (!di.bwd_attr_set[slot]) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     T::kSmemBytes) != cudaSuccess)
                return ATTN_ERR_CUDA;
            di.bwd_attr_set[slot] = true;
        }
    }
    const long long prows = (long long)p.BH * p.NqPad;
    constexpr int kRowsPerBlock = 256 / (D / 8);
    if (p.deterministic) {
        if (cudaMemsetAsync(p.bound, 0, 3 * sizeof(unsigned), stream) != cudaSuccess)
            return ATTN_ERR_CUDA;
        const long long kvrows = (long long)p.BH * p.Nkv;
        attn_bwd_kv_bound_kernel<D>
            <<<(unsigned)((kvrows + kRowsPerBlock - 1) / kRowsPerBlock), 256, 0, stream>>>(p);
    }
    attn_bwd_preprocess_kernel<D>
        <<<(unsigned)((prows + kRowsPerBlock - 1) / kRowsPerBlock), 256, 0, stream>>>(p);
    const long long rows = (long long)p.BH * p.Nq;
    // key blocks along x so that the CTAs resident at one time share a few
    // heads' Q and dO tiles in L2
    dim3 grid((p.Nkv + 127) / 128, p.BH);
    kern<<<grid, T::kThreads, T::kSmemBytes, stream>>>(tq, tk, tv, tdo, p);
    attn_bwd_postprocess_kernel<D>
        <<<(unsigned)((rows * D / 8 + 255) / 256), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t check_sizes(int B, int H, long long N1, long long N2) {
    if (B < 1 || H < 1 || N1 < 1 || N2 < 1) return ATTN_ERR_INVALID_ARG;
    if (N1 > kMaxSeq || N2 > kMaxSeq) return ATTN_ERR_INVALID_ARG;
    if ((long long)B * H > (1ll << 24)) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

}  // namespace

extern "C" {

int attn_abi_version(void) { return kAbiVersion; }

const char* attn_strerror(attn_status_t s) {
    switch (s) {
        case ATTN_OK: return "ok";
        case ATTN_ERR_INVALID_ARG: return "invalid argument (null pointer or bad size)";
        case ATTN_ERR_UNSUPPORTED: return "unsupported configuration (head dim must be 64 or 128)";
        case ATTN_ERR_ALIGNMENT: return "misaligned pointer (bf16 tensors need 16 bytes, fp32 4)";
        case ATTN_ERR_CUDA: return "CUDA error while launching or running a kernel";
        case ATTN_ERR_TIMEOUT: return "a kernel pipeline wait timed out; outputs are invalid";
        case ATTN_ERR_SCRATCH_LIMIT:
            return "partials exceed the library's fixed 32 MiB decode scratch array";
        case ATTN_ERR_BAD_INDEX:
            return "a block-table entry or sequence length was out of range; those keys were skipped";
        case ATTN_ERR_INDEX_CHECK:
            return "debug build: a kernel computed an index outside its tensor; the access was skipped";
    }
    return "unknown status";
}

attn_status_t attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int H, int Nq, int Nkv, int d, int causal, float scale, void* stream) {
    if (!q || !k || !v || !o || !lse) return ATTN_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_sizes(B, H, Nq, Nkv);
    if (s != ATTN_OK) return s;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
        !aligned(lse, 4))
        return ATTN_ERR_ALIGNMENT;

    const int BH = B * H;
    CUtensorMap tq, tk, tv, to;
    // O: stored by the softmax warps as boxes of 32 rows x 64 columns
    if (!encode_bf16_map(&tq, q, BH, Nq, d) || !encode_bf16_map(&tk, k, BH, Nkv, d) ||
        !encode_bf16_map(&tv, v, BH, Nkv, d) || !encode_bf16_map(&to, o, BH, Nq, d, 32))
        return ATTN_ERR_CUDA;
    FwdParams p;
    p.o = static_cast<uint16_t*>(o);
    p.lse = lse;
    p.q_descale = p.k_descale = p.v_descale = nullptr;
    p.BH = BH;
    p.Nq = Nq;
    p.Nkv = Nkv;
    p.num_qb = (Nq + 255) / 256;
    const long long units = (long long)BH * p.num_qb;
    if (units > (1ll << 30)) return ATTN_ERR_INVALID_ARG;
    p.num_units = (int)units;
    p.scale_log2 = scale * kLog2e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 128)
        return causal ? launch_fwd<128, true>(tq, tk, tv, to, p, st)
                      : launch_fwd<128, false>(tq, tk, tv, to, p, st);
    return causal ? launch_fwd<64, true>(tq, tk, tv, to, p, st)
                  : launch_fwd<64, false>(tq, tk, tv, to, p, st);
}

attn_status_t attn_fwd_fp8(const void* q, const void* k, const void* v, const float* q_descale,
                           const float* k_descale, const float* v_descale, void* o, float* lse,
                           int B, int H, int Nq, int Nkv, int d, int causal, float scale,
                           void* stream) {
    if (!q || !k || !v || !q_descale || !k_descale || !v_descale || !o || !lse)
        return ATTN_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_sizes(B, H, Nq, Nkv);
    if (s != ATTN_OK) return s;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
        !aligned(lse, 4) || !aligned(q_descale, 4) || !aligned(k_descale, 4) ||
        !aligned(v_descale, 4))
        return ATTN_ERR_ALIGNMENT;
    const int BH = B * H;
    CUtensorMap tq, tk, tv, to;
    if (!encode_u8_map(&tq, q, BH, Nq, d) || !encode_u8_map(&tk, k, BH, Nkv, d) ||
        !encode_u8_map(&tv, v, BH, Nkv, d) || !encode_bf16_map(&to, o, BH, Nq, d, 32))
        return ATTN_ERR_CUDA;
    FwdParams p;
    p.o = static_cast<uint16_t*>(o);
    p.lse = lse;
    p.q_descale = q_descale;
    p.k_descale = k_descale;
    p.v_descale = v_descale;
    p.BH = BH;
    p.Nq = Nq;
    p.Nkv = Nkv;
    p.num_qb = (Nq + 255) / 256;
    const long long units = (long long)BH * p.num_qb;
    if (units > (1ll << 30)) return ATTN_ERR_INVALID_ARG;
    p.num_units = (int)units;
    p.scale_log2 = scale * kLog2e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 128)
        return causal ? launch_fwd<128, true, true>(tq, tk, tv, to, p, st)
                      : launch_fwd<128, false, true>(tq, tk, tv, to, p, st);
    return causal ? launch_fwd<64, true, true>(tq, tk, tv, to, p, st)
                  : launch_fwd<64, false, true>(tq, tk, tv, to, p, st);
}

attn_status_t attn_decode_partials(const void* q, const void* k, const void* v, float* o_part,
                                   float* lse_part, int B, int H, int Nkv, int d, float scale,
                                   int num_splits, void* stream) {
    if (!q || !k || !v || !o_part || !lse_part) return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_sizes(B, H, Nkv, 1);
    if (s != ATTN_OK) return s;
    if (num_splits < 1 || num_splits > 65535) return ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o_part, 4) ||
        !aligned(lse_part, 4))
        return ATTN_ERR_ALIGNMENT;
    DecodeParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.o_part = o_part;
    p.lse_part = lse_part;
    p.Nkv = Nkv;
    p.S = num_splits;
    p.L = (int)(((long long)Nkv + num_splits - 1) / num_splits);
    p.scale_log2 = scale * kLog2e;
    dim3 grid(num_splits, B * H);
    if (B * H > 65535) return ATTN_ERR_INVALID_ARG;   // grid.y limit
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.block_table = nullptr;
    p.seq_lens = nullptr;
    p.H = H;
    p.page_shift = p.max_pages = p.num_pages = 0;
    if (d == 128)
        attn_decode_partials_kernel<128, false><<<grid, DecodeTraits<128>::kThreads, 0, st>>>(p);
    else
        attn_decode_partials_kernel<64, false><<<grid, DecodeTraits<64>::kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_decode_paged_partials(const void* q, const void* k_cache, const void* v_cache,
                                         const int* block_table, const int* seq_lens,
                                         float* o_part, float* lse_part, int B, int H, int d,
                                         int page_size, int max_pages_per_seq, int num_pages,
                                         float scale, int num_splits, void* stream) {
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o_part || !lse_part)
        return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_sizes(B, H, 1, 1);
    if (s != ATTN_OK) return s;
    if (num_splits < 1 || num_splits > 65535 || B * H > 65535) return ATTN_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
        return ATTN_ERR_INVALID_ARG;
    if (max_pages_per_seq < 1 || num_pages < 1) return ATTN_ERR_INVALID_ARG;
    if ((long long)max_pages_per_seq * page_size > kMaxSeq) return ATTN_ERR_INVALID_ARG;
    if ((long long)num_pages * H * page_size * d > (1ll << 46)) return ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(o_part, 4) ||
        !aligned(lse_part, 4))
        return ATTN_ERR_ALIGNMENT;
    DecodeParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k_cache);
    p.v = static_cast<const uint16_t*>(v_cache);
    p.o_part = o_part;
    p.lse_part = lse_part;
    p.Nkv = 0;
    p.L = 0;
    p.S = num_splits;
    p.scale_log2 = scale * kLog2e;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.H = H;
    p.page_shift = 0;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages;
    dim3 grid(num_splits, B * H);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 128)
        attn_decode_partials_kernel<128, true><<<grid, DecodeTraits<128>::kThreads, 0, st>>>(p);
    else
        attn_decode_partials_kernel<64, true><<<grid, DecodeTraits<64>::kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_decode_paged(const void* q, const void* k_cache, const void* v_cache,
                                const int* block_table, const int* seq_lens, void* o, float* lse,
                                int B, int H, int d, int page_size, int max_pages_per_seq,
                                int num_pages, float scale, int num_splits, void* workspace,
                                size_t workspace_bytes, void* stream) {
    if (!workspace || !o || !lse) return ATTN_ERR_INVALID_ARG;
    const size_t need = attn_decode_workspace_bytes(B, H, d, num_splits);
    if (need == 0) {
        if (d != 64 && d != 128 && B >= 1 && H >= 1 && num_splits >= 1)
            return ATTN_ERR_UNSUPPORTED;
        return ATTN_ERR_INVALID_ARG;
    }
    if (workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
    if (!aligned(workspace, 256) || !aligned(o, 2) || !aligned(lse, 4)) return ATTN_ERR_ALIGNMENT;
    float* o_part = static_cast<float*>(workspace);
    const size_t o_bytes = ((size_t)B * H * num_splits * d * 4 + 255) / 256 * 256;
    float* lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + o_bytes);
    attn_status_t s = attn_decode_paged_partials(q, k_cache, v_cache, block_table, seq_lens,
                                                 o_part, lse_part, B, H, d, page_size,
                                                 max_pages_per_seq, num_pages, scale, num_splits,
                                                 stream);
    if (s != ATTN_OK) return s;
    return attn_lse_merge(o_part, lse_part, o, lse, B, H, num_splits, d, stream);
}

}  // extern "C"

namespace {
attn_status_t launch_merge(const float* o_part, const float* lse_part, void* o, float* lse,
                           int B, int H, int S, int R, int d, void* stream) {
    if (!o_part || !lse_part || !o || !lse) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_sizes(B, H, 1, 1);
    if (s != ATTN_OK) return s;
    if (S < 1 || S > 65535 || R < 1 || R > 65535) return ATTN_ERR_INVALID_ARG;
    if ((long long)S * R > (1ll << 24)) return ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (!aligned(o_part, 4) || !aligned(lse_part, 4) || !aligned(o, 2) || !aligned(lse, 4))
        return ATTN_ERR_ALIGNMENT;
    const int BH = B * H;
    if ((long long)BH * S * R * d >= (1ll << 46)) return ATTN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint16_t* ob = static_cast<uint16_t*>(o);
    const bool vec = aligned(o_part, 16);
    if (d == 128) {
        if (vec)
            attn_lse_merge_kernel<128, true><<<BH, kMergeThreads, 0, st>>>(o_part, lse_part, ob,
                                                                          lse, S, R, BH);
        else
            attn_lse_merge_kernel<128, false><<<BH, kMergeThreads, 0, st>>>(o_part, lse_part, ob,
                                                                           lse, S, R, BH);
    } else {
        if (vec)
            attn_lse_merge_kernel<64, true><<<BH, kMergeThreads, 0, st>>>(o_part, lse_part, ob,
                                                                         lse, S, R, BH);
        else
            attn_lse_merge_kernel<64, false><<<BH, kMergeThreads, 0, st>>>(o_part, lse_part, ob,
                                                                          lse, S, R, BH);
    }
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
}  // namespace

extern "C" {

attn_status_t attn_lse_merge(const float* o_part, const float* lse_part, void* o, float* lse,
                             int B, int H, int S, int d, void* stream) {
    return launch_merge(o_part, lse_part, o, lse, B, H, S, 1, d, stream);
}

attn_status_t attn_lse_merge_gathered(const float* o_part, const float* lse_part, void* o,
                                      float* lse, int R, int B, int H, int S, int d,
                                      void* stream) {
    return launch_merge(o_part, lse_part, o, lse, B, H, S, R, d, stream);
}

size_t attn_decode_workspace_bytes(int B, int H, int d, int num_splits) {
    if (B < 1 || H < 1 || num_splits < 1 || (d != 64 && d != 128)) return 0;
    const size_t bhs = (size_t)B * H * num_splits;
    const size_t o_bytes = (bhs * d * 4 + 255) / 256 * 256;
    const size_t l_bytes = (bhs * 4 + 255) / 256 * 256;
    return o_bytes + l_bytes;
}

attn_status_t attn_decode_splitkv(const void* q, const void* k, const void* v, void* o,
                                  float* lse, int B, int H, int Nkv, int d, float scale,
                                  int num_splits, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    if (!workspace) return ATTN_ERR_INVALID_ARG;
    const size_t need = attn_decode_workspace_bytes(B, H, d, num_splits);
    if (need == 0) {
        if (d != 64 && d != 128 && B >= 1 && H >= 1 && num_splits >= 1)
            return ATTN_ERR_UNSUPPORTED;
        return ATTN_ERR_INVALID_ARG;
    }
    if (workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return ATTN_ERR_ALIGNMENT;
    if (!o || !lse) return ATTN_ERR_INVALID_ARG;
    if (!aligned(o, 2) || !aligned(lse, 4)) return ATTN_ERR_ALIGNMENT;
    float* o_part = static_cast<float*>(workspace);
    const size_t o_bytes = ((size_t)B * H * num_splits * d * 4 + 255) / 256 * 256;
    float* lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + o_bytes);
    attn_status_t s = attn_decode_partials(q, k, v, o_part, lse_part, B, H, Nkv, d, scale,
                                           num_splits, stream);
    if (s != ATTN_OK) return s;
    return attn_lse_merge(o_part, lse_part, o, lse, B, H, num_splits, d, stream);
}

size_t attn_bwd_workspace_bytes(int B, int H, int Nq, int d) {
    if (B < 1 || H < 1 || Nq < 1 || (d != 64 && d != 128)) return 0;
    const size_t prow = (size_t)B * H * (((size_t)Nq + 63) / 64 * 64);
    return 2 * ((prow * 4 + 255) / 256 * 256) + 256 + (size_t)B * H * Nq * d * 8;
}

}  // extern "C"

namespace {
attn_status_t bwd_entry(const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                        int H, int Nq, int Nkv, int d, int causal, float scale, void* workspace,
                        size_t workspace_bytes, void* stream, bool deterministic) {
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace)
        return ATTN_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_sizes(B, H, Nq, Nkv);
    if (s != ATTN_OK) return s;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    const int BH = B * H;
    if (BH > 65535) return ATTN_ERR_INVALID_ARG;   // grid.y limit
    if ((long long)BH * Nq * d / 2048 >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
    if (workspace_bytes < attn_bwd_workspace_bytes(B, H, Nq, d)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
        !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
        !aligned(lse, 4) || !aligned(workspace, 256))
        return ATTN_ERR_ALIGNMENT;
    CUtensorMap tq, tk, tv, tdo;
    if (!encode_bf16_map(&tq, q, BH, Nq, d, 64) || !encode_bf16_map(&tk, k, BH, Nkv, d) ||
        !encode_bf16_map(&tv, v, BH, Nkv, d) || !encode_bf16_map(&tdo, dout, BH, Nq, d, 64))
        return ATTN_ERR_CUDA;
    const int NqPad = (Nq + 63) / 64 * 64;
    const size_t pbytes = ((size_t)BH * NqPad * 4 + 255) / 256 * 256;
    BwdParams p;
    p.o = static_cast<const uint16_t*>(o);
    p.dout = static_cast<const uint16_t*>(dout);
    p.lse = lse;
    p.delta = static_cast<float*>(workspace);
    p.lse2 = reinterpret_cast<float*>(static_cast<char*>(workspace) + pbytes);
    p.bound = reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + 2 * pbytes);
    p.dq_acc = static_cast<char*>(workspace) + 2 * pbytes + 256;
    p.deterministic = deterministic ? 1 : 0;
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.NqPad = NqPad;
    p.dq = static_cast<uint16_t*>(dq);
    p.dk = static_cast<uint16_t*>(dk);
    p.dv = static_cast<uint16_t*>(dv);
    p.BH = BH;
    p.Nq = Nq;
    p.Nkv = Nkv;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 128)
        return causal ? launch_bwd<128, true>(tq, tk, tv, tdo, p, st)
                      : launch_bwd<128, false>(tq, tk, tv, tdo, p, st);
    return causal ? launch_bwd<64, true>(tq, tk, tv, tdo, p, st)
                  : launch_bwd<64, false>(tq, tk, tv, tdo, p, st);
}
}  // namespace

extern "C" {

attn_status_t attn_bwd(const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                       int H, int Nq, int Nkv, int d, int causal, float scale, void* workspace,
                       size_t workspace_bytes, void* stream) {
    return bwd_entry(q, k, v, o, dout, lse, dq, dk, dv, B, H, Nq, Nkv, d, causal, scale,
                     workspace, workspace_bytes, stream, false);
}

attn_status_t attn_bwd_deterministic(const void* q, const void* k, const void* v, const void* o,
                                     const void* dout, const float* lse, void* dq, void* dk,
                                     void* dv, int B, int H, int Nq, int Nkv, int d, int causal,
                                     float scale, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    return bwd_entry(q, k, v, o, dout, lse, dq, dk, dv, B, H, Nq, Nkv, d, causal, scale,
                     workspace, workspace_bytes, stream, true);
}

attn_status_t attn_selftest_wait_timeout(unsigned limit_us, void* stream) {
    if (limit_us < 1 || limit_us > 1000000) return ATTN_ERR_INVALID_ARG;
    attn_wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
        (unsigned long long)limit_us * 1000ull);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_status(void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(st) != cudaSuccess) return ATTN_ERR_CUDA;
    unsigned word = 0;
    if (cudaMemcpyFromSymbol(&word, g_attn_status, sizeof(word)) != cudaSuccess)
        return ATTN_ERR_CUDA;
    if (word != 0) {
        const unsigned zero = 0;
        if (cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(zero)) != cudaSuccess)
            return ATTN_ERR_CUDA;
    }
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
    if (word & kDevErrTimeout) return ATTN_ERR_TIMEOUT;
    if (word & kDevErrIndexCheck) return ATTN_ERR_INDEX_CHECK;
    if (word & kDevErrBadIndex) return ATTN_ERR_BAD_INDEX;
    return ATTN_OK;
}

}  // extern "C"

// ------------------------------------------------ serving on a paged cache --
namespace {

// Checks shared by the entry points that take a paged cache's geometry.
attn_status_t check_pages(int B, int Hkv, int d, int page_size, int max_pages, int num_pages) {
    if (B < 1 || Hkv < 1 || B > (1 << 24) || Hkv > 65535) return ATTN_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
        return ATTN_ERR_INVALID_ARG;
    if (max_pages < 1 || num_pages < 1) return ATTN_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size > kMaxSeq) return ATTN_ERR_INVALID_ARG;
    // the caches' rows of pages and heads are 32-bit tensor-map coordinates
    if ((long long)num_pages * Hkv >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
    if ((long long)num_pages * Hkv * page_size * 128 > (1ll << 46)) return ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

int shift_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

int score_tiles(int max_pages) { return (max_pages + kScorePages - 1) / kScorePages; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// N = 0: 128-row tiles; else at most N rows per unit
template <int D, int N, bool SPARSE>
attn_status_t launch_paged(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const PagedParams& p, cudaStream_t stream) {
    using T = PagedTraits<D, N>;
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return ATTN_ERR_CUDA;
    void (*kern)(CUtensorMap, CUtensorMap, CUtensorMap, PagedParams);
    if constexpr (N == 0) kern = attn_paged_sm100_kernel<D, SPARSE>;
    else kern = attn_paged_rows_sm100_kernel<D, N, SPARSE>;
    int sms;
    {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        DeviceInfo& di = g_dev[dev];
        if (di.sms == 0 &&
            cudaDeviceGetAttribute(&di.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return ATTN_ERR_CUDA;
        const int slot = (N == 16 ? 4 : N == 32 ? 8 : 0) + (SPARSE ? 2 : 0) +
                         (D == 128 ? 1 : 0);
        if (!di.paged_attr_set[slot]) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     T::kSmemBytes) != cudaSuccess)
                return ATTN_ERR_CUDA;
            di.paged_attr_set[slot] = true;
        }
        sms = di.sms;
    }
    const int grid = sms < kPagedMaxCtas ? sms : kPagedMaxCtas;
    // both launches overlap what runs before them: each kernel waits for its end itself
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(T::kThreads);
    cfg.dynamicSmemBytes = T::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    constexpr int kUnitRows = N ? N : 256;
    constexpr int kBlocks = kUnitRows * D / 4 / kPagedMergeThreads;   // one pass over the rows
    cfg.gridDim = dim3(grid, kBlocks < 8 ? kBlocks : 8);
    cfg.blockDim = dim3(kPagedMergeThreads);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, attn_paged_merge_kernel<D>, p, grid) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, bool SPARSE>
attn_status_t launch_paged_rows(int rows, const CUtensorMap& tq, const CUtensorMap& tk,
                                const CUtensorMap& tv, const PagedParams& p, cudaStream_t st) {
    switch (rows) {
        case 16: return launch_paged<D, 16, SPARSE>(tq, tk, tv, p, st);
        case 32: return launch_paged<D, 32, SPARSE>(tq, tk, tv, p, st);
    }
    return launch_paged<D, 0, SPARSE>(tq, tk, tv, p, st);
}

// attn_fwd_paged, and attn_sparse_paged (sel not null)
attn_status_t paged_entry(const void* q, const void* k_cache, const void* v_cache,
                          const int* block_table, const int* cu_q, const int* seq_lens,
                          const int* sel, int K, void* o, float* lse, int B, int T, int Hq,
                          int Hkv, int d, long long q_stride, int page_size, int max_pages,
                          int num_pages, int causal, float scale, void* workspace,
                          size_t workspace_bytes, void* stream) {
    if (!q || !k_cache || !v_cache || !block_table || !cu_q || !seq_lens || !o || !lse ||
        !workspace)
        return ATTN_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_pages(B, Hkv, d, page_size, max_pages, num_pages);
    if (s != ATTN_OK) return s;
    if (T < 1 || T > (1 << 30) || Hq < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    const int G = Hq / Hkv;
    if (G > 128) return ATTN_ERR_UNSUPPORTED;
    if (q_stride < (long long)Hq * d || q_stride > (1ll << 36)) return ATTN_ERR_INVALID_ARG;
    if (sel) {
        if (K < 1) return ATTN_ERR_INVALID_ARG;
        const int runs = page_size > 128 ? page_size / 128 : 1;   // list entries of a page
        if ((long long)K * runs > kPagedListMax) return ATTN_ERR_UNSUPPORTED;
        if (!aligned(sel, 4)) return ATTN_ERR_ALIGNMENT;
    }
    if (workspace_bytes < attn_fwd_paged_workspace_bytes(d)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) ||
        !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(cu_q, 4) ||
        !aligned(seq_lens, 4) || !aligned(workspace, 256) || q_stride % 8 != 0)
        return ATTN_ERR_ALIGNMENT;

    PagedParams p;
    // Rows of a unit: with few tokens per sequence the turned kernel, whose work follows the rows
    // in use, else 128-row tiles. One form for the whole call, by the average, as the lengths are
    // on the device. 16 columns / 32 / 128-row tiles, 16 sequences of 4,000 keys, 32 heads on 8:
    // 4 rows 54.4 / 53.3 / 58.4 us, 32 rows 92.8 / 55.9 / 60.6, 64 rows 168 / 94 / 64, 128 rows
    // 292 / 170 / 72; 7 drafts of 42 rows: - / 24.9 / 25.0. (So from 33 rows on 128-row tiles are as
    // fast or faster; and sequences far from the average pay: 256 that decode at 2,048 keys and a
    // chunk of 512 tokens behind 8,000 take 610 us in one call, 331 and 100 apart.)
    const long long avg = sel ? 1 : (T + (long long)B - 1) / B;
    const int rows = avg * G <= 16 ? 16 : G <= 32 && avg * G <= 64 ? 32 : 0;
    p.tpt = sel ? 1 : (rows ? rows : 128) / G;
    p.unit_tok = sel || rows ? p.tpt : 2 * p.tpt;
    const int box = page_size < 128 ? page_size : 128;
    CUtensorMap tq, tk, tv;
    if (!encode_q_map(&tq, q, T, Hq, d, q_stride, G, p.tpt) ||
        !encode_bf16_map(&tk, k_cache, num_pages * Hkv, page_size, d, box) ||
        !encode_bf16_map(&tv, v_cache, num_pages * Hkv, page_size, d, box))
        return ATTN_ERR_CUDA;
    char* ws = static_cast<char*>(workspace);
    p.o = static_cast<uint16_t*>(o);
    p.lse = lse;
    p.block_table = block_table;
    p.cu_q = cu_q;
    p.seq_lens = seq_lens;
    p.sel = sel;
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_lse = reinterpret_cast<float*>(ws + (size_t)512 * kPagedMaxCtas * d * 4);
    p.pieces = reinterpret_cast<PagedPiece*>(ws + (size_t)512 * kPagedMaxCtas * (d + 1) * 4);
    p.B = B;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = G;
    p.K = K;
    p.page_shift = shift_of(page_size);
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.causal = causal;
    p.scale_log2 = scale * kLog2e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 128)
        return sel ? launch_paged_rows<128, true>(rows, tq, tk, tv, p, st)
                   : launch_paged_rows<128, false>(rows, tq, tk, tv, p, st);
    return sel ? launch_paged_rows<64, true>(rows, tq, tk, tv, p, st)
               : launch_paged_rows<64, false>(rows, tq, tk, tv, p, st);
}

}  // namespace

extern "C" {

attn_status_t attn_page_tables(const int* ctx_lens, const int* new_lens, const int* free_pages,
                               const int* free_head, int* free_head_out, int* block_table,
                               int* seq_lens, int* cu_q, long long* slot_map, int B, int T,
                               int num_free, int page_size, int max_pages_per_seq, int num_pages,
                               void* stream) {
    if (!ctx_lens || !new_lens || !free_pages || !free_head || !free_head_out || !block_table ||
        !seq_lens || !cu_q || !slot_map)
        return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_pages(B, 1, 64, page_size, max_pages_per_seq, num_pages);
    if (s != ATTN_OK) return s;
    if (T < 1 || T > (1 << 30) || num_free < 1) return ATTN_ERR_INVALID_ARG;
    if (B > kTablesMaxSeqs) return ATTN_ERR_UNSUPPORTED;
    if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) ||
        !aligned(free_head, 4) || !aligned(free_head_out, 4) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(slot_map, 8))
        return ATTN_ERR_ALIGNMENT;
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return ATTN_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kTablesThreads);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int ctas;
    {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        DeviceInfo& di = g_dev[dev];
        if (!di.tables_attr_set) {
            if (cudaFuncSetAttribute(attn_page_tables_kernel,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (3 * kTablesMaxSeqs + 1) * 4) != cudaSuccess ||
                cudaFuncSetAttribute(attn_page_tables_kernel,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed,
                                     1) != cudaSuccess)
                return ATTN_ERR_CUDA;
            // whether this process has room for a cluster of 16 (an answer of no, or none: 8 will do)
            cfg.gridDim = dim3(16);
            cfg.dynamicSmemBytes = (3 * kTablesMaxSeqs + 1) * 4;
            attr[0].val.clusterDim.x = 16;
            int fit = 0;
            if (cudaOccupancyMaxActiveClusters(&fit, attn_page_tables_kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                fit = 0;
            }
            di.tables_sixteen = fit > 0;
            di.tables_attr_set = true;
        }
        ctas = tables_ctas(T, kTablesThreads, di.tables_sixteen);
    }
    TablesParams p{ctx_lens, new_lens,  free_pages, free_head, free_head_out,
                   block_table, seq_lens, cu_q,     slot_map,  B,
                   T,        num_free,  shift_of(page_size), max_pages_per_seq, num_pages};
    cfg.gridDim = dim3(ctas);
    cfg.dynamicSmemBytes = (size_t)(3 * B + 1) * 4;
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].val.clusterDim.x = ctas;
    if (cudaLaunchKernelEx(&cfg, attn_page_tables_kernel, p) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return ATTN_OK;
}

attn_status_t attn_paged_append(const void* k, const void* v, const long long* slot_map,
                                void* k_cache, void* v_cache, void* k_bounds, int T, int Hkv,
                                int d, long long kv_stride, int page_size, int num_pages,
                                void* stream) {
    if (!k || !v || !slot_map || !k_cache || !v_cache) return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_pages(1, Hkv, d, page_size, 1, num_pages);
    if (s != ATTN_OK) return s;
    if (T < 1 || T > (1 << 30)) return ATTN_ERR_INVALID_ARG;
    if (kv_stride < (long long)Hkv * d || kv_stride > (1ll << 36)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        (k_bounds && !aligned(k_bounds, 16)) || !aligned(slot_map, 8) || kv_stride % 8 != 0)
        return ATTN_ERR_ALIGNMENT;
    AppendParams p;
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.slot_map = slot_map;
    p.k_cache = static_cast<uint16_t*>(k_cache);
    p.v_cache = static_cast<uint16_t*>(v_cache);
    p.bounds = static_cast<uint16_t*>(k_bounds);
    p.kv_stride = kv_stride;
    p.num_slots = (long long)num_pages * page_size;
    p.T = T;
    p.Hkv = Hkv;
    p.page_shift = shift_of(page_size);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Rows of a block. 32 of them share a block's launch and copy together, but the pages that end
    // among them are taken one after another; one row a block spreads those. The host does not
    // know how many rows share a page, so small calls are taken for decode (every row ends its
    // page) and large ones for prompts. One row / 32, 8 heads of 128: decode 16 rows 3.8 / 20.6
    // us, 256 rows 10.7 / 47, 1,024 rows 41 / 74; consecutive rows 128: 4.6 / 4.2, 1,024: 12.5 /
    // 4.8, 4,095: 31.6 / 6.8, 4,096: 41.9 / 9.6.
    const bool many = (long long)T * Hkv >= 32768;
    const dim3 grid(many ? (T + 31) / 32 : T, Hkv);
    if (d == 128) {
        if (many) attn_paged_append_kernel<128, 32><<<grid, kAppendThreads, 0, st>>>(p);
        else attn_paged_append_kernel<128, 1><<<grid, kAppendThreads, 0, st>>>(p);
    } else {
        if (many) attn_paged_append_kernel<64, 32><<<grid, kAppendThreads, 0, st>>>(p);
        else attn_paged_append_kernel<64, 1><<<grid, kAppendThreads, 0, st>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

size_t attn_fwd_paged_workspace_bytes(int d) {
    if (d != 64 && d != 128) return 0;
    return (size_t)512 * kPagedMaxCtas * (d + 1) * 4 + round256(2 * kPagedMaxCtas * sizeof(PagedPiece));
}

attn_status_t attn_fwd_paged(const void* q, const void* k_cache, const void* v_cache,
                             const int* block_table, const int* cu_q, const int* seq_lens, void* o,
                             float* lse, int B, int T, int Hq, int Hkv, int d, long long q_stride,
                             int page_size, int max_pages_per_seq, int num_pages, int causal,
                             float scale, void* workspace, size_t workspace_bytes, void* stream) {
    return paged_entry(q, k_cache, v_cache, block_table, cu_q, seq_lens, nullptr, 0, o, lse, B, T,
                       Hq, Hkv, d, q_stride, page_size, max_pages_per_seq, num_pages, causal,
                       scale, workspace, workspace_bytes, stream);
}

attn_status_t attn_sparse_paged(const void* q, const void* k_cache, const void* v_cache,
                                const int* block_table, const int* cu_q, const int* seq_lens,
                                const int* sel, void* o, float* lse, int B, int T, int Hq, int Hkv,
                                int d, int num_sel, long long q_stride, int page_size,
                                int max_pages_per_seq, int num_pages, float scale, void* workspace,
                                size_t workspace_bytes, void* stream) {
    if (!sel) return ATTN_ERR_INVALID_ARG;
    return paged_entry(q, k_cache, v_cache, block_table, cu_q, seq_lens, sel, num_sel, o, lse, B,
                       T, Hq, Hkv, d, q_stride, page_size, max_pages_per_seq, num_pages, 1, scale,
                       workspace, workspace_bytes, stream);
}

size_t attn_page_select_workspace_bytes(int T, int Hkv, int max_pages_per_seq) {
    if (T < 1 || Hkv < 1 || max_pages_per_seq < 1) return 0;
    const size_t rows = (size_t)T * Hkv;
    return round256(rows * max_pages_per_seq * 8) + round256(rows * score_tiles(max_pages_per_seq) * 4);
}

}  // extern "C"

namespace {
template <int D, int THREADS, int PER>
bool launch_topk(const SelectParams& p, cudaStream_t st) {
    const long long rows = (long long)p.T * p.Hkv, groups = THREADS == 32 ? 4 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + groups - 1) / groups));
    cfg.blockDim = dim3(THREADS == 32 ? 128 : THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_page_topk_kernel<D, THREADS, PER>, p) == cudaSuccess;
}

template <int D, int ROWS>
bool launch_score(const SelectParams& p, cudaStream_t st) {
    constexpr int kSmem = kScoreABytes<D, ROWS> + kScorePages * 4 * D;
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return false;
    {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        bool& set = g_dev[dev].score_attr_set[(D == 128 ? 1 : 0) + (ROWS == 64 ? 2 : 0)];
        if (!set) {
            if (cudaFuncSetAttribute(attn_page_score_kernel<D, ROWS>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSmem) != cudaSuccess)
                return false;
            set = true;
        }
    }
    const dim3 grid((unsigned)((long long)p.tiles * ((p.T + p.tile_tok - 1) / p.tile_tok)), p.Hkv);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kScoreThreads<ROWS>);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_page_score_kernel<D, ROWS>, p) == cudaSuccess;
}

template <int D>
attn_status_t launch_select(const SelectParams& p, cudaStream_t st) {
    if (!(p.tile_tok * p.G <= 16 ? launch_score<D, 16>(p, st) : launch_score<D, 64>(p, st))) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    // the fewest threads per row whose registers hold its keys
    const bool ok = p.max_pages <= 32 * 8      ? launch_topk<D, 32, 8>(p, st)
                    // few rows: more threads for each, or the row's own steps set the time
                    : p.max_pages <= 32 * 32   ? ((long long)p.T * p.Hkv <= 1024
                                                      ? launch_topk<D, 128, 8>(p, st)
                                                      : launch_topk<D, 32, 32>(p, st))
                    : p.max_pages <= 256 * 16  ? launch_topk<D, 256, 16>(p, st)
                                               : launch_topk<D, 1024, 16>(p, st);
    if (!ok) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
}  // namespace

extern "C" {

attn_status_t attn_page_select(const void* q, const void* k_bounds, const int* block_table,
                               const int* cu_q, const int* seq_lens, int* sel, int B, int T,
                               int Hq, int Hkv, int d, int num_sel, int keep_first, int keep_last,
                               long long q_stride, int page_size, int max_pages_per_seq,
                               int num_pages, void* workspace, size_t workspace_bytes,
                               void* stream) {
    if (!q || !k_bounds || !block_table || !cu_q || !seq_lens || !sel || !workspace)
        return ATTN_ERR_INVALID_ARG;
    attn_status_t s = check_pages(B, Hkv, d, page_size, max_pages_per_seq, num_pages);
    if (s != ATTN_OK) return s;
    if (T < 1 || T > (1 << 30) || Hq < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if (num_sel < 1 || keep_first < 0 || keep_last < 0 ||
        (long long)keep_first + keep_last > num_sel)
        return ATTN_ERR_INVALID_ARG;
    if (Hq / Hkv > 128 || max_pages_per_seq > 16384) return ATTN_ERR_UNSUPPORTED;
    // rows and blocks are counted in 32 bits
    if ((long long)T * Hkv > (1ll << 30) || (long long)T * score_tiles(max_pages_per_seq) > (1ll << 30))
        return ATTN_ERR_INVALID_ARG;
    if (q_stride < (long long)Hq * d || q_stride > (1ll << 36)) return ATTN_ERR_INVALID_ARG;
    if (workspace_bytes < attn_page_select_workspace_bytes(T, Hkv, max_pages_per_seq))
        return ATTN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_bounds, 16) || !aligned(block_table, 4) ||
        !aligned(cu_q, 4) || !aligned(seq_lens, 4) || !aligned(sel, 4) ||
        !aligned(workspace, 256) || q_stride % 8 != 0)
        return ATTN_ERR_ALIGNMENT;
    SelectParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.bounds = static_cast<const uint16_t*>(k_bounds);
    p.block_table = block_table;
    p.cu_q = cu_q;
    p.seq_lens = seq_lens;
    p.sel = sel;
    p.keys = static_cast<unsigned long long*>(workspace);
    p.err = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                     round256((size_t)T * Hkv * max_pages_per_seq * 8));
    p.tiles = score_tiles(max_pages_per_seq);
    // 64 tokens share a tile's read of the bounds (the choice for 1,098 tokens: 56 us; 48, 32 or 16
    // tokens: 61, 58, 62), one sequence after another; where sequences have a token or two, one (its
    // pages are its own). 1 token / 64, 16 sequences of 512 pages: 1 token each 23 / 78 us, 2: 32 /
    // 80, 4: 49 / 81, 8: 84 / 54; 64 sequences of 125 pages: 1: 25 / 279, 4: 48 / 85; one
    // sequence of 256 tokens and 250 pages: 75 / 33.5
    p.tile_tok = (long long)T <= 2ll * B ? 1 : 64;
    p.q_stride = q_stride;
    p.B = B;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.K = num_sel;
    p.first = keep_first;
    p.last = keep_last;
    p.page_shift = shift_of(page_size);
    p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return d == 128 ? launch_select<128>(p, st) : launch_select<64>(p, st);
}

}  // extern "C"
