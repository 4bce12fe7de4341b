// attn_api.cu -- the C ABI: argument checks, per-device state, tensor-map
// encoding, dispatch to the kernels, status reporting, and the host-side
// scheduling exports declared in attn.h.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <numeric>
#include <vector>

#include "bias.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "fwd_sched.h"

namespace gb300 {

// The library's device error word (one per device/context).  Kernels OR
// error bits into it; attn_last_device_error() reads and clears it.
__device__ unsigned int g_attn_error_word;

namespace {

constexpr int kMaxDevices = 64;
constexpr long long kMaxLen = 1ll << 24;
constexpr long long kMaxHeads = 1ll << 24;
constexpr int kMaxBiasSpan = 1 << 16;   // distances of a bias map, and buckets
constexpr long long kMaxBiasTiles = 1ll << 30;  // key tiles whose sums a table's gradient adds up
constexpr int kMaxPackedRows = 1 << 30;  // rows of a packed batch (ragged maps, fwd_sched.h)

struct DevState {
    bool ready;
    int num_sms;
    unsigned int* err_word;
};

std::mutex g_mu;
DevState g_dev[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

attn_status_t current_device_info(DeviceInfo* out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(g_mu);
    DevState& s = g_dev[dev];
    if (!s.ready) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return ATTN_ERR_CUDA;
        if (major != 10 || minor != 3) return ATTN_ERR_UNSUPPORTED;  // built for sm_103a only
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_attn_error_word) != cudaSuccess) return ATTN_ERR_CUDA;
        s.num_sms = sms;
        s.err_word = static_cast<unsigned int*>(p);
        s.ready = true;
    }
    out->device = dev;
    out->num_sms = s.num_sms;
    out->err_word = s.err_word;
    return ATTN_OK;
}

static bool load_encoder() {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !fn)
            return false;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    return true;
}

attn_status_t encode_tmap_out_3d(CUtensorMap* map, void* base, bool f32, int d, int rows,
                                 long long heads, int box_cols, int box_rows) {
    if (!load_encoder()) return ATTN_ERR_CUDA;
    const cuuint64_t es = f32 ? 4 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)d * es, (cuuint64_t)d * es * (cuuint64_t)rows};
    cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1u};
    cuuint32_t elem[3] = {1u, 1u, 1u};
    CUresult r = g_encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          3, base, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t encode_tmap_paged_kv(CUtensorMap* map, const void* base, int d, int Hkv,
                                   int page_size, long long num_blocks) {
    if (!load_encoder()) return ATTN_ERR_CUDA;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)Hkv, (cuuint64_t)page_size, (cuuint64_t)num_blocks};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)Hkv * d * 2,
                             (cuuint64_t)page_size * Hkv * d * 2};
    cuuint32_t box[4] = {64u, 1u, 64u, 1u};
    cuuint32_t elem[4] = {1u, 1u, 1u, 1u};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                          strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t encode_tmap_pages(CUtensorMap* map, const void* base, bool e4m3, int d, int Hkv,
                                int page_size, long long num_blocks, int box_keys) {
    if (!load_encoder()) return ATTN_ERR_CUDA;
    const cuuint64_t es = e4m3 ? 1 : 2;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)Hkv, (cuuint64_t)page_size, (cuuint64_t)num_blocks};
    cuuint64_t strides[3] = {(cuuint64_t)d * es, (cuuint64_t)Hkv * d * es,
                             (cuuint64_t)page_size * Hkv * d * es};
    cuuint32_t box[4] = {(cuuint32_t)(128 / es), 1u, (cuuint32_t)box_keys, 1u};
    cuuint32_t elem[4] = {1u, 1u, 1u, 1u};
    // a key's row of one head is d * es bytes, its neighbour another head's, which
    // another CTA reads at another time: 256-byte L2 fetches of 128-byte rows are
    // half wasted (decode over 8 heads of 128 codes: 4442 -> 5251 GB/s)
    CUresult r = g_encode(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                          const_cast<void*>(base), dims, strides, box, elem,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          (long long)d * (long long)es < 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                             : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t encode_tmap_f32_sw128_3d(CUtensorMap* map, void* base, int d, int rows,
                                       long long heads, int box_rows) {
    if (!load_encoder()) return ATTN_ERR_CUDA;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)d * 4, (cuuint64_t)d * 4 * (cuuint64_t)rows};
    cuuint32_t box[3] = {32u, (cuuint32_t)box_rows, 1u};
    cuuint32_t elem[3] = {1u, 1u, 1u};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, elem,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// Bytes below a packed array at which its map begins.  Rows outside a sequence are filled
// with zeros, but for these maps (not for dense ones) the hardware looks at memory that lies
// 64 to 128 KB past the map's base: a shorter array that begins near the end of its 2 MB
// block (the unit in which device memory is mapped) gets a map that begins 256 KB lower,
// and its columns start that far on.  (A 9 KB array 25 KB before the end of what was mapped
// gave an invalid access.  The reach is an observation, on pages of host memory that
// became resident: the same for rows of 16 bytes to 512 KB, head dims 8 to 256, boxes of 64 and
// 128 rows of bf16, sequences of 0 to 500 rows; never for the stores of gradients, bf16 or
// fp32.  256 KB is twice what was seen.)
static uintptr_t packed_map_shift(uintptr_t at, long long rows, size_t row_bytes) {
    constexpr uintptr_t kReach = 256 << 10, kBlock = 2 << 20;
    return (unsigned long long)rows * row_bytes < kReach && at % kBlock > kBlock - kReach ? kReach : 0;
}

attn_status_t encode_tmap_ragged(CUtensorMap* map, int* col, const void* base, int rows, bool f32, int d,
                                 int heads, int box_cols, int box_rows, bool swizzle128) {
    if (!load_encoder()) return ATTN_ERR_CUDA;
    const cuuint64_t es = f32 ? 4 : 2;
    const cuuint64_t rs = (cuuint64_t)heads * d * es;  // row stride (bytes)
    if (rs >= (1ull << 34)) return ATTN_ERR_UNSUPPORTED;
    const uintptr_t at = reinterpret_cast<uintptr_t>(base);
    const uintptr_t lower = packed_map_shift(at, rows, rs);
    *col = (int)(lower / es);
    cuuint64_t dims[5] = {(cuuint64_t)(d + *col), (cuuint64_t)heads, (cuuint64_t)kRaggedWindow,
                          (cuuint64_t)kRaggedOuterExtent, (cuuint64_t)kRaggedOuterExtent};
    cuuint64_t strides[4] = {(cuuint64_t)d * es, rs, rs, (1ull << 34) - rs};
    cuuint32_t box[5] = {(cuuint32_t)box_cols, 1u, (cuuint32_t)box_rows, 1u, 1u};
    cuuint32_t elem[5] = {1u, 1u, 1u, 1u, 1u};
    CUresult r = g_encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          5, reinterpret_cast<void*>(at - lower), dims, strides, box, elem,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                          swizzle128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t encode_tmap_u8_3d(CUtensorMap* map, const void* base, int inner, long long pitch,
                                int rows, long long heads, int box_inner, int box_rows) {
    if (!load_encoder()) return ATTN_ERR_CUDA;
    cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)pitch * (cuuint64_t)rows};
    cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows, 1u};
    cuuint32_t elem[3] = {1u, 1u, 1u};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims,
                          strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t encode_tmap_bf16_3d(CUtensorMap* map, const void* base, int d, int rows,
                                  long long heads, int box_rows) {
    if (!load_encoder()) return ATTN_ERR_CUDA;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * (cuuint64_t)rows};
    cuuint32_t box[3] = {64u, (cuuint32_t)box_rows, 1u};
    cuuint32_t elem[3] = {1u, 1u, 1u};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                          strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// Diagnostic of the kernels' bounded waits: warp 0 waits, with the same
// mbar_wait every kernel uses, on an mbarrier that nothing ever arrives on.
// mode 0: the wait runs out its time limit; the kernel then ORs kErrTimeout
// into the error word as the real kernels do.  mode 1: warp 1 raises the CTA's
// abort flag after about a millisecond and the wait must return early.
// result: 1 = left through the abort flag, 2 = ran out of time, 3 = the phase
// completed (impossible).
__global__ void attn_selftest_wait_kernel(int mode, int* result, unsigned int* err) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        const uint64_t t0 = global_timer_ns();
        const bool ok = mbar_wait(smem_u32(&bar), 0, (const volatile int*)&abort_flag);
        const uint64_t waited = global_timer_ns() - t0;
        if (threadIdx.x == 0) {
            if (ok) {
                *result = 3;
            } else if (waited > kWaitLimitNs) {
                *result = 2;
                atomicOr(err, kErrTimeout);
            } else {
                *result = 1;
            }
        }
    } else if (warp == 1 && mode == 1 && threadIdx.x == 32) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
        *((volatile int*)&abort_flag) = 1;
    }
}

}  // namespace gb300

using namespace gb300;

namespace {

attn_status_t check_common(int B, int Hq, int Hkv, int d, float scale, attn_out_dtype_t o_dtype) {
    if (B < 1 || Hq < 1 || Hkv < 1 || d < 1) return ATTN_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if ((long long)B * Hq > kMaxHeads || (long long)B * Hkv > kMaxHeads) return ATTN_ERR_INVALID_ARG;
    if (!(scale >= 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    if (o_dtype != ATTN_OUT_BF16 && o_dtype != ATTN_OUT_F32) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

attn_status_t check_fwd(const void* q, const void* k, const void* v, const void* o,
                        const float* lse, int B, int Hq, int Hkv, int Nq, int Nk, int d,
                        int causal, float scale, attn_out_dtype_t o_dtype) {
    if (!q || !k || !v || !o) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
    if (lse && !aligned4(lse)) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_common(B, Hq, Hkv, d, scale, o_dtype);
    if (st != ATTN_OK) return st;
    if (Nq < 1 || Nk < 1 || Nq > kMaxLen || Nk > kMaxLen) return ATTN_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if (causal && Nq > Nk) return ATTN_ERR_INVALID_ARG;
    if (!fwd_head_dim_supported(d)) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

attn_status_t check_decode_shape(int B, int Hq, int Hkv, int Nmax, int d, int num_splits) {
    if (B < 1 || Hq < 1 || Hkv < 1 || d < 1) return ATTN_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if ((long long)B * Hq > kMaxHeads || (long long)B * Hkv > kMaxHeads) return ATTN_ERR_INVALID_ARG;
    if (Nmax < 1 || Nmax > kMaxLen) return ATTN_ERR_INVALID_ARG;
    if (num_splits < 0) return ATTN_ERR_INVALID_ARG;
    if (!decode_head_dim_supported(d)) return ATTN_ERR_UNSUPPORTED;
    if (Hq / Hkv > 16) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

}  // namespace

// Pointer, shape and value checks of a contiguous-cache decode call (no device
// is touched), shared by attn_decode and attn_decode_noalloc.
attn_status_t gb300::check_decode_call(const void* q, const void* k_cache, const void* v_cache,
                                       const int* seqlens, const void* o, const float* lse, int B,
                                       int Hq, int Hkv, int Nmax, int d, float scale,
                                       int num_splits, attn_out_dtype_t o_dtype) {
    if (!q || !k_cache || !v_cache || !seqlens || !o) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
        !aligned4(seqlens))
        return ATTN_ERR_INVALID_ARG;
    if (lse && !aligned4(lse)) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_common(B, Hq, Hkv, d, scale, o_dtype);
    if (st != ATTN_OK) return st;
    return check_decode_shape(B, Hq, Hkv, Nmax, d, num_splits);
}

namespace {

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// A contiguous [B, H, N, d] array's strides, for callers that pass none.
struct Strides {
    long long s[3];
    Strides(const long long* given, int H, int N, int d) {
        s[0] = given ? given[0] : (long long)H * N * d;
        s[1] = given ? given[1] : (long long)N * d;
        s[2] = given ? given[2] : d;
    }
};

// Strides {batch, head, token} (elements) of a [B, H, N, d] view whose rows are
// 16-byte aligned; `written`: no two elements may share a place.
bool strides_ok(const long long* s, int B, int H, int N, int d, int element_bytes, bool written) {
    const int sizes[3] = {B, H, N};
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] % (16 / element_bytes) != 0) return false;
    if (!written) return true;
    // from the smallest stride up, each has to clear what the ones below span
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int x, int y) { return s[x] < s[y]; });
    long long span = d;
    for (int i : order) {
        if (sizes[i] == 1) continue;
        if (s[i] < span) return false;
        span += s[i] * (sizes[i] - 1);
    }
    return true;
}

// Shape checks shared by the paged-cache entry points.
attn_status_t check_pages(int Hkv, int d, long long num_blocks, int page_size,
                          attn_cache_dtype_t cache_dtype, const void* k_pages, const void* v_pages,
                          const float* k_descale, const float* v_descale) {
    if (cache_dtype != ATTN_CACHE_BF16 && cache_dtype != ATTN_CACHE_E4M3) return ATTN_ERR_INVALID_ARG;
    if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages)) return ATTN_ERR_INVALID_ARG;
    const bool e4m3 = cache_dtype == ATTN_CACHE_E4M3;
    if (e4m3 && (!k_descale || !v_descale || !aligned16(k_descale) || !aligned16(v_descale)))
        return ATTN_ERR_INVALID_ARG;
    if (Hkv < 1 || d < 1 || num_blocks < 1 || page_size < 1) return ATTN_ERR_INVALID_ARG;
    if (num_blocks > (1ll << 31) - 1 || page_size > kMaxLen || Hkv > kMaxHeads) return ATTN_ERR_INVALID_ARG;
    if (!fwd_head_dim_supported(d) || (e4m3 && d % 16 != 0)) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

attn_status_t check_tree_shape(int B, int Hq, int Hkv, int T, int max_blocks, int page_size, int d,
                               attn_cache_dtype_t cache_dtype) {
    if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || max_blocks < 1 || page_size < 1 || d < 1)
        return ATTN_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || (long long)B * Hq > kMaxHeads) return ATTN_ERR_INVALID_ARG;
    if (cache_dtype != ATTN_CACHE_BF16 && cache_dtype != ATTN_CACHE_E4M3) return ATTN_ERR_INVALID_ARG;
    if ((long long)max_blocks * page_size > kMaxLen) return ATTN_ERR_INVALID_ARG;
    if (T > 1024 || page_size % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    // (rows of a head group, and rows in all, are counted in 32 bits)
    if ((long long)T * (Hq / Hkv) > (1ll << 20) || (long long)B * Hq * T > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
    if (!fwd_head_dim_supported(d) || (cache_dtype == ATTN_CACHE_E4M3 && d % 16 != 0))
        return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// Packed batches: the offsets' pointers and the row counts.
attn_status_t check_varlen(const int* cu_q, const int* cu_k, int total_q, int total_k, int max_q, int max_k) {
    if (!cu_q || !cu_k || !aligned4(cu_q) || !aligned4(cu_k)) return ATTN_ERR_INVALID_ARG;
    if (total_q < 1 || total_k < 1 || total_q > kMaxPackedRows || total_k > kMaxPackedRows)
        return ATTN_ERR_INVALID_ARG;
    if (max_q > total_q || max_k > total_k) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

// A backward's further arrays.
attn_status_t check_grads(const void* dout, const float* lse, const void* dq, const void* dk, const void* dv,
                          attn_out_dtype_t grad_dtype) {
    if (!dout || !lse || !dq || !dk || !dv) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv)) return ATTN_ERR_INVALID_ARG;
    if (grad_dtype != ATTN_OUT_BF16 && grad_dtype != ATTN_OUT_F32) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

attn_status_t check_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                                 const int* seqlens, const void* o, const float* lse, int B, int Hq, int Hkv,
                                 long long num_blocks, int page_size, int max_blocks, int d, float scale,
                                 int num_splits, attn_out_dtype_t o_dtype) {
    if (!q || !k_pages || !v_pages || !block_table || !seqlens || !o) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) ||
        !aligned4(seqlens) || !aligned4(block_table))
        return ATTN_ERR_INVALID_ARG;
    if (lse && !aligned4(lse)) return ATTN_ERR_INVALID_ARG;
    if (num_blocks < 1 || max_blocks < 1 || page_size < 64) return ATTN_ERR_INVALID_ARG;
    if (page_size % 64 != 0) return ATTN_ERR_UNSUPPORTED;
    if ((long long)max_blocks * page_size > kMaxLen || num_blocks >= (1ll << 31))
        return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_common(B, Hq, Hkv, d, scale, o_dtype);
    if (st != ATTN_OK) return st;
    return check_decode_shape(B, Hq, Hkv, max_blocks * page_size, d, num_splits);
}

attn_status_t check_page_tables(const int* pool, int num_blocks, const int* block_table, const int* seqlens,
                                const int* lens, int B, int max_blocks, int page_size) {
    if (!pool || !block_table || !seqlens || !lens) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(pool) || !aligned4(block_table) || !aligned4(seqlens) || !aligned4(lens))
        return ATTN_ERR_INVALID_ARG;
    if (B < 1 || max_blocks < 1 || page_size < 1 || num_blocks < 1) return ATTN_ERR_INVALID_ARG;
    if ((long long)max_blocks * page_size > kMaxLen) return ATTN_ERR_INVALID_ARG;
    if (num_blocks > kMaxPackedRows) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// A relative position bias: what the host can see of it (the buckets live on the
// device, where each is checked as it is read), and the kernels' limits.
attn_status_t check_bias(const void* table, attn_out_dtype_t table_dtype, const int* buckets, int first,
                         int span, int num_buckets, int d) {
    if (!table || !buckets || !aligned4(buckets)) return ATTN_ERR_INVALID_ARG;
    if (table_dtype != ATTN_OUT_BF16 && table_dtype != ATTN_OUT_F32) return ATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(table) % (table_dtype == ATTN_OUT_F32 ? 4 : 2) != 0) return ATTN_ERR_INVALID_ARG;
    if (span < 1 || num_buckets < 1 || first < -kMaxLen || first > kMaxLen) return ATTN_ERR_INVALID_ARG;
    if (span > kMaxBiasSpan || num_buckets > kMaxBiasSpan || !head_dim_supported(d)) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// Whether a backward's key tiles (the longest sequence's for each of a packed batch) are
// too many for its sums' index arithmetic.
bool too_many_bias_tiles(int B, int Nk) { return (long long)B * ((Nk + 127) / 128) > kMaxBiasTiles; }

BiasArgs bias_args(const void* table, attn_out_dtype_t table_dtype, const int* buckets, int first, int span,
                   int num_buckets) {
    return BiasArgs{table, buckets, first, span, num_buckets, table_dtype == ATTN_OUT_BF16};
}

// base^n and products of such, exactly: whether r^s e^k >= D^k e^s.
bool bucket_reached(long long r, int s, long long e, int k, long long D) {
    auto times = [](std::vector<uint32_t>& x, long long by, int n) {
        for (; n > 0; --n) {
            uint64_t carry = 0;
            for (uint32_t& w : x) {
                carry += (uint64_t)w * (uint64_t)by;
                w = (uint32_t)carry;
                carry >>= 32;
            }
            if (carry) x.push_back((uint32_t)carry);
        }
    };
    std::vector<uint32_t> a{1}, b{1};
    times(a, r, s);
    times(a, e, k);
    times(b, D, k);
    times(b, e, s);
    if (a.size() != b.size()) return a.size() > b.size();
    return !std::lexicographical_compare(a.rbegin(), a.rend(), b.rbegin(), b.rend());
}

// SM count of the current device, for the size queries (the launches read the
// same per-device value).  -1 when no device can be queried.
int current_num_sms(int* sms) {
    DeviceInfo dev;
    if (current_device_info(&dev) == ATTN_OK) {
        *sms = dev.num_sms;
        return 0;
    }
    return -1;
}

}  // namespace

extern "C" {

size_t attn_fwd_workspace_size(int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal) {
    if (check_common(B, Hq, Hkv, d, 1.0f, ATTN_OUT_BF16) != ATTN_OK) return 0;
    if (Nq < 1 || Nk < 1 || Nq > kMaxLen || Nk > kMaxLen) return 0;
    if ((causal != 0 && causal != 1) || (causal && Nq > Nk)) return 0;
    if (!fwd_head_dim_supported(d)) return 0;
    int sms = 0;
    if (current_num_sms(&sms) != 0) return 0;
    return fwd_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, causal, sms);
}

attn_status_t attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int Hq, int Hkv, int Nq, int Nk, int d, int causal, float scale,
                       attn_out_dtype_t o_dtype, void* workspace, size_t workspace_bytes,
                       void* stream) {
    attn_status_t st = check_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, o_dtype);
    if (st != ATTN_OK) return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    const size_t need = fwd_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, causal, dev.num_sms);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
        return ATTN_ERR_WORKSPACE;
    return launch_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, o_dtype, workspace,
                      static_cast<cudaStream_t>(stream), dev);
}

size_t attn_fp8_codes_bytes(int B, int H, int N, int d, int transpose) {
    if (B < 1 || H < 1 || N < 1 || d != 128 || (transpose != 0 && transpose != 1)) return 0;
    if ((long long)B * H > kMaxHeads || N > kMaxLen) return 0;
    const long long n = transpose ? (long long)(N + 15) / 16 * 16 : (long long)N;
    return (size_t)((long long)B * H * n * d);
}

size_t attn_fp8_descale_count(int B, int H, int N) {
    if (B < 1 || H < 1 || N < 1 || (long long)B * H > kMaxHeads || N > kMaxLen) return 0;
    return (size_t)((long long)B * H * ((N + 127) / 128));
}

attn_status_t attn_fp8_quantize(const void* x, void* codes, float* descale, const int8_t* signs,
                                int B, int H, int N, int d, int transpose, void* stream) {
    if (!x || !codes || !descale || !aligned16(x) || !aligned16(codes) || !aligned4(descale))
        return ATTN_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || N < 1 || N > kMaxLen || (long long)B * H > kMaxHeads)
        return ATTN_ERR_INVALID_ARG;
    if (transpose != 0 && transpose != 1) return ATTN_ERR_INVALID_ARG;
    if ((long long)B * H > 65535) return ATTN_ERR_UNSUPPORTED;  // grid.y
    if (d != 128) return ATTN_ERR_UNSUPPORTED;
    DeviceInfo dev;
    attn_status_t st = current_device_info(&dev);
    if (st != ATTN_OK) return st;
    return launch_fp8_quantize(x, codes, descale, signs, B * H, N, transpose,
                               static_cast<cudaStream_t>(stream), dev);
}

attn_status_t attn_fwd_fp8(const void* q8, const void* k8, const void* vt8, const float* q_descale,
                           const float* k_descale, const float* v_descale, void* o, float* lse,
                           int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal, float scale,
                           int rotated, attn_out_dtype_t o_dtype, void* stream) {
    if (!q_descale || !k_descale || !v_descale || !aligned4(q_descale) || !aligned4(k_descale) ||
        !aligned4(v_descale))
        return ATTN_ERR_INVALID_ARG;
    if (rotated != 0 && rotated != 1) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_fwd(q8, k8, vt8, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, o_dtype);
    if (st != ATTN_OK) return st;
    if (d != 128) return ATTN_ERR_UNSUPPORTED;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    // Q and K rotated by the same signed Hadamard matrix H (entries +-1, H H^T
    // = d I): (Q D H)(K D H)^T = d Q K^T, so the scores carry a factor d that
    // the scale takes back (exact: d = 128 is a power of two).
    const float eff = rotated ? scale / (float)d : scale;
    return launch_fwd_fp8(q8, k8, vt8, q_descale, k_descale, v_descale, o, lse, B, Hq, Hkv, Nq, Nk,
                          causal, eff, o_dtype, static_cast<cudaStream_t>(stream), dev);
}

attn_status_t attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                              const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int Hq,
                              int Hkv, int total_q, int total_k, int max_seqlen_q,
                              int max_seqlen_k, int d, int causal, float scale,
                              attn_out_dtype_t o_dtype, void* stream) {
    attn_status_t st = check_varlen(cu_seqlens_q, cu_seqlens_k, total_q, total_k, max_seqlen_q, max_seqlen_k);
    if (st != ATTN_OK) return st;
    // (the per-sequence causal condition is checked on the device)
    st = check_fwd(q, k, v, o, lse, B, Hq, Hkv, max_seqlen_q, max_seqlen_k, d, 0,
                                 scale, o_dtype);
    if (st != ATTN_OK) return st;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if (!fwd_head_dim_supported(d)) return ATTN_ERR_UNSUPPORTED;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    if (d > 128)
        return launch_fwd_wide_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, Hq, Hkv,
                                      total_q, total_k, max_seqlen_q, max_seqlen_k, d, causal,
                                      scale, o_dtype, static_cast<cudaStream_t>(stream), dev);
    return launch_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, Hq, Hkv, total_q,
                             total_k, max_seqlen_q, max_seqlen_k, d, causal, scale, o_dtype,
                             static_cast<cudaStream_t>(stream), dev);
}

size_t attn_bwd_workspace_size(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
    if (check_common(B, Hq, Hkv, d, 1.0f, ATTN_OUT_BF16) != ATTN_OK) return 0;
    if (Nq < 1 || Nk < 1 || Nq > kMaxLen || Nk > kMaxLen) return 0;
    if (!fwd_head_dim_supported(d)) return 0;
    return bwd_workspace_bytes(B, Hq, Nq, d);
}

attn_status_t attn_bwd(const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                       int Hq, int Hkv, int Nq, int Nk, int d, int causal, float scale,
                       attn_out_dtype_t o_dtype, attn_out_dtype_t grad_dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
    attn_status_t st = check_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, o_dtype);
    if (st != ATTN_OK) return st;
    // (check_fwd has limited d to the forward's head dims, which the backward takes too)
    if ((st = check_grads(dout, lse, dq, dk, dv, grad_dtype)) != ATTN_OK) return st;
    const size_t need = bwd_workspace_bytes(B, Hq, Nq, d);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    return launch_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, causal, scale,
                      o_dtype, grad_dtype, workspace, static_cast<cudaStream_t>(stream), dev);
}

size_t attn_bwd_varlen_workspace_size(int B, int Hq, int Hkv, int total_q, int d) {
    if (check_common(B, Hq, Hkv, d, 1.0f, ATTN_OUT_BF16) != ATTN_OK) return 0;
    if (total_q < 1 || total_q > kMaxPackedRows || !fwd_head_dim_supported(d)) return 0;
    return bwd_varlen_workspace_bytes(B, Hq, total_q);
}

attn_status_t attn_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                              const void* dout, const float* lse, void* dq, void* dk, void* dv,
                              const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int Hq,
                              int Hkv, int total_q, int total_k, int max_seqlen_q,
                              int max_seqlen_k, int d, int causal, float scale,
                              attn_out_dtype_t o_dtype, attn_out_dtype_t grad_dtype,
                              void* workspace, size_t workspace_bytes, void* stream) {
    attn_status_t st = check_varlen(cu_seqlens_q, cu_seqlens_k, total_q, total_k, max_seqlen_q, max_seqlen_k);
    if (st != ATTN_OK) return st;
    // (the per-sequence causal condition is checked on the device)
    st = check_fwd(q, k, v, o, lse, B, Hq, Hkv, max_seqlen_q, max_seqlen_k, d, 0,
                                 scale, o_dtype);
    if (st != ATTN_OK) return st;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if ((st = check_grads(dout, lse, dq, dk, dv, grad_dtype)) != ATTN_OK) return st;
    if (!fwd_head_dim_supported(d)) return ATTN_ERR_UNSUPPORTED;
    const size_t need = bwd_varlen_workspace_bytes(B, Hq, total_q);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    return launch_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, B, Hq,
                             Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, d, causal, scale,
                             o_dtype, grad_dtype, workspace, static_cast<cudaStream_t>(stream), dev);
}

size_t attn_decode_workspace_size(int B, int Hq, int Hkv, int Nmax, int d, int num_splits) {
    if (check_decode_shape(B, Hq, Hkv, Nmax, d, num_splits) != ATTN_OK) return 0;
    int sms = 0;
    if (current_num_sms(&sms) != 0) return 0;
    const int chunk = decode_chunk(Nmax, B, Hkv, sms, num_splits);
    return decode_workspace_bytes(B, Hq, Nmax, decode_pad_head_dim(d), chunk);
}

int attn_decode_kernel_launches(int B, int Hq, int Hkv, int Nmax, int d, int num_splits) {
    if (check_decode_shape(B, Hq, Hkv, Nmax, d, num_splits) != ATTN_OK) return -1;
    int sms = 0;
    if (current_num_sms(&sms) != 0) return -1;
    const int chunk = decode_chunk(Nmax, B, Hkv, sms, num_splits);
    const int max_splits = (Nmax + chunk - 1) / chunk;
    return decode_merges_in_kernel(B, Hkv, Hq / Hkv, max_splits, decode_pad_head_dim(d)) ? 1 : 2;
}

attn_status_t attn_decode(const void* q, const void* k_cache, const void* v_cache,
                          const int* seqlens, void* o, float* lse, int B, int Hq, int Hkv,
                          int Nmax, int d, float scale, int num_splits, void* workspace,
                          size_t workspace_bytes, attn_out_dtype_t o_dtype, void* stream) {
    attn_status_t st = check_decode_call(q, k_cache, v_cache, seqlens, o, lse, B, Hq, Hkv, Nmax,
                                         d, scale, num_splits, o_dtype);
    if (st != ATTN_OK) return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    const int chunk = decode_chunk(Nmax, B, Hkv, dev.num_sms, num_splits);
    const size_t need = decode_workspace_bytes(B, Hq, Nmax, decode_pad_head_dim(d), chunk);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
    return launch_decode(q, k_cache, v_cache, seqlens, o, lse, B, Hq, Hkv, Nmax, d, scale, chunk,
                         workspace, o_dtype, static_cast<cudaStream_t>(stream), dev);
}

attn_status_t attn_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                                const int* block_table, const int* seqlens, void* o, float* lse,
                                int B, int Hq, int Hkv, long long num_blocks, int page_size,
                                int max_blocks, int d, float scale, int num_splits, void* workspace,
                                size_t workspace_bytes, attn_out_dtype_t o_dtype, void* stream) {
    attn_status_t st = check_decode_paged(q, k_pages, v_pages, block_table, seqlens, o, lse, B, Hq, Hkv,
                                          num_blocks, page_size, max_blocks, d, scale, num_splits, o_dtype);
    if (st != ATTN_OK) return st;
    const int Nmax = max_blocks * page_size;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    const int chunk = decode_chunk(Nmax, B, Hkv, dev.num_sms, num_splits);
    const size_t need = decode_workspace_bytes(B, Hq, Nmax, decode_pad_head_dim(d), chunk);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
    return launch_decode_paged(q, k_pages, v_pages, block_table, seqlens, o, lse, B, Hq, Hkv,
                               num_blocks, page_size, max_blocks, d, scale, chunk, workspace,
                               o_dtype, static_cast<cudaStream_t>(stream), dev);
}

attn_status_t attn_bias_buckets(int num_buckets, int max_distance, int bidirectional, int* buckets,
                                int capacity, int* first, int* span) try {
    if (!first || !span || (bidirectional != 0 && bidirectional != 1)) return ATTN_ERR_INVALID_ARG;
    if (num_buckets < (bidirectional ? 4 : 2) || (bidirectional && num_buckets % 2 != 0)) return ATTN_ERR_INVALID_ARG;
    const int n = bidirectional ? num_buckets / 2 : num_buckets, e = n / 2, s = n - e;
    if (max_distance <= e) return ATTN_ERR_INVALID_ARG;
    if (num_buckets > 1024 || max_distance > kMaxLen) return ATTN_ERR_UNSUPPORTED;
    // the smallest distance of bucket e + k: ceil(e (D / e)^(k / s)).  Where that is
    // too near a whole number for floating point, whole numbers decide.
    std::vector<long long> from(s);
    for (int k = 0; k < s; ++k) {
        const double t = (double)e * std::pow((double)max_distance / e, (double)k / s);
        const double m = std::round(t);
        from[k] = std::fabs(t - m) > 1e-6 * t ? (long long)std::ceil(t)
                                              : (long long)m + (bucket_reached((long long)m, s, e, k, max_distance) ? 0 : 1);
    }
    const long long far = from[s - 1];
    const long long length = bidirectional ? 2 * far + 1 : far + 1;
    if (length > kMaxBiasSpan) return ATTN_ERR_UNSUPPORTED;
    *first = (int)-far;
    *span = (int)length;
    if (!buckets) return ATTN_OK;
    if (capacity < length) return ATTN_ERR_INVALID_ARG;
    for (long long r = 0, k = 0; r <= far; ++r) {
        while (k + 1 < s && r >= from[k + 1]) ++k;
        const int b = (int)(r < e ? r : e + k);
        buckets[far - r] = b;
        if (bidirectional && r > 0) buckets[far + r] = n + b;
    }
    return ATTN_OK;
} catch (...) {   // (no memory for a few kilobytes of host vectors)
    return ATTN_ERR_UNSUPPORTED;
}

attn_status_t attn_fwd_bias(const void* q, const void* k, const void* v, const void* table,
                            attn_out_dtype_t table_dtype, const int* buckets, int first, int span,
                            int num_buckets, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int Nk,
                            int d, int causal, float scale, attn_out_dtype_t o_dtype, void* workspace,
                            size_t workspace_bytes, void* stream) {
    attn_status_t st = check_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, o_dtype);
    if (st != ATTN_OK) return st;
    if ((st = check_bias(table, table_dtype, buckets, first, span, num_buckets, d)) != ATTN_OK) return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    const size_t need = fwd_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, causal, dev.num_sms);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
        return ATTN_ERR_WORKSPACE;
    const BiasArgs bias = bias_args(table, table_dtype, buckets, first, span, num_buckets);
    return launch_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, o_dtype, workspace,
                      static_cast<cudaStream_t>(stream), dev, &bias);
}

attn_status_t attn_fwd_varlen_bias(const void* q, const void* k, const void* v, const void* table,
                                   attn_out_dtype_t table_dtype, const int* buckets, int first, int span,
                                   int num_buckets, void* o, float* lse, const int* cu_seqlens_q,
                                   const int* cu_seqlens_k, int B, int Hq, int Hkv, int total_q, int total_k,
                                   int max_seqlen_q, int max_seqlen_k, int d, int causal, float scale,
                                   attn_out_dtype_t o_dtype, void* stream) {
    attn_status_t st = check_varlen(cu_seqlens_q, cu_seqlens_k, total_q, total_k, max_seqlen_q, max_seqlen_k);
    if (st != ATTN_OK) return st;
    // (the per-sequence causal condition is checked on the device)
    st = check_fwd(q, k, v, o, lse, B, Hq, Hkv, max_seqlen_q, max_seqlen_k, d, 0, scale, o_dtype);
    if (st != ATTN_OK) return st;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if ((st = check_bias(table, table_dtype, buckets, first, span, num_buckets, d)) != ATTN_OK) return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    const BiasArgs bias = bias_args(table, table_dtype, buckets, first, span, num_buckets);
    return launch_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, Hq, Hkv, total_q, total_k,
                             max_seqlen_q, max_seqlen_k, d, causal, scale, o_dtype,
                             static_cast<cudaStream_t>(stream), dev, &bias);
}

size_t attn_bwd_bias_workspace_size(int B, int Hq, int Hkv, int Nq, int Nk, int d, int span) {
    const size_t base = attn_bwd_workspace_size(B, Hq, Hkv, Nq, Nk, d);
    if (base == 0 || !head_dim_supported(d) || span < 1 || span > kMaxBiasSpan) return 0;
    if (Hq > 65535 || too_many_bias_tiles(B, Nk)) return 0;
    return base + bwd_bias_workspace_bytes(B, Hq, Nk, span);
}

attn_status_t attn_bwd_bias(const void* q, const void* k, const void* v, const void* o, const void* dout,
                            const float* lse, const void* table, attn_out_dtype_t table_dtype,
                            const int* buckets, int first, int span, int num_buckets, void* dq, void* dk,
                            void* dv, float* dtable, int B, int Hq, int Hkv, int Nq, int Nk, int d,
                            int causal, float scale, attn_out_dtype_t o_dtype, attn_out_dtype_t grad_dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
    attn_status_t st = check_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, o_dtype);
    if (st != ATTN_OK) return st;
    if ((st = check_grads(dout, lse, dq, dk, dv, grad_dtype)) != ATTN_OK) return st;
    if (!dtable || !aligned4(dtable)) return ATTN_ERR_INVALID_ARG;
    if (Hq > 65535 || too_many_bias_tiles(B, Nk)) return ATTN_ERR_UNSUPPORTED;   // (Hq: a grid's second dimension)
    if ((st = check_bias(table, table_dtype, buckets, first, span, num_buckets, d)) != ATTN_OK) return st;
    const size_t need = bwd_workspace_bytes(B, Hq, Nq, d) + bwd_bias_workspace_bytes(B, Hq, Nk, span);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    const BiasArgs bias = bias_args(table, table_dtype, buckets, first, span, num_buckets);
    return launch_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, causal, scale, o_dtype,
                      grad_dtype, workspace, static_cast<cudaStream_t>(stream), dev, &bias, dtable);
}

size_t attn_bwd_varlen_bias_workspace_size(int B, int Hq, int Hkv, int total_q, int max_seqlen_k, int d,
                                           int span) {
    const size_t base = attn_bwd_varlen_workspace_size(B, Hq, Hkv, total_q, d);
    if (base == 0 || !head_dim_supported(d) || span < 1 || span > kMaxBiasSpan) return 0;
    if (max_seqlen_k < 1 || max_seqlen_k > kMaxLen || Hq > 65535 || too_many_bias_tiles(B, max_seqlen_k)) return 0;
    return base + bwd_bias_workspace_bytes(B, Hq, max_seqlen_k, span);
}

attn_status_t attn_bwd_varlen_bias(const void* q, const void* k, const void* v, const void* o,
                                   const void* dout, const float* lse, const void* table,
                                   attn_out_dtype_t table_dtype, const int* buckets, int first, int span,
                                   int num_buckets, void* dq, void* dk, void* dv, float* dtable,
                                   const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int Hq, int Hkv,
                                   int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, int d,
                                   int causal, float scale, attn_out_dtype_t o_dtype,
                                   attn_out_dtype_t grad_dtype, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    attn_status_t st = check_varlen(cu_seqlens_q, cu_seqlens_k, total_q, total_k, max_seqlen_q, max_seqlen_k);
    if (st != ATTN_OK) return st;
    st = check_fwd(q, k, v, o, lse, B, Hq, Hkv, max_seqlen_q, max_seqlen_k, d, 0, scale, o_dtype);
    if (st != ATTN_OK) return st;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
    if ((st = check_grads(dout, lse, dq, dk, dv, grad_dtype)) != ATTN_OK) return st;
    if (!dtable || !aligned4(dtable)) return ATTN_ERR_INVALID_ARG;
    if (Hq > 65535 || too_many_bias_tiles(B, max_seqlen_k)) return ATTN_ERR_UNSUPPORTED;
    if ((st = check_bias(table, table_dtype, buckets, first, span, num_buckets, d)) != ATTN_OK) return st;
    const size_t need = bwd_varlen_workspace_bytes(B, Hq, total_q) +
                        bwd_bias_workspace_bytes(B, Hq, max_seqlen_k, span);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    const BiasArgs bias = bias_args(table, table_dtype, buckets, first, span, num_buckets);
    return launch_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, B, Hq, Hkv,
                             total_q, total_k, max_seqlen_q, max_seqlen_k, d, causal, scale, o_dtype,
                             grad_dtype, workspace, static_cast<cudaStream_t>(stream), dev, &bias, dtable);
}

attn_status_t attn_decode_paged_bias(const void* q, const void* k_pages, const void* v_pages,
                                     const int* block_table, const int* seqlens, const void* table,
                                     attn_out_dtype_t table_dtype, const int* buckets, int first, int span,
                                     int num_buckets, void* o, float* lse, int B, int Hq, int Hkv,
                                     long long num_blocks, int page_size, int max_blocks, int d, float scale,
                                     int num_splits, void* workspace, size_t workspace_bytes,
                                     attn_out_dtype_t o_dtype, void* stream) {
    attn_status_t st = check_decode_paged(q, k_pages, v_pages, block_table, seqlens, o, lse, B, Hq, Hkv,
                                          num_blocks, page_size, max_blocks, d, scale, num_splits, o_dtype);
    if (st != ATTN_OK) return st;
    if ((st = check_bias(table, table_dtype, buckets, first, span, num_buckets, d)) != ATTN_OK) return st;
    const int Nmax = max_blocks * page_size;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    const int chunk = decode_chunk(Nmax, B, Hkv, dev.num_sms, num_splits);
    const size_t need = decode_workspace_bytes(B, Hq, Nmax, decode_pad_head_dim(d), chunk);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
    const BiasArgs bias = bias_args(table, table_dtype, buckets, first, span, num_buckets);
    return launch_decode_paged(q, k_pages, v_pages, block_table, seqlens, o, lse, B, Hq, Hkv, num_blocks,
                               page_size, max_blocks, d, scale, chunk, workspace, o_dtype,
                               static_cast<cudaStream_t>(stream), dev, &bias);
}

attn_status_t attn_page_pool_init(int* pool, int num_blocks, void* stream) {
    if (!pool || !aligned16(pool) || num_blocks < 1) return ATTN_ERR_INVALID_ARG;
    if (num_blocks > kMaxPackedRows) return ATTN_ERR_UNSUPPORTED;
    DeviceInfo dev;
    attn_status_t st = current_device_info(&dev);
    if (st != ATTN_OK) return st;
    return launch_pages_init(pool, num_blocks, static_cast<cudaStream_t>(stream));
}

attn_status_t attn_pages_extend(int* pool, int num_blocks, int* block_table, int* seqlens,
                                const int* new_lens, long long* slots, int* positions, int* cu_seqlens,
                                int* granted, int B, int max_blocks, int page_size, int width, int total,
                                void* stream) {
    attn_status_t st = check_page_tables(pool, num_blocks, block_table, seqlens, new_lens, B, max_blocks, page_size);
    if (st != ATTN_OK) return st;
    if (width < 0 || total < 0 || (width > 0 && (total != 0 || cu_seqlens))) return ATTN_ERR_INVALID_ARG;
    const long long n = width > 0 ? (long long)B * width : total;
    if (n > kMaxPackedRows) return ATTN_ERR_INVALID_ARG;
    if ((n > 0 && !slots) || !aligned16(slots) || !aligned16(positions) || !aligned4(cu_seqlens) ||
        !aligned4(granted))
        return ATTN_ERR_INVALID_ARG;
    // (every block reads the lengths while the first one writes these)
    for (const int* out : {positions, cu_seqlens, granted})
        if (out && (out == new_lens || out == seqlens || out == pool || out == block_table)) return ATTN_ERR_INVALID_ARG;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    return launch_pages_extend(pool, num_blocks, block_table, seqlens, new_lens, slots, positions, cu_seqlens,
                               granted, B, max_blocks, page_size, width, n, static_cast<cudaStream_t>(stream), dev);
}

attn_status_t attn_pages_trim(int* pool, int num_blocks, const int* block_table, int* seqlens,
                              const int* keep_lens, int B, int max_blocks, int page_size, void* stream) {
    attn_status_t st = check_page_tables(pool, num_blocks, block_table, seqlens, keep_lens, B, max_blocks, page_size);
    if (st != ATTN_OK) return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    return launch_pages_trim(pool, num_blocks, block_table, seqlens, keep_lens, B, max_blocks, page_size,
                             static_cast<cudaStream_t>(stream), dev);
}

attn_status_t attn_rope_frequencies(int rotary_dim, double base, attn_rope_scaling_t scaling,
                                    double factor, int original_len, double beta_fast,
                                    double beta_slow, double* inv_freq, float* magnitude) {
    if (!inv_freq || rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > 256) return ATTN_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base)) return ATTN_ERR_INVALID_ARG;
    if (scaling < ATTN_ROPE_PLAIN || scaling > ATTN_ROPE_BY_PARTS) return ATTN_ERR_INVALID_ARG;
    if (scaling != ATTN_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return ATTN_ERR_INVALID_ARG;
    if (scaling == ATTN_ROPE_BY_PARTS &&
        (original_len < 1 || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast)))
        return ATTN_ERR_INVALID_ARG;
    const int n = rotary_dim / 2;
    if (scaling == ATTN_ROPE_NTK && rotary_dim > 2)
        base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
    double lo = 0.0, hi = 0.0;
    if (scaling == ATTN_ROPE_BY_PARTS) {
        // the (fractional) pair that turns `turns` times over original_len positions
        auto pair_of = [&](double turns) {
            return rotary_dim * std::log(original_len / (turns * 6.283185307179586)) / (2.0 * std::log(base));
        };
        lo = std::max(std::floor(pair_of(beta_fast)), 0.0);
        hi = std::min(std::ceil(pair_of(beta_slow)), (double)(rotary_dim - 1));  // (may lie past the last pair)
    }
    for (int i = 0; i < n; ++i) {
        double f = std::pow(base, -2.0 * i / rotary_dim);
        if (scaling == ATTN_ROPE_LINEAR) f /= factor;
        if (scaling == ATTN_ROPE_BY_PARTS) {
            const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        inv_freq[i] = f;
    }
    if (magnitude)
        *magnitude = scaling == ATTN_ROPE_BY_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return ATTN_OK;
}

attn_status_t attn_rope(const void* q, const void* k, void* q_out, void* k_out,
                        const long long* q_strides, const long long* k_strides,
                        const long long* q_out_strides, const long long* k_out_strides,
                        const int* positions, long long positions_stride, const double* inv_freq,
                        int B, int Hq, int Hkv, int N, int d, int rotary_dim, int interleaved,
                        int inverse, float magnitude, attn_out_dtype_t in_dtype,
                        attn_out_dtype_t out_dtype, void* stream) {
    if (!q || !q_out || !positions || !inv_freq) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(q_out) || !aligned4(positions) || !aligned8(inv_freq))
        return ATTN_ERR_INVALID_ARG;
    if (!k != !k_out || (k && (!aligned16(k) || !aligned16(k_out)))) return ATTN_ERR_INVALID_ARG;
    if (in_dtype != ATTN_OUT_BF16 && in_dtype != ATTN_OUT_F32) return ATTN_ERR_INVALID_ARG;
    if (out_dtype != ATTN_OUT_BF16 && out_dtype != ATTN_OUT_F32) return ATTN_ERR_INVALID_ARG;
    if (B < 1 || Hq < 1 || N < 1 || d < 1 || (k ? Hkv < 1 : Hkv != 0)) return ATTN_ERR_INVALID_ARG;
    if (Hq > kMaxHeads || Hkv > kMaxHeads || (long long)B * N > kMaxPackedRows) return ATTN_ERR_INVALID_ARG;
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > d) return ATTN_ERR_INVALID_ARG;
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return ATTN_ERR_INVALID_ARG;
    if (!std::isfinite(magnitude) || positions_stride < 0) return ATTN_ERR_INVALID_ARG;
    if (!fwd_head_dim_supported(d)) return ATTN_ERR_UNSUPPORTED;
    const int bi = in_dtype == ATTN_OUT_F32 ? 4 : 2, bo = out_dtype == ATTN_OUT_F32 ? 4 : 2;
    const Strides sq(q_strides, Hq, N, d), sk(k_strides, Hkv, N, d), sqo(q_out_strides, Hq, N, d),
        sko(k_out_strides, Hkv, N, d);
    q_strides = sq.s;
    k_strides = sk.s;
    q_out_strides = sqo.s;
    k_out_strides = sko.s;
    if (!strides_ok(q_strides, B, Hq, N, d, bi, false) || !strides_ok(q_out_strides, B, Hq, N, d, bo, true))
        return ATTN_ERR_INVALID_ARG;
    if (k && (!strides_ok(k_strides, B, Hkv, N, d, bi, false) ||
              !strides_ok(k_out_strides, B, Hkv, N, d, bo, true)))
        return ATTN_ERR_INVALID_ARG;
    // in place: every element has to be read and written at the same address
    auto in_place_ok = [&](const void* x, const void* out, const long long* xs, const long long* os) {
        return x != out || (bi == bo && std::equal(xs, xs + 3, os));
    };
    if (!in_place_ok(q, q_out, q_strides, q_out_strides) ||
        (k && !in_place_ok(k, k_out, k_strides, k_out_strides)))
        return ATTN_ERR_INVALID_ARG;
    DeviceInfo dev;
    attn_status_t st = current_device_info(&dev);
    if (st != ATTN_OK) return st;
    return launch_rope(q, k, q_out, k_out, q_strides, k_strides, q_out_strides, k_out_strides,
                       positions, positions_stride, inv_freq, B, Hq, Hkv, N, d, rotary_dim,
                       interleaved, inverse, magnitude, in_dtype, out_dtype,
                       static_cast<cudaStream_t>(stream), dev);
}

attn_status_t attn_cache_write(const void* k, const void* v, const long long* k_strides,
                               const long long* v_strides, void* k_pages, void* v_pages,
                               float* k_descale, float* v_descale, const long long* slots, int B,
                               int N, int Hkv, int d, long long num_blocks, int page_size,
                               attn_cache_dtype_t cache_dtype, void* stream) {
    if (!k || !v || !slots || !aligned16(k) || !aligned16(v) || !aligned8(slots)) return ATTN_ERR_INVALID_ARG;
    if (B < 1 || N < 1 || (long long)B * N > kMaxPackedRows) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_pages(Hkv, d, num_blocks, page_size, cache_dtype, k_pages, v_pages,
                                   k_descale, v_descale);
    if (st != ATTN_OK) return st;
    const Strides sk(k_strides, Hkv, N, d), sv(v_strides, Hkv, N, d);
    k_strides = sk.s;
    v_strides = sv.s;
    if (!strides_ok(k_strides, B, Hkv, N, d, 2, false) || !strides_ok(v_strides, B, Hkv, N, d, 2, false))
        return ATTN_ERR_INVALID_ARG;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    return launch_cache_write(k, v, k_strides, v_strides, k_pages, v_pages, k_descale, v_descale,
                              slots, B, N, Hkv, d, num_blocks, page_size, cache_dtype,
                              static_cast<cudaStream_t>(stream), dev);
}

attn_status_t attn_cache_read(const void* k_pages, const void* v_pages, const float* k_descale,
                              const float* v_descale, const int* block_table,
                              const int* cu_seqlens, void* k_out, void* v_out, int B, int Hkv,
                              int total, long long num_blocks, int page_size, int max_blocks,
                              int d, attn_cache_dtype_t cache_dtype, attn_out_dtype_t out_dtype,
                              void* stream) {
    if (!block_table || !cu_seqlens || !k_out || !v_out || !aligned4(block_table) ||
        !aligned4(cu_seqlens) || !aligned16(k_out) || !aligned16(v_out))
        return ATTN_ERR_INVALID_ARG;
    if (B < 1 || total < 1 || total > kMaxPackedRows || max_blocks < 1) return ATTN_ERR_INVALID_ARG;
    if (out_dtype != ATTN_OUT_BF16 && out_dtype != ATTN_OUT_F32) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_pages(Hkv, d, num_blocks, page_size, cache_dtype, k_pages, v_pages,
                                   k_descale, v_descale);
    if (st != ATTN_OK) return st;
    if ((long long)Hkv * d > (1ll << 24)) return ATTN_ERR_UNSUPPORTED;  // (32-bit indexes within a token)
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    return launch_cache_read(k_pages, v_pages, k_descale, v_descale, block_table, cu_seqlens, k_out,
                             v_out, B, Hkv, total, num_blocks, page_size, max_blocks, d,
                             cache_dtype, out_dtype, static_cast<cudaStream_t>(stream), dev);
}

size_t attn_decode_tree_workspace_size(int B, int Hq, int Hkv, int T, int max_blocks, int page_size,
                                       int d, attn_cache_dtype_t cache_dtype) {
    if (check_tree_shape(B, Hq, Hkv, T, max_blocks, page_size, d, cache_dtype) != ATTN_OK) return 0;
    int sms = 0;
    if (current_num_sms(&sms) != 0) return 0;
    return tree_workspace_bytes(Hq, Hkv, T, d, cache_dtype, sms);
}

attn_status_t attn_decode_tree(const void* q, const void* k_pages, const void* v_pages,
                               const float* k_descale, const float* v_descale,
                               const int* block_table, const int* seqlens, const int* q_lens,
                               const uint64_t* tree_mask, void* o, float* lse, int B, int Hq,
                               int Hkv, int T, long long num_blocks, int page_size, int max_blocks,
                               int d, float scale, attn_cache_dtype_t cache_dtype, void* workspace,
                               size_t workspace_bytes, attn_out_dtype_t o_dtype, void* stream) {
    if (!q || !block_table || !seqlens || !o) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || !aligned4(block_table) || !aligned4(seqlens))
        return ATTN_ERR_INVALID_ARG;
    if ((q_lens && !aligned4(q_lens)) || (tree_mask && !aligned8(tree_mask)) || (lse && !aligned4(lse)))
        return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_common(B, Hq, Hkv, d, scale, o_dtype);
    if (st != ATTN_OK) return st;
    if ((st = check_tree_shape(B, Hq, Hkv, T, max_blocks, page_size, d, cache_dtype)) != ATTN_OK) return st;
    if ((st = check_pages(Hkv, d, num_blocks, page_size, cache_dtype, k_pages, v_pages, k_descale,
                          v_descale)) != ATTN_OK)
        return st;
    DeviceInfo dev;
    if ((st = current_device_info(&dev)) != ATTN_OK) return st;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < tree_workspace_bytes(Hq, Hkv, T, d, cache_dtype, dev.num_sms))
        return ATTN_ERR_WORKSPACE;
    return launch_decode_tree(q, k_pages, v_pages, k_descale, v_descale, block_table, seqlens,
                              q_lens, tree_mask, o, lse, B, Hq, Hkv, T, num_blocks, page_size,
                              max_blocks, d, scale, cache_dtype, workspace, o_dtype,
                              static_cast<cudaStream_t>(stream), dev);
}

const char* attn_status_string(attn_status_t s) {
    switch (s) {
        case ATTN_OK: return "ATTN_OK";
        case ATTN_ERR_INVALID_ARG: return "ATTN_ERR_INVALID_ARG";
        case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED";
        case ATTN_ERR_CUDA: return "ATTN_ERR_CUDA";
        case ATTN_ERR_TIMEOUT: return "ATTN_ERR_TIMEOUT";
        case ATTN_ERR_WORKSPACE: return "ATTN_ERR_WORKSPACE";
    }
    return "ATTN_ERR_UNKNOWN";
}

attn_status_t attn_selftest_bounded_wait(int mode, int* result, void* stream) {
    if ((mode != 0 && mode != 1) || !result || !aligned4(result)) return ATTN_ERR_INVALID_ARG;
    DeviceInfo dev;
    attn_status_t st = current_device_info(&dev);
    if (st != ATTN_OK) return st;
    attn_selftest_wait_kernel<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(mode, result, dev.err_word);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_last_device_error(void* stream) {
    DeviceInfo dev;
    attn_status_t st = current_device_info(&dev);
    if (st != ATTN_OK) return st;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return ATTN_ERR_CUDA;
    unsigned int word = 0;
    if (cudaMemcpy(&word, dev.err_word, sizeof word, cudaMemcpyDeviceToHost) != cudaSuccess)
        return ATTN_ERR_CUDA;
    const unsigned int zero = 0;
    if (word != 0 && cudaMemcpy(dev.err_word, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess)
        return ATTN_ERR_CUDA;
    if (word & kErrTimeout) return ATTN_ERR_TIMEOUT;
    if (word & kErrLayout) return ATTN_ERR_CUDA;
    if (word & kErrBadSeqlen) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

int attn_decode_num_splits(int units, int num_sms, int max_splits) {
    if (units < 1 || num_sms < 1 || max_splits < 1) return 0;
    std::vector<double> eff((size_t)max_splits + 1, 0.0);
    double best = 0.0;
    for (int s = 1; s <= max_splits; ++s) {
        const double waves = (double)units * s / num_sms;
        eff[s] = waves / std::ceil(waves);
        best = std::max(best, eff[s]);
    }
    for (int s = 1; s <= max_splits; ++s)
        if (eff[s] >= 0.85 * best) return s;
    return 1;
}

long long attn_list_schedule(const int* costs, int n, int workers, int lpt, long long* loads_out) {
    if (n < 0 || workers < 1 || (n > 0 && !costs)) return -1;
    std::vector<int> order((size_t)n);
    std::iota(order.begin(), order.end(), 0);
    if (lpt)
        std::stable_sort(order.begin(), order.end(),
                         [&](int a, int b) { return costs[a] > costs[b]; });
    std::vector<long long> load((size_t)workers, 0);
    for (int idx : order) {
        if (costs[idx] < 0) return -1;
        int w = 0;
        for (int i = 1; i < workers; ++i)
            if (load[i] < load[w]) w = i;
        load[w] += costs[idx];
    }
    if (loads_out) std::copy(load.begin(), load.end(), loads_out);
    return workers ? *std::max_element(load.begin(), load.end()) : 0;
}

int attn_kv_tiles(int row0, int rows, int Nq, int Nk, int causal, int block) {
    return kv_tiles_for_rows(row0, rows, Nq, Nk, causal, block);
}

long long attn_fwd_num_units(int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Nk < 1 || d < 1 || Hq % Hkv) return -1;
    return make_fwd_shape(B, Hq, Hkv, Nq, Nk, d, causal).units;
}

int attn_fwd_schedule(int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal, int num_sms,
                      long long n, int* units_out, int* cost_out) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Nk < 1 || d < 1 || Hq % Hkv || !units_out ||
        num_sms < 0)
        return -1;
    const FwdShape s = make_fwd_shape(B, Hq, Hkv, Nq, Nk, d, causal, num_sms);
    if (n != s.units || s.units >= (1ll << 31)) return -1;
    for (long long i = 0; i < n; ++i) {
        int bh, mb;
        unit_of(s, (uint32_t)i, bh, mb);
        units_out[3 * i] = bh / Hq;
        units_out[3 * i + 1] = bh % Hq;
        units_out[3 * i + 2] = mb;
        if (cost_out) cost_out[i] = tile_kv_count(mb, 0, s) + tile_kv_count(mb, 1, s);
    }
    return 0;
}

long long attn_packed_map_shift(unsigned long long address, long long rows, long long row_bytes) {
    if (rows < 1 || rows > kMaxPackedRows || row_bytes < 1 || row_bytes >= (1ll << 34)) return -1;
    return (long long)packed_map_shift((uintptr_t)address, rows, (size_t)row_bytes);
}

int attn_fwd_split_plan(int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal, int num_sms,
                        int* n_full, int* n_split, int* parts) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Nk < 1 || d < 1 || Hq % Hkv || num_sms < 1 ||
        !n_full || !n_split || !parts)
        return -1;
    const FwdShape s = make_fwd_shape(B, Hq, Hkv, Nq, Nk, d, causal);
    if (s.units >= (1ll << 31)) return -1;
    const FwdSplit sp = plan_tail_split(s, num_sms);
    *n_full = sp.n_full;
    *n_split = sp.n_split;
    *parts = sp.parts;
    return 0;
}

}  // extern "C"
