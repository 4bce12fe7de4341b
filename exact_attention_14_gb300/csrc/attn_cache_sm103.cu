// attn_cache_sm103.cu -- writing keys and values into a paged KV cache and
// reading them back.
//
// The cache is the one attn_decode_paged reads, pages [num_blocks, page_size,
// Hkv, d], in bf16 or in E4M3 with one fp32 descale per (key, KV head), held
// [num_blocks, Hkv, page_size] so that an attention tile's descales are
// contiguous.
//
// Write, one row x of d values (a token and KV head):
//   amax = max |x_i|, a = max(amax, 2^-100),
//   code_i = E4M3(x_i * (448 / a)) (nearest even, saturating),
//   descale = a / 448;   all-zero rows get codes 0 and descale 1.
// The floor 2^-100 keeps 448 / a and a / 448 finite and normal.  A NaN element
// keeps a NaN code, an infinite one makes its row NaN.
// Read: code * descale (fp32 product) rounded to the output type.
//
// Bound: HBM.  Both kernels move 16 elements per lane with 16-byte accesses;
// nothing is staged in shared memory, since no element is used twice.
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kCacheThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kTinyAmax = 7.888609052210118e-31f;  // 2^-100

struct WriteSide {
    const __nv_bfloat16* x;
    long long xb, xh, xn;  // element strides: batch, head, token
    uint8_t* pages;
    float* descale;        // E4M3 only
};

struct WriteParams {
    WriteSide side[2];     // k, v
    const long long* slots;  // [B, N]
    long long tokens, num_slots;
    int N, Hkv, d, page_size;
    int lanes;             // lanes of a row (a power of two, 16 elements each)
    unsigned int* err;
};

// Two packed bf16 values quantized: low 16 bits of the result.
__device__ __forceinline__ uint32_t quant2(uint32_t w, float s) {
    return pack_e4m3x2(bf16lo_to_f32(w) * s, bf16hi_to_f32(w) * s);
}
__device__ __forceinline__ uint32_t quant4(uint32_t a, uint32_t b, float s) {
    return quant2(a, s) | (quant2(b, s) << 16);
}
__device__ __forceinline__ float amax2(float m, uint32_t w) {
    return fmaxf(m, fmaxf(fabsf(bf16lo_to_f32(w)), fabsf(bf16hi_to_f32(w))));
}

// Row r of the call = (tile of 32 tokens, KV head, token in the tile): a
// block's rows are consecutive tokens of a head, so that the descales of a
// page are written as whole lines.  Each lane holds 16 columns of the K row and
// of the V row of its token and head.
template <bool E4M3>
__global__ void __launch_bounds__(kCacheThreads)
attn_cache_write_kernel(const __grid_constant__ WriteParams p) {
    const int lanes = p.lanes;
    const long long at = (long long)blockIdx.x * kCacheThreads + threadIdx.x;
    const long long row = at / lanes;
    const int col = 16 * (int)(at - row * lanes);
    const long long tile = row / (32 * p.Hkv);
    const int in_tile = (int)(row - tile * (32 * p.Hkv));
    const int h = in_tile >> 5;
    const long long token = tile * 32 + (in_tile & 31);
    const bool live_token = token < p.tokens;
    long long slot = live_token ? __ldg(p.slots + token) : -1;
    if (slot >= p.num_slots || slot < -1) {
        if (h == 0 && col == 0) atomicOr(p.err, kErrBadSeqlen);
        slot = -1;
    }
    const bool live = slot >= 0 && col < p.d;
    const long long b = token / p.N;
    const int n = (int)(token - b * p.N);
    uint4 w[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        w[s][0] = w[s][1] = make_uint4(0u, 0u, 0u, 0u);
        if (live) {
            const WriteSide& sd = p.side[s];
            const uint4* x = reinterpret_cast<const uint4*>(sd.x + b * sd.xb + (long long)h * sd.xh +
                                                            (long long)n * sd.xn + col);
            w[s][0] = __ldcs(x);
            if (col + 8 < p.d) w[s][1] = __ldcs(x + 1);
        }
    }
    const long long out = (slot * p.Hkv + h) * p.d + col;  // element of the cache
    if constexpr (!E4M3) {
        if (!live) return;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint4* o = reinterpret_cast<uint4*>(p.side[s].pages + 2 * out);
            o[0] = w[s][0];
            if (col + 8 < p.d) o[1] = w[s][1];
        }
    } else {
        float m[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float a = 0.f;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                a = amax2(a, w[s][v].x);
                a = amax2(a, w[s][v].y);
                a = amax2(a, w[s][v].z);
                a = amax2(a, w[s][v].w);
            }
            m[s] = a;
        }
        for (int off = lanes >> 1; off > 0; off >>= 1) {
            m[0] = fmaxf(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], off));
            m[1] = fmaxf(m[1], __shfl_xor_sync(0xFFFFFFFFu, m[1], off));
        }
        if (!live) return;
        // (slot, h) -> its descale: 32-bit division where the slot allows it
        long long blk;
        if (slot <= 0x7FFFFFFFll) blk = (long long)((unsigned)slot / (unsigned)p.page_size);
        else blk = slot / p.page_size;
        const long long dsc = (blk * p.Hkv + h) * p.page_size + (slot - blk * p.page_size);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const float a = fmaxf(m[s], kTinyAmax);
            const float scale = m[s] > 0.f ? kE4m3Max / a : 1.0f;
            *reinterpret_cast<uint4*>(p.side[s].pages + out) =
                make_uint4(quant4(w[s][0].x, w[s][0].y, scale), quant4(w[s][0].z, w[s][0].w, scale),
                           quant4(w[s][1].x, w[s][1].y, scale), quant4(w[s][1].z, w[s][1].w, scale));
            if (col == 0) p.side[s].descale[dsc] = m[s] > 0.f ? a / kE4m3Max : 1.0f;
        }
    }
}

struct ReadParams {
    const uint8_t* pages[2];   // k, v
    const float* descale[2];
    void* out[2];              // [total, Hkv, d]
    const int* block_table;    // [B, max_blocks]
    const int* cu;             // [B + 1]
    long long num_blocks;
    int B, Hkv, d, page_size, max_blocks, total;
    unsigned int* err;
};

constexpr int kReadTokens = 16;  // tokens of a block

__device__ __forceinline__ float2 e4m3x2_f32(uint32_t pair16) {
    uint32_t h2;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h2) : "r"(pair16));
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h2));
    return f;
}

template <typename TO>
__device__ __forceinline__ void store4(TO* p, float a, float b, float c, float d);
template <>
__device__ __forceinline__ void store4<float>(float* p, float a, float b, float c, float d) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(a, b, c, d));
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, float a, float b, float c, float d) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d)));
}

// A block reads kReadTokens consecutive packed tokens, all heads, K or V
// (blockIdx.y).  The first lanes find each token's sequence by bisection and
// its row in the cache; then every thread streams groups of columns.
template <bool E4M3, typename TO>
__global__ void __launch_bounds__(kCacheThreads)
attn_cache_read_kernel(const __grid_constant__ ReadParams p) {
    __shared__ long long s_slot[kReadTokens];  // row in the cache; -1: zeros; -2: leave
    const int side = blockIdx.y;
    const int token0 = blockIdx.x * kReadTokens;
    if (threadIdx.x < kReadTokens) {
        const int token = token0 + threadIdx.x;
        long long slot = -2;
        if (token < p.total) {
            // the last b with cu[b] <= token
            int lo = 0, hi = p.B;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (__ldg(p.cu + mid) <= token) lo = mid;
                else hi = mid - 1;
            }
            if (lo < p.B) {
                const int s = __ldg(p.cu + lo), e = __ldg(p.cu + lo + 1);
                const long long len = (long long)e - s;
                if (s < 0 || e > p.total || len < 0 || len > (long long)p.max_blocks * p.page_size) {
                    atomicOr(p.err, kErrBadSeqlen);
                } else if (token >= s && token < e) {
                    const int pos = token - s;
                    const int blk = pos / p.page_size;
                    const long long page = __ldg(p.block_table + (size_t)lo * p.max_blocks + blk);
                    slot = page >= 0 && page < p.num_blocks
                               ? page * p.page_size + (pos - blk * p.page_size)
                               : -1;
                }
            }
        }
        s_slot[threadIdx.x] = slot;
    }
    __syncthreads();
    constexpr int kCols = E4M3 ? 16 : 8;  // columns of 16 bytes
    const int per_row = p.d / kCols;
    const int per_token = p.Hkv * per_row;
    const uint8_t* pages = p.pages[side];
    const float* descale = p.descale[side];
    TO* out = static_cast<TO*>(p.out[side]);
    const int n = kReadTokens * per_token;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kCacheThreads) {
        const int t = i / per_token;
        const int c = i - t * per_token;
        const long long slot = s_slot[t];
        if (slot == -2) continue;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        float s = 1.0f;
        if (slot >= 0) {
            w = __ldcs(reinterpret_cast<const uint4*>(pages + (slot * per_token + c) * 16));
            if constexpr (E4M3) {
                const int h = c / per_row;
                const long long blk = slot / p.page_size;
                s = __ldg(descale + (blk * p.Hkv + h) * p.page_size + (slot - blk * p.page_size));
            }
        }
        TO* o = out + ((long long)(token0 + t) * per_token + c) * kCols;
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        if constexpr (E4M3) {
            float f[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 a = e4m3x2_f32(ws[j] & 0xFFFFu), b = e4m3x2_f32(ws[j] >> 16);
                f[4 * j] = a.x * s; f[4 * j + 1] = a.y * s;
                f[4 * j + 2] = b.x * s; f[4 * j + 3] = b.y * s;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) store4<TO>(o + 4 * j, f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                store4<TO>(o + 4 * j, bf16lo_to_f32(ws[2 * j]), bf16hi_to_f32(ws[2 * j]),
                           bf16lo_to_f32(ws[2 * j + 1]), bf16hi_to_f32(ws[2 * j + 1]));
        }
    }
}

}  // namespace

attn_status_t launch_cache_write(const void* k, const void* v, const long long* k_strides,
                                 const long long* v_strides, void* k_pages, void* v_pages,
                                 float* k_descale, float* v_descale, const long long* slots, int B,
                                 int N, int Hkv, int d, long long num_blocks, int page_size,
                                 attn_cache_dtype_t cache_dtype, cudaStream_t stream,
                                 const DeviceInfo& dev) {
    WriteParams p;
    auto side = [](const void* x, const long long* st, void* pages, float* descale) {
        WriteSide s;
        s.x = static_cast<const __nv_bfloat16*>(x);
        s.xb = st[0]; s.xh = st[1]; s.xn = st[2];
        s.pages = static_cast<uint8_t*>(pages);
        s.descale = descale;
        return s;
    };
    p.side[0] = side(k, k_strides, k_pages, k_descale);
    p.side[1] = side(v, v_strides, v_pages, v_descale);
    p.slots = slots;
    p.tokens = (long long)B * N;
    p.num_slots = num_blocks * page_size;
    p.N = N;
    p.Hkv = Hkv;
    p.d = d;
    p.page_size = page_size;
    p.err = dev.err_word;
    p.lanes = 1;
    while (p.lanes * 16 < d) p.lanes *= 2;
    const long long rows = (p.tokens + 31) / 32 * 32 * Hkv;
    const long long blocks = (rows * p.lanes + kCacheThreads - 1) / kCacheThreads;
    if (blocks > 0x7FFFFFFFll) return ATTN_ERR_UNSUPPORTED;
    if (cache_dtype == ATTN_CACHE_E4M3)
        attn_cache_write_kernel<true><<<(unsigned)blocks, kCacheThreads, 0, stream>>>(p);
    else
        attn_cache_write_kernel<false><<<(unsigned)blocks, kCacheThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t launch_cache_read(const void* k_pages, const void* v_pages, const float* k_descale,
                                const float* v_descale, const int* block_table,
                                const int* cu_seqlens, void* k_out, void* v_out, int B, int Hkv,
                                int total, long long num_blocks, int page_size, int max_blocks,
                                int d, attn_cache_dtype_t cache_dtype, attn_out_dtype_t out_dtype,
                                cudaStream_t stream, const DeviceInfo& dev) {
    ReadParams p;
    p.pages[0] = static_cast<const uint8_t*>(k_pages);
    p.pages[1] = static_cast<const uint8_t*>(v_pages);
    p.descale[0] = k_descale;
    p.descale[1] = v_descale;
    p.out[0] = k_out;
    p.out[1] = v_out;
    p.block_table = block_table;
    p.cu = cu_seqlens;
    p.num_blocks = num_blocks;
    p.B = B;
    p.Hkv = Hkv;
    p.d = d;
    p.page_size = page_size;
    p.max_blocks = max_blocks;
    p.total = total;
    p.err = dev.err_word;
    const dim3 grid((unsigned)((total + kReadTokens - 1) / kReadTokens), 2u);
    const bool f32 = out_dtype == ATTN_OUT_F32;
    if (cache_dtype == ATTN_CACHE_E4M3) {
        if (f32) attn_cache_read_kernel<true, float><<<grid, kCacheThreads, 0, stream>>>(p);
        else attn_cache_read_kernel<true, __nv_bfloat16><<<grid, kCacheThreads, 0, stream>>>(p);
    } else {
        if (f32) attn_cache_read_kernel<false, float><<<grid, kCacheThreads, 0, stream>>>(p);
        else attn_cache_read_kernel<false, __nv_bfloat16><<<grid, kCacheThreads, 0, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace gb300
