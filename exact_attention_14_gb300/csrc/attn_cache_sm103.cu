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
// Bound: HBM.  Neighbouring lanes move neighbouring 16-byte pieces of the bf16
// side; nothing is staged in shared memory, since no element is used twice.
// Measured, 8 KV heads of 128, call after call on changing inputs: write, 32768 tokens
// to E4M3 (some of them padding), 175 MB in 38.6 us, 4520 GB/s (67% of a plain copy's
// rate: the rows of codes go to scattered places, 128 bytes each; 32 us when the same
// inputs come again, part of which the L2 keeps); to bf16, 230 MB in 41 us, 5620 GB/s;
// read, a 16-sequence cache from E4M3 to bf16, 1.68 GB in 251 us, 6700 GB/s, 99% of the
// copy's rate (with integer divisions for a piece's token and head 291 us).
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
    long long num_slots;
    int tokens, N, Hkv, d, page_size;
    int lanes_log2;        // lanes of a row: 2^, 16 elements each
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

// A block's rows are consecutive tokens of one KV head (blockIdx.y, strided), so
// that the descales of a page are written as whole lines.  A lane holds the
// 8-column chunks c and c + lanes of the K row and of the V row of its token.
template <bool E4M3>
__global__ void __launch_bounds__(kCacheThreads)
attn_cache_write_kernel(const __grid_constant__ WriteParams p) {
    const int lanes = 1 << p.lanes_log2;
    const int c = threadIdx.x & (lanes - 1);
    const int token = blockIdx.x * (kCacheThreads >> p.lanes_log2) + (threadIdx.x >> p.lanes_log2);
    const bool live_token = token < p.tokens;
    long long slot = live_token ? __ldg(p.slots + token) : -1;
    if (slot >= p.num_slots || slot < -1) {
        if (blockIdx.y == 0 && c == 0) atomicOr(p.err, kErrBadSeqlen);
        slot = -1;
    }
    const int col[2] = {8 * c, 8 * (c + lanes)};
    const bool in[2] = {slot >= 0 && col[0] < p.d, slot >= 0 && col[1] < p.d};
    const int b = (int)((unsigned)token / (unsigned)p.N);
    const int n = token - b * p.N;
    long long dsc = 0;  // E4M3: the descale's place for head 0
    if (E4M3 && slot >= 0) {
        long long blk;
        if (slot <= 0x7FFFFFFFll) blk = (long long)((unsigned)slot / (unsigned)p.page_size);
        else blk = slot / p.page_size;
        dsc = blk * p.Hkv * p.page_size + (slot - blk * p.page_size);
    }
    for (int h = blockIdx.y; h < p.Hkv; h += 2 * gridDim.y) {  // two heads' loads in flight
        uint4 w[2][2][2];  // [head][k, v][chunk]
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const WriteSide& sd = p.side[s];
                const int hg = h + g * gridDim.y;
                const __nv_bfloat16* x = sd.x + b * sd.xb + (long long)hg * sd.xh + (long long)n * sd.xn;
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    w[g][s][v] = in[v] && hg < p.Hkv ? __ldcs(reinterpret_cast<const uint4*>(x + col[v]))
                                                     : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int hg = h + g * gridDim.y;
            if (hg >= p.Hkv) break;
            const long long row = (slot * p.Hkv + hg) * p.d;  // first element of the cached row
            if constexpr (!E4M3) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        if (in[v]) *reinterpret_cast<uint4*>(p.side[s].pages + 2 * (row + col[v])) = w[g][s][v];
            } else {
                float m[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    float a = 0.f;
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        a = amax2(a, w[g][s][v].x);
                        a = amax2(a, w[g][s][v].y);
                        a = amax2(a, w[g][s][v].z);
                        a = amax2(a, w[g][s][v].w);
                    }
                    m[s] = a;
                }
                for (int off = lanes >> 1; off > 0; off >>= 1) {
                    m[0] = fmaxf(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], off));
                    m[1] = fmaxf(m[1], __shfl_xor_sync(0xFFFFFFFFu, m[1], off));
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float a = fmaxf(m[s], kTinyAmax);
                    const float scale = m[s] > 0.f ? kE4m3Max / a : 1.0f;
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        if (in[v])
                            *reinterpret_cast<uint2*>(p.side[s].pages + row + col[v]) =
                                make_uint2(quant4(w[g][s][v].x, w[g][s][v].y, scale),
                                           quant4(w[g][s][v].z, w[g][s][v].w, scale));
                    if (c == 0 && slot >= 0)
                        p.side[s].descale[dsc + (long long)hg * p.page_size] = m[s] > 0.f ? a / kE4m3Max : 1.0f;
                }
            }
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
constexpr int kReadFlight = 4;   // pieces of a thread whose loads are in flight

__device__ __forceinline__ float2 e4m3x2_f32(uint32_t pair16) {
    uint32_t h2;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h2) : "r"(pair16));
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h2));
    return f;
}

__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                   pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
}

// a / b for a < 2^25 and a quotient below 2^21, given inv = 1 / b in fp32: the
// estimate is off by less than one.
__device__ __forceinline__ unsigned small_div(unsigned a, unsigned b, float inv) {
    unsigned q = (unsigned)((float)a * inv);
    const int r = (int)(a - q * b);
    if (r < 0) --q;
    else if ((unsigned)r >= b) ++q;
    return q;
}

// A block reads kReadTokens consecutive packed tokens, all heads, K or V
// (blockIdx.y).  The first lanes find each token's sequence by bisection and
// its row in the cache; then every thread streams pieces of 8 columns.
template <bool E4M3, typename TO>
__global__ void __launch_bounds__(kCacheThreads)
attn_cache_read_kernel(const __grid_constant__ ReadParams p) {
    __shared__ long long s_slot[kReadTokens];  // row in the cache; -1: zeros; -2: leave
    __shared__ long long s_descale[kReadTokens];  // its descale's place for head 0
    const int side = blockIdx.y;
    const int token0 = blockIdx.x * kReadTokens;
    if (threadIdx.x < kReadTokens) {
        const int token = token0 + threadIdx.x;
        long long slot = -2, ds = 0;
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
                    const int blk = pos / p.page_size, off = pos - blk * p.page_size;
                    const long long page = __ldg(p.block_table + (size_t)lo * p.max_blocks + blk);
                    if (page >= 0 && page < p.num_blocks) {
                        slot = page * p.page_size + off;
                        ds = page * p.Hkv * p.page_size + off;
                    } else {
                        slot = -1;
                    }
                }
            }
        }
        s_slot[threadIdx.x] = slot;
        s_descale[threadIdx.x] = ds;
    }
    __syncthreads();
    constexpr int kBytes = E4M3 ? 8 : 16;  // of a piece in the cache
    const unsigned per_row = p.d / 8;
    const unsigned per_token = p.Hkv * per_row;
    const uint8_t* pages = p.pages[side];
    const float* descale = p.descale[side];
    TO* out = static_cast<TO*>(p.out[side]);
    const unsigned n = kReadTokens * per_token;
    const float inv_token = 1.0f / (float)per_token, inv_row = 1.0f / (float)per_row;
    for (unsigned i0 = threadIdx.x; i0 < n; i0 += kReadFlight * kCacheThreads) {
        uint4 w[kReadFlight];
        float s[kReadFlight];
        bool put[kReadFlight];
#pragma unroll
        for (int k = 0; k < kReadFlight; ++k) {
            const unsigned i = i0 + k * kCacheThreads;
            w[k] = make_uint4(0u, 0u, 0u, 0u);
            s[k] = 1.0f;
            put[k] = false;
            if (i >= n) continue;
            const unsigned t = small_div(i, per_token, inv_token), c = i - t * per_token;
            const long long slot = s_slot[t];
            put[k] = slot != -2;
            if (slot < 0) continue;
            const uint8_t* src = pages + (slot * per_token + c) * kBytes;
            if constexpr (E4M3) {
                const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
                w[k].x = v.x;
                w[k].y = v.y;
                s[k] = __ldg(descale + s_descale[t] + (long long)small_div(c, per_row, inv_row) * p.page_size);
            } else {
                w[k] = __ldcs(reinterpret_cast<const uint4*>(src));
            }
        }
#pragma unroll
        for (int k = 0; k < kReadFlight; ++k) {
            const unsigned i = i0 + k * kCacheThreads;
            if (!put[k]) continue;
            float f[8];
            if constexpr (E4M3) {
                const float2 a = e4m3x2_f32(w[k].x & 0xFFFFu), b = e4m3x2_f32(w[k].x >> 16);
                const float2 c = e4m3x2_f32(w[k].y & 0xFFFFu), d = e4m3x2_f32(w[k].y >> 16);
                f[0] = a.x * s[k]; f[1] = a.y * s[k]; f[2] = b.x * s[k]; f[3] = b.y * s[k];
                f[4] = c.x * s[k]; f[5] = c.y * s[k]; f[6] = d.x * s[k]; f[7] = d.y * s[k];
            } else {
                f[0] = bf16lo_to_f32(w[k].x); f[1] = bf16hi_to_f32(w[k].x);
                f[2] = bf16lo_to_f32(w[k].y); f[3] = bf16hi_to_f32(w[k].y);
                f[4] = bf16lo_to_f32(w[k].z); f[5] = bf16hi_to_f32(w[k].z);
                f[6] = bf16lo_to_f32(w[k].w); f[7] = bf16hi_to_f32(w[k].w);
            }
            store8(out + ((long long)token0 * per_token + i) * 8, f);
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
    p.tokens = B * N;
    p.num_slots = num_blocks * page_size;
    p.N = N;
    p.Hkv = Hkv;
    p.d = d;
    p.page_size = page_size;
    p.err = dev.err_word;
    p.lanes_log2 = 0;
    while ((16 << p.lanes_log2) < d) ++p.lanes_log2;
    const int per_block = kCacheThreads >> p.lanes_log2;  // tokens
    // a thread walks over up to four heads (its slot is looked up once), fewer
    // where the blocks would not fill the SMs
    const int tiles = (p.tokens + per_block - 1) / per_block;
    int split = Hkv;
    while (split > (Hkv + 3) / 4 && (long long)tiles * ((split + 1) / 2) >= 8ll * dev.num_sms) split = (split + 1) / 2;
    const dim3 blocks((unsigned)tiles, (unsigned)(split < 65535 ? split : 65535));
    if (cache_dtype == ATTN_CACHE_E4M3)
        attn_cache_write_kernel<true><<<blocks, kCacheThreads, 0, stream>>>(p);
    else
        attn_cache_write_kernel<false><<<blocks, kCacheThreads, 0, stream>>>(p);
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
