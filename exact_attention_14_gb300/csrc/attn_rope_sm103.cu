// attn_rope_sm103.cu -- rotary positions on Q and K (and their gradient).
//
// For a token at position pos, pair i of the first `rotary_dim` columns of
// every head turns by theta_i = pos * f_i:
//   (a, b) -> mag * (a cos theta - b sin theta, a sin theta + b cos theta)
// with (a, b) = columns (i, i + rotary_dim/2), or (2i, 2i + 1) when
// interleaved; the other columns are copied.  `inverse` turns by -theta, which
// is the transpose (times mag) and so the gradient.
//
// The angle: f_i in radians becomes a 64-bit fraction of a turn,
// u_i = f_i / (2 pi) mod 1 in units of 2^-64 (fp64 product carried to two
// doubles, once per block), and pos * u_i mod 2^64 is the exact phase of any
// 32-bit position: no range reduction and no loss far into a context.  Its top
// 32 bits give cos and sin through sincospif.
//
// Bound: HBM (each element is read and written once).  A thread keeps the
// cos / sin of its 8 pairs of one token in registers and walks over heads, so
// the angles (about 40 instructions a pair) are shared by all heads it walks.
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnitPairs = 8;   // pairs of one thread
constexpr int kMaxPairs = 128;  // rotary_dim <= 256

enum RopeMode {
    kHalfVec = 0,      // pairs (i, i + r/2), r/2 a multiple of 8: 8 consecutive pairs, 16-byte accesses
    kInterVec = 1,     // pairs (2i, 2i + 1): 16 consecutive columns, 16-byte accesses
    kHalfScalar = 2    // any other r: pairs j, j + P, ...: consecutive lanes on consecutive pairs
};

struct RopeSide {
    const void* x;
    void* out;
    long long xb, xh, xn;  // element strides: batch, head, token
    long long ob, oh, on;
    int H;
};

struct RopeParams {
    RopeSide side[2];  // q, k
    const int* positions;
    long long pos_b;   // positions' batch stride
    const double* inv_freq;
    long long tokens;  // B * N
    int N, d, pairs, units, pair_units;
    int heads, heads_per_thread;
    int inverse;
    float mag;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 8 consecutive elements (16-byte aligned) as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
    v[0] = bf16lo_to_f32(w.x); v[1] = bf16hi_to_f32(w.x);
    v[2] = bf16lo_to_f32(w.y); v[3] = bf16hi_to_f32(w.y);
    v[4] = bf16lo_to_f32(w.z); v[5] = bf16hi_to_f32(w.z);
    v[6] = bf16lo_to_f32(w.w); v[7] = bf16hi_to_f32(w.w);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// f radians as a fraction of a turn in units of 2^-64 (mod 1).  1/(2 pi) is
// held in two doubles, so the product is good to about 2^-100 of its size.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    const double c_hi = 0.15915494309189535, c_lo = -9.839338337591243e-18;
    const double a = fabs(f);  // (the fraction of a negative turn would lose bits)
    const double hi = a * c_hi;
    const double lo = fma(a, c_hi, -hi) + a * c_lo;
    const double two64 = 18446744073709551616.0;
    const double frac = hi - floor(hi);  // in [0, 1), exact
    const unsigned long long u = __double2ull_rn(frac * two64) + (unsigned long long)__double2ll_rn(lo * two64);
    return f < 0.0 ? 0ull - u : u;
}

template <typename TI, typename TO, int MODE>
__global__ void __launch_bounds__(kRopeThreads)
attn_rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ unsigned long long s_turn[kMaxPairs];
    for (int i = threadIdx.x; i < p.pairs; i += kRopeThreads) s_turn[i] = turn_fraction(p.inv_freq[i]);
    __syncthreads();
    const long long at = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
    const long long token = at / p.units;
    if (token >= p.tokens) return;
    const int u = (int)(at - token * p.units);
    const long long b = token / p.N;
    const int n = (int)(token - b * p.N);
    const int h0 = blockIdx.y * p.heads_per_thread;
    const int h1 = min(h0 + p.heads_per_thread, p.heads);
    const int half = p.pairs;
    const bool rotates = u < p.pair_units;

    // cos and sin of this thread's pairs
    float cs[kUnitPairs], sn[kUnitPairs];
    int first = 0, step = 1;  // pair of e: first + step * e
    if (rotates) {
        if constexpr (MODE == kHalfScalar) {
            first = u;
            step = p.pair_units;
        } else {
            first = u * kUnitPairs;
        }
        const unsigned long long pos = (unsigned long long)(long long)p.positions[b * p.pos_b + n];
#pragma unroll
        for (int e = 0; e < kUnitPairs; ++e) {
            const int i = first + step * e;
            cs[e] = 1.f;
            sn[e] = 0.f;
            if (i < half) {
                const unsigned long long phase = pos * s_turn[i];
                // [-1, 1): the angle in units of pi
                const float x = (float)(int)(unsigned)(phase >> 32) * 4.656612873077393e-10f;
                float s, c;
                sincospif(x, &s, &c);
                cs[e] = c * p.mag;
                sn[e] = (p.inverse ? -s : s) * p.mag;
            }
        }
    }
#pragma unroll 2
    for (int h = h0; h < h1; ++h) {
        const bool is_k = h >= p.side[0].H;
        const RopeSide& s = p.side[is_k ? 1 : 0];
        const int hh = is_k ? h - p.side[0].H : h;
        const TI* x = static_cast<const TI*>(s.x) + b * s.xb + (long long)hh * s.xh + (long long)n * s.xn;
        TO* o = static_cast<TO*>(s.out) + b * s.ob + (long long)hh * s.oh + (long long)n * s.on;
        if constexpr (MODE == kHalfScalar) {
            if (rotates) {
                float a[kUnitPairs], c[kUnitPairs];
#pragma unroll
                for (int e = 0; e < kUnitPairs; ++e) {
                    const int i = first + step * e;
                    if (i < half) {
                        a[e] = to_f32(x[i]);
                        c[e] = to_f32(x[i + half]);
                    }
                }
#pragma unroll
                for (int e = 0; e < kUnitPairs; ++e) {
                    const int i = first + step * e;
                    if (i < half) {
                        o[i] = from_f32<TO>(a[e] * cs[e] - c[e] * sn[e]);
                        o[i + half] = from_f32<TO>(a[e] * sn[e] + c[e] * cs[e]);
                    }
                }
            } else {
                for (int i = 2 * half + (u - p.pair_units); i < p.d; i += p.units - p.pair_units)
                    o[i] = from_f32<TO>(to_f32(x[i]));
            }
        } else if (MODE == kHalfVec && rotates) {
            float a[8], c[8], ra[8], rc[8];
            load8(x + first, a);
            load8(x + first + half, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ra[e] = a[e] * cs[e] - c[e] * sn[e];
                rc[e] = a[e] * sn[e] + c[e] * cs[e];
            }
            store8(o + first, ra);
            store8(o + first + half, rc);
        } else {
            // 16 consecutive columns: interleaved pairs, or columns to copy
            const int col = rotates ? 2 * first : 2 * (MODE == kInterVec ? kUnitPairs * p.pair_units : half) +
                                                      16 * (u - p.pair_units);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (col + 8 * v < p.d) {
                    float a[8];
                    load8(x + col + 8 * v, a);
                    if (MODE == kInterVec && rotates) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float c = cs[4 * v + e], sx = sn[4 * v + e];
                            const float r0 = a[2 * e] * c - a[2 * e + 1] * sx;
                            const float r1 = a[2 * e] * sx + a[2 * e + 1] * c;
                            if (first + 4 * v + e < half) {  // pairs past the rotated part stay
                                a[2 * e] = r0;
                                a[2 * e + 1] = r1;
                            }
                        }
                    }
                    store8(o + col + 8 * v, a);
                }
            }
        }
    }
}

template <typename TI, typename TO>
void launch_rope_t(const RopeParams& p, int mode, dim3 grid, cudaStream_t stream) {
    if (mode == kHalfVec)
        attn_rope_kernel<TI, TO, kHalfVec><<<grid, kRopeThreads, 0, stream>>>(p);
    else if (mode == kInterVec)
        attn_rope_kernel<TI, TO, kInterVec><<<grid, kRopeThreads, 0, stream>>>(p);
    else
        attn_rope_kernel<TI, TO, kHalfScalar><<<grid, kRopeThreads, 0, stream>>>(p);
}

}  // namespace

attn_status_t launch_rope(const void* q, const void* k, void* q_out, void* k_out,
                          const long long* q_strides, const long long* k_strides,
                          const long long* q_out_strides, const long long* k_out_strides,
                          const int* positions, long long positions_stride, const double* inv_freq,
                          int B, int Hq, int Hkv, int N, int d, int rotary_dim, int interleaved,
                          int inverse, float magnitude, attn_out_dtype_t in_dtype,
                          attn_out_dtype_t out_dtype, cudaStream_t stream, const DeviceInfo& dev) {
    RopeParams p;
    auto side = [](const void* x, void* out, const long long* xs, const long long* os, int H) {
        RopeSide s;
        s.x = x;
        s.out = out;
        s.xb = xs[0]; s.xh = xs[1]; s.xn = xs[2];
        s.ob = os[0]; s.oh = os[1]; s.on = os[2];
        s.H = H;
        return s;
    };
    p.side[0] = side(q, q_out, q_strides, q_out_strides, Hq);
    p.side[1] = k ? side(k, k_out, k_strides, k_out_strides, Hkv) : p.side[0];
    if (!k) p.side[1].H = 0;
    p.positions = positions;
    p.pos_b = positions_stride;
    p.inv_freq = inv_freq;
    p.tokens = (long long)B * N;
    p.N = N;
    p.d = d;
    p.pairs = rotary_dim / 2;
    p.inverse = inverse;
    p.mag = magnitude;
    p.pair_units = (p.pairs + kUnitPairs - 1) / kUnitPairs;
    const int mode = interleaved ? kInterVec : (p.pairs % 8 == 0 ? kHalfVec : kHalfScalar);
    // columns left to copy, 16 to a unit
    const int rest = mode == kInterVec ? d - 2 * kUnitPairs * p.pair_units : d - rotary_dim;
    p.units = p.pair_units + (rest > 0 ? (rest + 15) / 16 : 0);
    p.heads = Hq + (k ? Hkv : 0);
    // As many heads to a thread as leave about 1024 threads for every SM: the
    // angles are computed once per thread, and a call of few tokens spreads
    // over the heads instead.
    const long long per_head = p.tokens * p.units;
    long long hpt = per_head * p.heads / ((long long)dev.num_sms * 1024);
    hpt = hpt < 1 ? 1 : (hpt > p.heads ? p.heads : hpt);
    const long long groups_min = (p.heads + 65534) / 65535;
    if (hpt < groups_min) hpt = groups_min;
    p.heads_per_thread = (int)hpt;
    const long long blocks = (per_head + kRopeThreads - 1) / kRopeThreads;
    const dim3 grid((unsigned)blocks, (unsigned)((p.heads + hpt - 1) / hpt));
    const bool fi = in_dtype == ATTN_OUT_F32, fo = out_dtype == ATTN_OUT_F32;
    if (fi && fo) launch_rope_t<float, float>(p, mode, grid, stream);
    else if (fi) launch_rope_t<float, __nv_bfloat16>(p, mode, grid, stream);
    else if (fo) launch_rope_t<__nv_bfloat16, float>(p, mode, grid, stream);
    else launch_rope_t<__nv_bfloat16, __nv_bfloat16>(p, mode, grid, stream);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace gb300
