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
// Bound: HBM (each element is read and written once): 671 MB in 108 us, 6210 GB/s,
// 92% of a plain copy's rate, call after call on changing inputs; a single token's call is
// a launch, 3 us on the GPU.  Half pairs whose rotary_dim / 2 is no multiple of a chunk go
// an element at a time (kHalfScalar), since a chunk's partners lie at other alignments:
// the same 671 MB in 222 us (rotary_dim 40) to 248 us (30), fp32's 1342 MB in 246 us (34).
// A thread keeps the
// cos / sin of its 8 pairs of one token in registers and walks over heads, so
// the angles (about 40 instructions a pair) are shared by all heads it walks.
// A row is a list of jobs, two chunks of 16 bytes each: the chunks of a half and
// their partners, then the columns to copy; neighbouring lanes take neighbouring
// jobs.  Two heads' loads are in flight at a time, the first ones during the
// angles.
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnitPairs = 8;   // pairs of one thread
constexpr int kMaxPairs = 128;  // rotary_dim <= 256

enum RopeMode {
    kHalfVec = 0,      // pairs (i, i + r/2), r/2 a multiple of a chunk
    kInterVec = 1,     // pairs (2i, 2i + 1): a job is one chunk
    kHalfScalar = 2    // pairs (i, i + r/2), any other r: chunks of one element
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
    int N, d, pairs;
    int turn_jobs, jobs;  // jobs that turn, and all (the rest copies)
    int units;            // threads of a (token, head)
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

// A chunk of E consecutive elements (16-byte aligned pieces) as it is loaded.
template <typename T, int E>
struct Chunk {
    static constexpr int kWords = E * (int)sizeof(T) / 16;
    uint4 w[kWords];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void get(float (&v)[E]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    v[4 * i + j] = __uint_as_float(u[j]);
                } else {
                    v[8 * i + 2 * j] = bf16lo_to_f32(u[j]);
                    v[8 * i + 2 * j + 1] = bf16hi_to_f32(u[j]);
                }
            }
        }
    }
};
template <int E>
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float (&v)[E]) {
    static_assert(E == 8, "16 bytes of bf16");
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
template <int E>
__device__ __forceinline__ void store_chunk(float* p, const float (&v)[E]) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
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

// An element on its own (chunks of one).
template <typename T>
struct Chunk<T, 1> {
    T w;
    __device__ __forceinline__ void load(const T* p) { w = *p; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f32(w); }
};
template <>
__device__ __forceinline__ void store_chunk<1>(__nv_bfloat16* p, const float (&v)[1]) { *p = from_f32<__nv_bfloat16>(v[0]); }
template <>
__device__ __forceinline__ void store_chunk<1>(float* p, const float (&v)[1]) { *p = v[0]; }

template <typename TI, typename TO, int MODE>
__global__ void __launch_bounds__(kRopeThreads)
attn_rope_kernel(const __grid_constant__ RopeParams p) {
    // columns of a chunk; jobs of a thread; pairs of a job
    constexpr int E = MODE == kHalfScalar ? 1 : (sizeof(TI) == 4 && sizeof(TO) == 4 ? 4 : 8);
    constexpr int kJobPairs = MODE == kInterVec ? E / 2 : E;
    constexpr int kOwn = kUnitPairs / kJobPairs;
    constexpr bool kTwo = MODE != kInterVec;  // a job has a second chunk
    __shared__ unsigned long long s_turn[kMaxPairs];
    for (int i = threadIdx.x; i < p.pairs; i += kRopeThreads) s_turn[i] = turn_fraction(p.inv_freq[i]);
    __syncthreads();
    const long long at = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
    long long token;
    if (at <= 0xFFFFFFFFll) token = (long long)((unsigned)at / (unsigned)p.units);
    else token = at / p.units;
    if (token >= p.tokens) return;
    const int u = (int)(at - token * p.units);
    const int b = (int)((unsigned)token / (unsigned)p.N);  // (tokens <= 2^30)
    const int n = (int)token - b * p.N;
    const int h0 = blockIdx.y * p.heads_per_thread;
    const int h1 = min(h0 + p.heads_per_thread, p.heads);
    const int half = p.pairs, copies = p.jobs - p.turn_jobs;
    // first columns of job v's chunks (second: -1 where there is none); the job turns
    int col[kOwn], col2[kOwn];
    bool turns[kOwn];
#pragma unroll
    for (int v = 0; v < kOwn; ++v) {
        const int k = u + p.units * v, kc = k - p.turn_jobs;
        turns[v] = kc < 0;
        if constexpr (MODE == kInterVec) {
            col[v] = k < p.jobs ? E * k : -1;
            col2[v] = -1;
        } else {
            col[v] = k >= p.jobs ? -1 : (turns[v] ? E * k : 2 * half + E * kc);
            col2[v] = k >= p.jobs ? -1 : (turns[v] ? half + E * k : 2 * half + E * (kc + copies));
            if (col2[v] >= p.d) col2[v] = -1;
        }
    }
    Chunk<TI, E> a[2][kOwn], c[2][kOwn];
    auto load = [&](int h) {  // heads h and h + 1 (the last one again past the end)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int hg = min(h + g, h1 - 1);
            const RopeSide& s = p.side[hg >= p.side[0].H ? 1 : 0];
            const int hh = hg >= p.side[0].H ? hg - p.side[0].H : hg;
            const TI* x = static_cast<const TI*>(s.x) + b * s.xb + (long long)hh * s.xh + (long long)n * s.xn;
#pragma unroll
            for (int v = 0; v < kOwn; ++v) {
                if (col[v] >= 0) a[g][v].load(x + col[v]);
                if (kTwo && col2[v] >= 0) c[g][v].load(x + col2[v]);
            }
        }
    };
    load(h0);
    // cos and sin of this thread's pairs
    float cs[kUnitPairs], sn[kUnitPairs];
    {
        const unsigned long long pos = (unsigned long long)(long long)p.positions[b * p.pos_b + n];
#pragma unroll
        for (int e = 0; e < kUnitPairs; ++e) {
            const int i = kJobPairs * (u + p.units * (e / kJobPairs)) + e % kJobPairs;
            cs[e] = 1.f;
            sn[e] = 0.f;
            if (i < half) {
                const unsigned long long phase = pos * s_turn[i];
                // [-1, 1): the angle in units of pi
                const float x = (float)(int)(unsigned)(phase >> 32) * 4.656612873077393e-10f;
                float s, co;
                sincospif(x, &s, &co);
                cs[e] = co * p.mag;
                sn[e] = (p.inverse ? -s : s) * p.mag;
            }
        }
    }
    for (int h = h0; h < h1; h += 2) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            if (h + g >= h1) break;
            const RopeSide& s = p.side[h + g >= p.side[0].H ? 1 : 0];
            const int hh = h + g >= p.side[0].H ? h + g - p.side[0].H : h + g;
            TO* o = static_cast<TO*>(s.out) + b * s.ob + (long long)hh * s.oh + (long long)n * s.on;
#pragma unroll
            for (int v = 0; v < kOwn; ++v) {
                if (col[v] < 0) continue;
                float x0[E], x1[E], y0[E], y1[E];
                a[g][v].get(x0);
                if constexpr (kTwo) {
                    c[g][v].get(x1);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float co = cs[v * kJobPairs + e], si = sn[v * kJobPairs + e];
                        y0[e] = turns[v] ? x0[e] * co - x1[e] * si : x0[e];
                        y1[e] = turns[v] ? x0[e] * si + x1[e] * co : x1[e];
                    }
                    if (col2[v] >= 0) store_chunk<E>(o + col2[v], y1);
                } else {
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        const float co = cs[v * kJobPairs + e], si = sn[v * kJobPairs + e];
                        const bool in = col[v] / 2 + e < half;
                        y0[2 * e] = in ? x0[2 * e] * co - x0[2 * e + 1] * si : x0[2 * e];
                        y0[2 * e + 1] = in ? x0[2 * e] * si + x0[2 * e + 1] * co : x0[2 * e + 1];
                    }
                }
                store_chunk<E>(o + col[v], y0);
            }
        }
        if (h + 2 < h1) load(h + 2);
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
    const bool f32 = in_dtype == ATTN_OUT_F32 && out_dtype == ATTN_OUT_F32;
    const int chunk = f32 ? 4 : 8;  // columns (the kernel's E)
    const int mode = interleaved ? kInterVec : (p.pairs % chunk == 0 ? kHalfVec : kHalfScalar);
    if (mode == kInterVec) {
        p.jobs = d / chunk;
        p.turn_jobs = p.jobs;  // (pairs past the rotated part stay as they are)
        p.units = (p.jobs + 16 / chunk - 1) / (16 / chunk);
    } else {
        const int e = mode == kHalfVec ? chunk : 1;
        p.turn_jobs = p.pairs / e;
        p.jobs = p.turn_jobs + ((d - rotary_dim) / e + 1) / 2;
        p.units = (p.jobs + kUnitPairs / e - 1) / (kUnitPairs / e);
    }
    p.heads = Hq + (k ? Hkv : 0);
    // Up to 8 heads to a thread (their angles are computed once), fewer where that
    // leaves less than 1024 threads for every SM: a call of few tokens spreads over
    // the heads instead.  (40 heads, 32768 tokens, 671 MB, replayed in a graph: all heads on
    // one thread 123 us, 16 heads 106.5, 8 heads 105.4, 4 heads 109.)
    const long long per_head = p.tokens * p.units;
    long long hpt = per_head * p.heads / ((long long)dev.num_sms * 1024);
    hpt = hpt < 1 ? 1 : (hpt > 8 ? 8 : hpt);
    if (hpt > p.heads) hpt = p.heads;
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
