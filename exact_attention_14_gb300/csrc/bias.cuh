// bias.cuh -- the learned relative position bias as the attention kernels read it.
//
// The bias of query head h at relative distance r = (key) - (query + Nk - Nq) is
// table[buckets[clamp(r - first, 0, span - 1)], h]: the map lists the distances
// first .. first + span - 1, and farther ones count as its ends.  The kernels
// hold it times log2(e), since their scores are in base 2.
//
// A tile of 128 query rows and 128 keys meets 255 distances, base .. base + 254: a
// window of 256 floats in shared memory, one per distance, that a warp of its own
// fills: there are two, so the next tile's is full while one is in use, and the biases
// of the tile after it are on their way to registers.
// Forward: where all distances lie on one side of the map (or at its end) the whole
// tile has one bias, which costs a term of the exponent that is there anyway; other
// tiles take theirs from the window.  Lanes of a warp hold consecutive rows, so a
// column's 32 reads are 32 consecutive floats: no bank conflict.
// Backward: always from the window, on MMA-like fragments of which a thread's 64
// elements meet 22 distances (pds_tile_bias).
// Decode: a thread looks up its own 4 keys x 2 heads.
#pragma once

#include <climits>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace gb300 {

struct BiasArgs {
    const void* table;   // [num_buckets, Hq], fp32 or bf16
    const int* buckets;  // [span]
    int first, span, num_buckets, bf16;
};

constexpr int kBiasWindow = 256;         // floats of one tile's window
constexpr float kBiasLog2e = 1.44269504088896340736f;
// A bias below this (-1e9, a type's lowest value: masks) counts as -inf: its key is
// left out.  Were a whole row at -1e9, the backward's P = 2^(score + bias - LSE) would
// be the rounding of LSE (64 there) to the power of 2, infinite or 0; at 1e6 that rounding is
// below 2^0.5.
constexpr float kBiasMasked = -1e6f;

// Biases of head h at the distances r, r + 32, ..., times log2(e); -inf for those above
// `last` (causal masking is a bias of -inf at every distance above 0, so a window
// masks by itself).  A bucket outside the table adds nothing and is recorded in the
// error word.  Every bucket is fetched
// before the first table entry: two waits for memory, however many there are.
template <int N>
__device__ __forceinline__ void bias_at(const BiasArgs& a, int Hq, int h, int r, int last, float (&v)[N], unsigned int* err) {
    int bk[N];
    bool bad = false;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = r + 32 * n - a.first;
        bk[n] = __ldg(a.buckets + min(max(i, 0), a.span - 1));
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const bool ok = (unsigned)bk[n] < (unsigned)a.num_buckets;
        const size_t at = (size_t)(ok ? bk[n] : 0) * Hq + h;
        const float x = a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.table)[at])
                               : __ldg(static_cast<const float*>(a.table) + at);
        v[n] = r + 32 * n > last || (ok && x < kBiasMasked) ? -INFINITY : ok ? x * kBiasLog2e : 0.f;
        bad |= !ok;
    }
    if (bad) atomicOr(err, kErrBadSeqlen);
}
// The decode's: heads h0 (v[n][0], v[n][1]) and h1 (v[n][2], v[n][3]) at the distances
// r + 8 n and r + 8 n + 1, n < 2.
__device__ __forceinline__ void bias_at(const BiasArgs& a, int Hq, int h0, int h1, int r, float (&v)[2][4],
                                        unsigned int* err) {
    int bk[4];
    bool bad = false;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const int i = r + 8 * (n >> 1) + (n & 1) - a.first;
        bk[n] = __ldg(a.buckets + min(max(i, 0), a.span - 1));
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const bool ok = (unsigned)bk[n] < (unsigned)a.num_buckets;
        const size_t row = (size_t)(ok ? bk[n] : 0) * Hq;
        bad |= !ok;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const size_t at = row + (e ? h1 : h0);
            const float x = a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.table)[at])
                                   : __ldg(static_cast<const float*>(a.table) + at);
            v[n >> 1][2 * e + (n & 1)] = ok && x < kBiasMasked ? -INFINITY : ok ? x * kBiasLog2e : 0.f;
        }
    }
    if (bad) atomicOr(err, kErrBadSeqlen);
}
__device__ __forceinline__ float bias_at(const BiasArgs& a, int Hq, int h, int r, unsigned int* err) {
    float v[1];
    bias_at(a, Hq, h, r, INT_MAX, v, err);
    return v[0];
}

// Whether the 255 distances from `base` on need a window: some of them lie strictly
// inside the map.  Otherwise all of them have the bias of its left end (base + 254
// <= first) or of its right one.
__device__ __forceinline__ bool bias_near(const BiasArgs& a, int base) {
    return base + 254 > a.first && base < a.first + a.span - 1;
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ float2 lds64_f32(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

}  // namespace gb300
