// attn_tree_sm103.cu -- attention of the drafted tokens of each sequence (a
// tree, a chain, or a single token) over a paged KV cache, bf16 or E4M3.
//
// Row (t, g) of sequence b and KV head h is drafted token t, query head
// h * G + g.  It attends every key before the drafted ones, and drafted token
// u (key keys - drafted + u) iff its mask says so:
//   s_j = scale * q . k_j,  O = sum_j softmax(s)_j v_j,  LSE = log sum_j e^{s_j}.
// E4M3 rows stand for code * descale: s_j = scale * kd_j (q . kc_j) and
// O = sum_j p_j vd_j vc_j / sum_j p_j, the codes exact in fp16.
//
// This file: the kernel for 16 query rows at a time on mma.sync (m16n8k16;
// more rows of head dims up to 128 go to attn_tree_tc_sm103.cu), and the merge of cut items (tree_plan.h has the work list).  A producer warp
// streams 64-key tiles of K and V (and their descales) by TMA into a ring; each
// of four consumer warps takes 16 keys of every tile with its own online
// softmax (base 2), and the four are merged through shared memory at the end of
// a piece.  Bound: HBM (each cached byte is read once per row tile).
//
// E4M3 fragments: a lane takes 16 consecutive code bytes of a key with one
// shared load and spreads them over four k-steps (Q is laid out to match), so
// K needs no transposition.  V^T needs four keys' codes of one column in a
// register: four 16-byte rows are transposed with byte permutes.  P multiplies
// vd_j / F in fp16, F the power of two above the largest vd seen so far (O is
// rescaled when F grows), times 2^15: weights down to 2^-29 of the largest keep
// fp16's 11 bits.  bf16 caches use bf16 P, as the library's decode does.
//
// Masked places: scores are selected, never added to.  V rows past the
// sequence are zeroed in shared memory; a drafted token's V row that holds a
// NaN or an infinity is taken out of the product (0 * NaN would reach the rows
// that do not see it) and added to the rows that do see it by itself.
#include <cmath>
#include <cstdint>

#include "tree_plan.h"

namespace gb300 {
namespace {

constexpr int kConsumers = 4;
constexpr int kTreeThreads = (kConsumers + 1) * 32;
constexpr int kTileKeys = 64;
constexpr int kRows = 16;
constexpr float kLn2t = 0.69314718055994530942f;
constexpr float kLog2et = 1.44269504088896340736f;
constexpr float kPFrame = 32768.0f;  // E4M3: P is held times 2^15 / F

template <int D, bool F8>
struct TreeCfg {
    // bytes of a 64-key K (or V) tile: 128-byte-wide swizzled boxes
    static constexpr int kBoxes = F8 ? D / 128 : D / 64;
    static constexpr int kHalf = kBoxes * kTileKeys * 128;
    static constexpr int kDescale = F8 ? 2 * kTileKeys * 4 : 0;  // kd, vd of a tile
    static constexpr int kStage = 2 * kHalf + (F8 ? 1024 : 0);   // (tiles stay 1024-byte aligned)
    static constexpr int kStages = D <= 128 ? (F8 ? 5 : 3) : (F8 ? 5 : 3);
    static constexpr int kScratch = kStages * kStage;            // O of two warps
    static constexpr int kScratchBytes = 2 * kRows * D * 4;
    static constexpr int kBar = kScratch + kScratchBytes;
    static constexpr int kSmem = kBar + 1024;
};

struct TreeBars {
    uint64_t full[5], empty[5];
    TreeRange range;
    int abort;
    float m[kConsumers][kRows], l[kConsumers][kRows], x[kConsumers][kRows], f[kConsumers];
};
static_assert(sizeof(TreeBars) <= 1024, "barrier block");

__device__ __forceinline__ void tree_consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}
// Whether any consumer says so (every consumer warp gets here: all leave together).
__device__ __forceinline__ bool tree_consumers_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(kConsumers * 32)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(a));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float lds32f(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two E4M3 codes (low and high byte of a 16-bit half) as two fp16.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ float e4m3_f32(uint32_t code) {
    uint32_t r = e4m3_lo(code & 0xFFu);
    float f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(r));
    return f;
}
// Power of two 2^e (e in [-126, 127]).
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Byte offset of 16-byte chunk `ch` (counted over the whole row) of key row
// `key` in a tile of 64-key, 128-byte-wide swizzled boxes.
__device__ __forceinline__ uint32_t tile_off(int key, int ch) {
    return (uint32_t)((ch >> 3) * (kTileKeys * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
}

// Whether a 16-byte piece of a V row holds a NaN or an infinity.
template <bool F8>
__device__ __forceinline__ bool not_finite(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool hit = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) hit |= ((w[i] >> (8 * j)) & 0x7Fu) == 0x7Fu;
        } else {
            hit |= (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
        }
    }
    return hit;
}

template <int D, bool F8>
__device__ __forceinline__ void produce(const CUtensorMap* tk, const CUtensorMap* tv, uint8_t* smem,
                                        TreeBars* bars, const TreeParams& p) {
    using C = TreeCfg<D, F8>;
    const volatile int* abort_flag = &bars->abort;
    TreeWalk walk;
    walk.start(bars->range);
    TreePiece w;
    long long issued = 0;
    bool ok = true;
    const int boxes = kTileKeys / p.box_keys;
    while (ok && walk.next(p, w)) {
        for (int kt = w.k0; kt < w.k1; ++kt, ++issued) {
            const int slot = (int)(issued % C::kStages);
            const long long round = issued / C::kStages;
            if (round > 0) {
                ok = mbar_wait(smem_u32(&bars->empty[slot]), (uint32_t)((round - 1) & 1), abort_flag);
                if (!ok) break;
            }
            const uint32_t bar = smem_u32(&bars->full[slot]);
            mbar_arrive_expect_tx(bar, 2 * C::kHalf + C::kDescale);
            const uint32_t dk = smem_u32(smem + slot * C::kStage);
            const uint32_t dv = dk + C::kHalf;
            for (int x = 0; x < boxes; ++x) {
                int off;
                const int page = tree_page(p, w.b, kt * kTileKeys + x * p.box_keys, w.keys, off);
#pragma unroll
                for (int c = 0; c < C::kBoxes; ++c) {
                    const uint32_t to = c * (kTileKeys * 128) + x * p.box_keys * 128;
                    tma_load_4d(dk + to, tk, bar, (F8 ? 128 : 64) * c, w.h, off, page);
                    tma_load_4d(dv + to, tv, bar, (F8 ? 128 : 64) * c, w.h, off, page);
                }
                if constexpr (F8) {
                    // a missing page's codes are zeros: any descale that exists will do
                    const long long at = ((long long)(page < 0 ? 0 : page) * p.Hkv + w.h) * p.page_size + off;
                    const uint32_t ds = dk + 2 * C::kHalf + x * p.box_keys * 4;
                    bulk_load(ds, p.k_descale + at, p.box_keys * 4, bar);
                    bulk_load(ds + kTileKeys * 4, p.v_descale + at, p.box_keys * 4, bar);
                }
            }
        }
    }
    if (!ok) {
        atomicOr(p.err, kErrTimeout);
        *((volatile int*)&bars->abort) = 1;
    }
    // every issued copy lands before the CTA may leave
    for (int slot = 0; slot < C::kStages && slot < issued; ++slot) {
        const long long n = (issued - slot + C::kStages - 1) / C::kStages;
        mbar_wait(smem_u32(&bars->full[slot]), (uint32_t)((n - 1) & 1), nullptr);
    }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kTreeThreads, D <= 128 ? 2 : 1)
attn_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ TreeParams p) {
    using C = TreeCfg<D, F8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    TreeBars* bars = reinterpret_cast<TreeBars*>(smem + C::kBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {  // the swizzled boxes need 1024-byte bases
        if (threadIdx.x == 0) atomicOr(p.err, kErrLayout);
        return;
    }
    if (warp == 0) {
        const TreeRange r = tree_range(p, blockIdx.x);
        if (lane == 0) bars->range = r;
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&bars->full[i]), 1);
            mbar_init(smem_u32(&bars->empty[i]), kConsumers);
        }
        bars->abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (warp == kConsumers) {
        if (lane == 0) produce<D, F8>(&tk, &tv, smem, bars, p);
        return;
    }

    const volatile int* abort_flag = &bars->abort;
    const int qr = lane >> 2, qc = lane & 3;
    const int mi = lane >> 3, ri = lane & 7;
    const int wk0 = warp * 16;
    // key (of this warp's 16) and column of an accumulator element
    auto key_of = [&](int nt, int e) { return F8 ? nt * 8 + qc + 4 * (e & 1) : nt * 8 + 2 * qc + (e & 1); };
    auto col_of = [&](int i, int e) {
        return F8 ? (i >> 4) * 128 + 64 * (e & 1) + 16 * qc + (i & 15) : i * 8 + 2 * qc + (e & 1);
    };
    float* so = reinterpret_cast<float*>(smem + C::kScratch);
    TreeWalk walk;
    walk.start(bars->range);
    TreePiece w;
    long long used = 0;
    bool ok = true, first_piece = true;
    while (ok && walk.next(p, w)) {
        const int rows = min(kRows, w.drafted * p.G - w.rt * kRows);  // >= 1
        const int prefix = w.keys - w.drafted;
        int tok[2];
        const __nv_bfloat16* qrow[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = w.rt * kRows + min(qr + 8 * r, rows - 1);
            tok[r] = row / p.G;
            qrow[r] = p.q + (((size_t)w.b * p.Hq + (size_t)w.h * p.G + (row - tok[r] * p.G)) * p.T + tok[r]) * p.dh;
        }
        // ---- Q fragments (rows past the last repeat it; never written)
        uint32_t qa[D / 16][4];
        float qs[2] = {p.c, p.c};  // what a product is multiplied with
        if constexpr (!F8) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int c0 = ks * 16 + 2 * qc + 8 * hf;
                        qa[ks][r + 2 * hf] = c0 < p.dh ? *reinterpret_cast<const uint32_t*>(qrow[r] + c0) : 0u;
                    }
        } else {
            // fp16, each row scaled by a power of two that puts its largest value
            // in [2^14, 2^15): exact but for values below 2^-38 of it
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const int c0 = (ks >> 2) * 64 + 16 * qc + 4 * (ks & 3);
                    const uint2 v = c0 < p.dh ? *reinterpret_cast<const uint2*>(qrow[r] + c0) : make_uint2(0u, 0u);
                    qa[ks][r] = v.x;
                    qa[ks][r + 2] = v.y;
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(bf16lo_to_f32(v.x)), fabsf(bf16hi_to_f32(v.x))),
                                         fmaxf(fabsf(bf16lo_to_f32(v.y)), fabsf(bf16hi_to_f32(v.y)))));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                int e = (int)(__float_as_uint(mx) >> 23) - 127;
                e = e < -100 ? -100 : (e > 126 ? 126 : e);
                const float up = pow2i(14 - e);
                qs[r] = p.c * pow2i(e - 14);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qa[ks][r] = pack_f16x2(bf16lo_to_f32(qa[ks][r]) * up, bf16hi_to_f32(qa[ks][r]) * up);
                    qa[ks][r + 2] = pack_f16x2(bf16lo_to_f32(qa[ks][r + 2]) * up, bf16hi_to_f32(qa[ks][r + 2]) * up);
                }
            }
        }
        float acc[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY};
        float l[2] = {0.f, 0.f};  // this lane's part of the sum that normalises O
        float xs[2] = {0.f, 0.f};  // ... of the unrounded P (the LSE's)
        int fexp = -126;           // E4M3: F = 2^fexp

        for (int kt = w.k0; kt < w.k1; ++kt, ++used) {
            const int slot = (int)(used % C::kStages);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&bars->full[slot]),
                                                   (uint32_t)((used / C::kStages) & 1), abort_flag));
            if (!ok) break;
            const int key0 = kt * kTileKeys + wk0;          // this warp's first key
            const int nvalid = min(16, w.keys - key0);
            const uint32_t sK = smem_u32(smem + slot * C::kStage);
            const uint32_t sV = sK + C::kHalf;
            bool wrote = false;
            if (nvalid > 0) {
                // ---- S
                float sf[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                float vd[2][2];  // E4M3: V's descale of this lane's keys
                if constexpr (!F8) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        uint32_t b0, b1, b2, b3;
                        ldsm4(sK + tile_off(wk0 + (mi >> 1) * 8 + ri, ks * 2 + (mi & 1)), b0, b1, b2, b3);
                        mma16816<false>(sf[0], qa[ks], b0, b1);
                        mma16816<false>(sf[1], qa[ks], b2, b3);
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const int key = wk0 + nt * 8 + (qr >> 1) + 4 * (qr & 1);
#pragma unroll
                        for (int blk = 0; blk < D / 64; ++blk) {
                            const uint4 kb = lds128(sK + tile_off(key, blk * 4 + qc));
                            mma16816<true>(sf[nt], qa[4 * blk], e4m3_lo(kb.x), e4m3_hi(kb.x));
                            mma16816<true>(sf[nt], qa[4 * blk + 1], e4m3_lo(kb.y), e4m3_hi(kb.y));
                            mma16816<true>(sf[nt], qa[4 * blk + 2], e4m3_lo(kb.z), e4m3_hi(kb.z));
                            mma16816<true>(sf[nt], qa[4 * blk + 3], e4m3_lo(kb.w), e4m3_hi(kb.w));
                        }
                    }
                }
                // ---- scale, mask, running maximum
                const bool drafted = key0 + nvalid > prefix;  // some of the keys are drafted tokens
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int kk = key_of(nt, e);
                        float f = qs[e >> 1];
                        if constexpr (F8) {
                            const uint32_t at = sK + 2 * C::kHalf + (wk0 + kk) * 4;
                            f *= lds32f(at);
                            if (e < 2) vd[nt][e] = kk < nvalid ? lds32f(at + kTileKeys * 4) : 0.f;
                        }
                        float v = kk < nvalid ? sf[nt][e] * f : -INFINITY;
                        if (drafted && kk < nvalid && key0 + kk >= prefix &&
                            !tree_sees(p, w.b, tok[e >> 1], key0 + kk - prefix))
                            v = -INFINITY;
                        sf[nt][e] = v;
                        mx[e >> 1] = fmaxf(mx[e >> 1], v);
                    }
                float al[2], ms[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 1));
                    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 2));
                    const float mn = fmaxf(m[r], mx[r]);
                    ms[r] = mn == -INFINITY ? 0.f : mn;  // (no key yet: every P is 0)
                    al[r] = ex2(m[r] - ms[r]);
                    m[r] = mn;
                }
                // ---- V rows that must not enter the product
                unsigned bad = 0u;  // of the 16 keys: drafted rows with a NaN or an infinity
                if (drafted) {
                    for (int i = lane; i < 16 * (F8 ? D / 16 : D / 8); i += 32) {
                        const int kk = i & 15;
                        if (kk < nvalid && key0 + kk >= prefix &&
                            not_finite<F8>(lds128(sV + tile_off(wk0 + kk, i >> 4))))
                            bad |= 1u << kk;
                    }
                    if constexpr (F8) {
                        if (lane < nvalid && key0 + lane >= prefix &&
                            !isfinite(lds32f(sK + 2 * C::kHalf + kTileKeys * 4 + (wk0 + lane) * 4)))
                            bad |= 1u << lane;
                    }
                    bad = __reduce_or_sync(0xFFFFFFFFu, bad);
                }
                // ---- P
                float add[2] = {0.f, 0.f}, addx[2] = {0.f, 0.f};
                uint32_t pa[4];
                float grow = 1.f;  // E4M3: F_old / F_new
                float wv[2][2];
                if constexpr (F8) {
                    float top = 0.f;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (bad >> key_of(nt, e) & 1u) wv[nt][e] = 0.f;
                            else wv[nt][e] = vd[nt][e];
                            top = fmaxf(top, fabsf(wv[nt][e]));
                        }
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    // 2^need > top (all rows of the quad's keys: the same in every lane)
                    const int need = max(min((int)(__float_as_uint(top) >> 23) - 126, 111), -100);
                    if (need > fexp) {
                        grow = fexp <= -126 ? 0.f : (fexp - need < -126 ? 0.f : pow2i(fexp - need));
                        fexp = need;
                    }
                    const float fr = kPFrame * pow2i(-fexp);
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) wv[nt][e] *= fr;
                }
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    float pr[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pr[e] = ex2(sf[nt][e] - ms[e >> 1]);
                        addx[e >> 1] += pr[e];
                    }
                    if constexpr (F8) {
                        pa[2 * nt] = pack_f16x2(pr[0] * wv[nt][0], pr[1] * wv[nt][1]);
                        pa[2 * nt + 1] = pack_f16x2(pr[2] * wv[nt][0], pr[3] * wv[nt][1]);
                    } else {
                        pa[2 * nt] = pack_bf16x2(pr[0], pr[1]);
                        pa[2 * nt + 1] = pack_bf16x2(pr[2], pr[3]);
                        add[0] += bf16lo_to_f32(pa[2 * nt]) + bf16hi_to_f32(pa[2 * nt]);
                        add[1] += bf16lo_to_f32(pa[2 * nt + 1]) + bf16hi_to_f32(pa[2 * nt + 1]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    xs[r] = xs[r] * al[r] + addx[r];
                    l[r] = l[r] * al[r] + (F8 ? addx[r] : add[r]);
                }
                const float o0 = al[0] * grow, o1 = al[1] * grow;
                if (!__all_sync(0xFFFFFFFFu, o0 == 1.f && o1 == 1.f)) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        acc[i][0] *= o0;
                        acc[i][1] *= o0;
                        acc[i][2] *= o1;
                        acc[i][3] *= o1;
                    }
                }
                // ---- rows past the sequence, and rows with a NaN or an infinity:
                // the latter are added to the rows that see them, both are zeroed
                if (bad) {
                    for (unsigned left = bad; left; left &= left - 1) {
                        const int kk = __ffs(left) - 1;
                        const int nt = kk >> 3;
                        // who holds its P: accumulator column of the key
                        const int owner = F8 ? (kk & 3) : ((kk & 7) >> 1);
                        const int el = F8 ? (kk & 7) >> 2 : kk & 1;
                        float sv[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float mine = nt == 0 ? (el == 0 ? sf[0][2 * r] : sf[0][2 * r + 1])
                                                       : (el == 0 ? sf[1][2 * r] : sf[1][2 * r + 1]);
                            sv[r] = __shfl_sync(0xFFFFFFFFu, mine, (lane & ~3) | owner);
                        }
                        float fr = 1.f;
                        if constexpr (F8)
                            fr = lds32f(sK + 2 * C::kHalf + kTileKeys * 4 + (wk0 + kk) * 4) * kPFrame * pow2i(-fexp);
#pragma unroll
                        for (int i = 0; i < D / 8; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int col = col_of(i, e);
                                float v;
                                if constexpr (F8) {
                                    const uint32_t at = sV + tile_off(wk0 + kk, col >> 4) + (col & 15);
                                    uint32_t byte;
                                    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(at));
                                    v = e4m3_f32(byte) * fr;
                                } else {
                                    const uint32_t at = sV + tile_off(wk0 + kk, col >> 3) + 2 * (col & 7);
                                    uint32_t half;
                                    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(half) : "r"(at));
                                    v = __uint_as_float(half << 16);
                                }
                                if (sv[0] != -INFINITY) acc[i][e] = fmaf(ex2(sv[0] - ms[0]), v, acc[i][e]);
                                if (sv[1] != -INFINITY) acc[i][2 + e] = fmaf(ex2(sv[1] - ms[1]), v, acc[i][2 + e]);
                            }
                    }
                    __syncwarp();
                }
                const unsigned zero = bad | (nvalid < 16 ? (0xFFFFu << nvalid) & 0xFFFFu : 0u);
                if (zero) {
                    for (int i = lane; i < 16 * (F8 ? D / 16 : D / 8); i += 32)
                        if (zero >> (i & 15) & 1u) sts128(sV + tile_off(wk0 + (i & 15), i >> 4), 0u, 0u, 0u, 0u);
                    wrote = true;
                    __syncwarp();
                }
                // ---- O += P V
                if constexpr (!F8) {
#pragma unroll
                    for (int pr = 0; pr < D / 16; ++pr) {
                        uint32_t v0, v1, v2, v3;
                        ldsm4_t(sV + tile_off(wk0 + (mi & 1) * 8 + ri, pr * 2 + (mi >> 1)), v0, v1, v2, v3);
                        mma16816<false>(acc[2 * pr], pa, v0, v1);
                        mma16816<false>(acc[2 * pr + 1], pa, v2, v3);
                    }
                } else {
                    // P's k index 2 qc + {0, 1, 8, 9} is key qc + {0, 4, 8, 12}; B's
                    // column qr is chunk (qr >> 1) + 4 (qr & 1) of the 128 columns
                    const int ch = (qr >> 1) + 4 * (qr & 1);
#pragma unroll
                    for (int hf = 0; hf < D / 128; ++hf) {
                        const uint4 r0 = lds128(sV + tile_off(wk0 + qc, hf * 8 + ch));
                        const uint4 r1 = lds128(sV + tile_off(wk0 + qc + 4, hf * 8 + ch));
                        const uint4 r2 = lds128(sV + tile_off(wk0 + qc + 8, hf * 8 + ch));
                        const uint4 r3 = lds128(sV + tile_off(wk0 + qc + 12, hf * 8 + ch));
                        const uint32_t a0[4] = {r0.x, r0.y, r0.z, r0.w}, a1[4] = {r1.x, r1.y, r1.z, r1.w};
                        const uint32_t a2[4] = {r2.x, r2.y, r2.z, r2.w}, a3[4] = {r3.x, r3.y, r3.z, r3.w};
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const uint32_t x01 = __byte_perm(a0[g], a1[g], 0x5140), y01 = __byte_perm(a0[g], a1[g], 0x7362);
                            const uint32_t x23 = __byte_perm(a2[g], a3[g], 0x5140), y23 = __byte_perm(a2[g], a3[g], 0x7362);
                            mma16816<true>(acc[16 * hf + 4 * g], pa, e4m3_lo(x01), e4m3_lo(x23));
                            mma16816<true>(acc[16 * hf + 4 * g + 1], pa, e4m3_hi(x01), e4m3_hi(x23));
                            mma16816<true>(acc[16 * hf + 4 * g + 2], pa, e4m3_lo(y01), e4m3_lo(y23));
                            mma16816<true>(acc[16 * hf + 4 * g + 3], pa, e4m3_hi(y01), e4m3_hi(y23));
                        }
                    }
                }
            }
            if (wrote) fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->empty[slot]));
        }
        if (tree_consumers_any(!ok)) {
            ok = false;
            break;
        }
        // ---- merge the four warps: sums over the quad, then the warps' maxima
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
            xs[r] += __shfl_xor_sync(0xFFFFFFFFu, xs[r], 1);
            xs[r] += __shfl_xor_sync(0xFFFFFFFFu, xs[r], 2);
            if (qc == 0) {
                bars->m[warp][qr + 8 * r] = m[r];
                bars->l[warp][qr + 8 * r] = l[r];
                bars->x[warp][qr + 8 * r] = xs[r];
            }
        }
        if (lane == 0) bars->f[warp] = F8 ? pow2i(max(fexp, -120)) / kPFrame : 1.f;
        tree_consumers_sync();
        float M[2], sum[2] = {0.f, 0.f}, sumx[2] = {0.f, 0.f}, mine[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = qr + 8 * r;
            M[r] = fmaxf(fmaxf(bars->m[0][row], bars->m[1][row]), fmaxf(bars->m[2][row], bars->m[3][row]));
            const float Ms = M[r] == -INFINITY ? 0.f : M[r];
#pragma unroll
            for (int x = 0; x < kConsumers; ++x) {
                const float wt = ex2(bars->m[x][row] - Ms);
                sum[r] += wt * bars->l[x][row];
                sumx[r] += wt * bars->x[x][row];
            }
            mine[r] = ex2(m[r] - Ms) * bars->f[warp];
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            acc[i][0] *= mine[0];
            acc[i][1] *= mine[0];
            acc[i][2] *= mine[1];
            acc[i][3] *= mine[1];
        }
        // O of warps 2, 3 to warps 0, 1, then of warp 1 to warp 0 (lane by lane)
#pragma unroll 1
        for (int from = 2; from >= 1; from >>= 1) {
            float* buf = so + (size_t)((warp & (from - 1)) * 32 + lane) * 2;
            if (warp >= from && warp < 2 * from) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    *reinterpret_cast<float2*>(buf + (2 * i) * 128) = make_float2(acc[i][0], acc[i][1]);
                    *reinterpret_cast<float2*>(buf + (2 * i + 1) * 128) = make_float2(acc[i][2], acc[i][3]);
                }
            }
            tree_consumers_sync();
            if (warp < from) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float2 a = *reinterpret_cast<const float2*>(buf + (2 * i) * 128);
                    const float2 b = *reinterpret_cast<const float2*>(buf + (2 * i + 1) * 128);
                    acc[i][0] += a.x;
                    acc[i][1] += a.y;
                    acc[i][2] += b.x;
                    acc[i][3] += b.y;
                }
            }
            tree_consumers_sync();
        }
        if (warp == 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = qr + 8 * r;
                if (row >= rows) continue;
                const float inv = sum[r] == 0.f ? 0.f : 1.0f / sum[r];
                const float lse2 = sumx[r] == 0.f ? -INFINITY : M[r] + log2f(sumx[r]);
                const size_t bht = (size_t)(qrow[r] - p.q) / p.dh;  // (b, hq, t)
                const size_t place = ((size_t)blockIdx.x * 2 + (first_piece ? 0 : 1)) * kRows + row;
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int col = col_of(i, e);
                        const float v = acc[i][2 * r + e] * inv;
                        if (!w.whole) p.ws_o[place * D + col] = v;
                        else if (col < p.dh) {
                            if (p.out_f32) static_cast<float*>(p.o)[bht * p.dh + col] = v;
                            else static_cast<__nv_bfloat16*>(p.o)[bht * p.dh + col] = __float2bfloat16_rn(v);
                        }
                    }
                if (qc == 0) {
                    if (!w.whole) p.ws_lse[place] = lse2;
                    else if (p.lse) p.lse[bht] = lse2 * kLn2t;
                }
            }
        }
        first_piece = false;
    }
    if (!ok) {
        if (lane == 0) atomicOr(p.err, kErrTimeout);
        *((volatile int*)&bars->abort) = 1;
    }
}

// One warp per row (b, h, t * G + g): merges the pieces of a cut item by
// log-sum-exp in piece order, M = max lse_p, O = sum 2^(lse_p - M) o_p / sum
// 2^(lse_p - M); rows past the sequence's drafted tokens get O = 0, LSE = -inf.
constexpr int kMergeWarps = 4;

__global__ void __launch_bounds__(kMergeWarps * 32)
attn_tree_merge_kernel(const __grid_constant__ TreeParams p) {
    const int lane = threadIdx.x & 31;
    const long long at = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    const int R = p.T * p.G;
    if (at >= (long long)p.B * p.Hkv * R) return;
    const long long bh = at / R;
    const int r = (int)(at - bh * R);
    const int b = (int)(bh / p.Hkv), h = (int)(bh - (long long)b * p.Hkv);
    const int t = r / p.G;
    const size_t bht = ((size_t)b * p.Hq + (size_t)h * p.G + (r - t * p.G)) * p.T + t;
    const TreeSeq s = tree_seq(p, b);
    int c0 = 0, c1 = -1, n = 1;  // CTAs that hold pieces of the item
    long long total = 1, start = 0;
    if (t < s.drafted) {
        total = tree_total(p, false);
        n = tree_ctas(p, total);
        const int rt = r / p.tile_rows;
        start = tree_base(p, b) + ((long long)h * s.row_tiles + rt) * s.key_tiles;
        const long long last = start + s.key_tiles - 1;
        c0 = (int)(start * n / total);
        while (c0 + 1 < n && tree_first(total, n, c0 + 1) <= start) ++c0;
        c1 = (int)(last * n / total);
        while (c1 + 1 < n && tree_first(total, n, c1 + 1) <= last) ++c1;
        if (c0 == c1) return;  // a whole item: the attention kernel wrote it
    }
    const int row = r % p.tile_rows;
    auto place = [&](int c) {
        return ((size_t)c * 2 + (start > tree_first(total, n, c) ? 1 : 0)) * p.tile_rows + row;
    };
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, __ldcg(p.ws_lse + place(c)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
    const float Ms = M == -INFINITY ? 0.f : M;
    for (int col = 4 * lane; col < p.dw; col += 128) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int c = c0; c <= c1; ++c) {
            const size_t pl = place(c);
            const float wt = ex2(__ldcg(p.ws_lse + pl) - Ms);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.ws_o + pl * p.dw + col));
            sum += wt;
            acc.x = fmaf(wt, v.x, acc.x);
            acc.y = fmaf(wt, v.y, acc.y);
            acc.z = fmaf(wt, v.z, acc.z);
            acc.w = fmaf(wt, v.w, acc.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
        if (col < p.dh) {
            if (p.out_f32)
                *reinterpret_cast<float4*>(static_cast<float*>(p.o) + bht * p.dh + col) =
                    make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            else
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + bht * p.dh + col) =
                    make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        }
        if (col == 0 && p.lse) p.lse[bht] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2t;
    }
}

template <int D, bool F8>
attn_status_t launch_tree_t(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                            cudaStream_t stream, const DeviceInfo& dev) {
    using C = TreeCfg<D, F8>;
    static int attr_set[64] = {0};
    if (dev.device >= 64 || !attr_set[dev.device]) {
        if (cudaFuncSetAttribute(attn_tree_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem) != cudaSuccess)
            return ATTN_ERR_CUDA;
        if (dev.device < 64) attr_set[dev.device] = 1;
    }
    attn_tree_kernel<D, F8><<<p.ctas, kTreeThreads, C::kSmem, stream>>>(tk, tv, p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Head dim that a cache runs at: 64, 128 or 256 columns (E4M3: 128 or 256).
int tree_width(int d, bool f8) { return d <= 64 && !f8 ? 64 : (d <= 128 ? 128 : 256); }

// CTAs of a launch: two to an SM (one at 256 columns of bf16, whose ring fills
// the shared memory).
int tree_grid(int d, bool f8, int num_sms) { return num_sms * (tree_width(d, f8) == 256 ? 1 : 2); }

size_t align16(size_t x) { return (x + 15) & ~size_t(15); }

}  // namespace

attn_status_t launch_tree_merge(const TreeParams& p, cudaStream_t stream) {
    const long long rows = (long long)p.B * p.Hkv * p.T * p.G;
    const long long blocks = (rows + kMergeWarps - 1) / kMergeWarps;
    attn_tree_merge_kernel<<<(unsigned)blocks, kMergeWarps * 32, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Whether a call runs on the tensor-core kernel of attn_tree_tc_sm103.cu.
static bool tree_on_tc(int d, int rows) { return d <= 128 && rows > kRows; }

static void tree_shape(TreeParams& p, int rows, bool f8, int num_sms) {
    if (tree_on_tc(p.dh, rows)) {
        tree_tc_shape(p, f8, num_sms);
        return;
    }
    p.tile_rows = kRows;
    p.tile_keys = kTileKeys;
    p.dw = tree_width(p.dh, f8);
    p.ctas = tree_grid(p.dh, f8, num_sms);
    p.min_units = 2;
}

size_t tree_workspace_bytes(int Hq, int Hkv, int T, int d, attn_cache_dtype_t cache_dtype, int num_sms) {
    TreeParams p;
    p.dh = d;
    tree_shape(p, T * (Hq / Hkv), cache_dtype == ATTN_CACHE_E4M3, num_sms);
    const size_t rows = (size_t)2 * p.ctas * p.tile_rows;
    return align16(rows * p.dw * 4) + align16(rows * 4);
}

attn_status_t launch_decode_tree(const void* q, const void* k_pages, const void* v_pages,
                                 const float* k_descale, const float* v_descale,
                                 const int* block_table, const int* seqlens, const int* q_lens,
                                 const uint64_t* tree_mask, void* o, float* lse, int B, int Hq,
                                 int Hkv, int T, long long num_blocks, int page_size,
                                 int max_blocks, int d, float scale,
                                 attn_cache_dtype_t cache_dtype, void* workspace,
                                 attn_out_dtype_t o_dtype, cudaStream_t stream,
                                 const DeviceInfo& dev) {
    const bool f8 = cache_dtype == ATTN_CACHE_E4M3;
    TreeParams p;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.T = T;
    p.W = (T + 63) / 64;
    p.max_blocks = max_blocks;
    p.page_size = page_size;
    p.num_blocks = num_blocks;
    p.dh = d;
    const int rows_kv = T * p.G;
    tree_shape(p, rows_kv, f8, dev.num_sms);
    p.box_keys = p.tile_keys;
    while (page_size % p.box_keys) p.box_keys /= 2;
    p.c = scale * kLog2et;
    p.block_table = block_table;
    p.seqlens = seqlens;
    p.q_lens = q_lens;
    p.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
    p.k_pages = static_cast<const uint8_t*>(k_pages);
    p.v_pages = static_cast<const uint8_t*>(v_pages);
    p.k_descale = k_descale;
    p.v_descale = v_descale;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.o = o;
    p.lse = lse;
    p.ws_o = static_cast<float*>(workspace);
    const size_t rows = (size_t)2 * p.ctas * p.tile_rows;
    p.ws_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align16(rows * p.dw * 4));
    p.out_f32 = o_dtype == ATTN_OUT_F32;
    p.err = dev.err_word;
    CUtensorMap tk, tv;
    attn_status_t st;
    if ((st = encode_tmap_pages(&tk, k_pages, f8, d, Hkv, page_size, num_blocks, p.box_keys)) != ATTN_OK) return st;
    if ((st = encode_tmap_pages(&tv, v_pages, f8, d, Hkv, page_size, num_blocks, p.box_keys)) != ATTN_OK) return st;
    if (tree_on_tc(d, rows_kv)) st = launch_tree_tc(tk, tv, p, f8, stream, dev);
    else if (f8) st = p.dw == 128 ? launch_tree_t<128, true>(tk, tv, p, stream, dev) : launch_tree_t<256, true>(tk, tv, p, stream, dev);
    else if (p.dw == 64) st = launch_tree_t<64, false>(tk, tv, p, stream, dev);
    else if (p.dw == 128) st = launch_tree_t<128, false>(tk, tv, p, stream, dev);
    else st = launch_tree_t<256, false>(tk, tv, p, stream, dev);
    if (st != ATTN_OK) return st;
    return launch_tree_merge(p, stream);
}

}  // namespace gb300
