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
// This file: the kernel for up to 16 query rows at a time on mma.sync
// (m16n8k16; tree_on_tc says which calls go to attn_tree_tc_sm103.cu), and
// the merge of cut items (tree_plan.h has the work list).  A producer warp
// streams 64-key tiles of K and V (and their descales) by TMA into a ring; two
// pairs of consumer warps take the tiles in turn, 32 keys a warp, each with its
// own online softmax (base 2), and the four are merged through shared memory at
// the end of a piece.  Bound: HBM (each cached byte is read once per row tile).
// One token, 16 sequences of 1024..32768 keys, calls on changing inputs, with the merge:
// bf16, d = 128, 8 heads 178 us, 6230 GB/s; E4M3, d = 128, 8 heads 107..116 us (cards
// differ), 4950..5350 GB/s, where the codes' conversion (cvt, 64 lanes a clock and SM) and
// the MMAs take about as long as the copies; E4M3, d = 256, 4 heads 108 us, 5200 GB/s;
// d = 64 in E4M3 takes a 128-column tile half of zeros: 98 us, 3000 GB/s.  (32 keys a
// warp: with 16 E4M3 took 128 us where this took 110, every shuffle and wait being paid
// twice as often.)
//
// The products are transposed, S^T = K Q^T and O^T = V^T P^T: keys and columns
// are the 16 rows of an MMA and the query rows its 8 columns, so up to 8 query
// rows (a single token's heads) cost half the MMAs and registers that a 16-row
// query operand would, which leaves room for three CTAs on an SM.  P^T becomes
// the second product's operand by an 8x8 transposition across the warp.
//
// E4M3 fragments: a lane takes 16 consecutive code bytes of a key with one
// shared load and spreads them over four k-steps (Q is laid out to match), so
// K needs no transposition.  V^T needs four keys' codes of one column in a
// register: four 16-byte rows are transposed with byte permutes.  P multiplies
// vd_j / F in fp16, F the power of two above the largest vd so far of the keys that
// the row sees (O is rescaled when F grows), times 2^15: weights times descales
// down to 2^-29 of the largest descale keep fp16's 11 bits, smaller ones are off by at
// most 2^-40 of F.  Each row has its own F, so that a V row which it does not see costs
// it no bits (one F for a warp's rows took 1% less; with F and the maximum raised in one
// branch 16 rows took 154 us instead of 149).  bf16 caches use bf16 P, as the library's decode does.
//
// Masked places: scores are selected, never added to.  V rows past the
// sequence are zeroed in shared memory; a drafted token's V row that holds a
// NaN or an infinity is taken out of the product (0 * NaN would reach the rows
// that do not see it) and added to the rows that do see it by itself.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "tree_plan.h"

namespace gb300 {
namespace {

constexpr int kConsumers = 4;
constexpr int kTreeThreads = (kConsumers + 1) * 32;
constexpr int kTileKeys = 64;
constexpr int kMaxRows = 16;
// An item's start and end, in 64-key tiles (16 drafts 188 us either way, 1 token over
// 16 short and long sequences 110 against 109 with 0: it matters where items are many).
constexpr int kExtraUnits = 2;
constexpr float kLn2t = 0.69314718055994530942f;
constexpr float kLog2et = 1.44269504088896340736f;
constexpr int kPFrame = 15;  // E4M3: P is held times 2^15 / F

// D columns, NT tiles of 8 query rows.
template <int D, bool F8, int NT>
struct TreeCfg {
    static constexpr int kRows = 8 * NT;
    static constexpr int kCtas = D == 256 ? (F8 && NT == 1 ? 2 : 1) : (NT == 1 ? 3 : 2);  // per SM
    // bytes of a 64-key K (or V) tile: 128-byte-wide swizzled boxes
    static constexpr int kBoxes = F8 ? D / 128 : D / 64;
    static constexpr int kHalf = kBoxes * kTileKeys * 128;
    static constexpr int kDescale = F8 ? 2 * kTileKeys * 4 : 0;  // kd, vd of a tile
    static constexpr int kStage = 2 * kHalf + kDescale;  // (the descales lie behind the tiles of all stages)
    static constexpr int kScratchBytes = 2 * kRows * D * 4;      // O of two warps
    // 228 KiB to an SM, 1 KiB of it the system's for each CTA
    static constexpr int kBudget = (228 / kCtas - 1) * 1024;
    static constexpr int kFit = (kBudget - kScratchBytes - 1024) / kStage;
    // an even number: every slot belongs to one pair of warps, which then sees each
    // of its barrier's phases
    static constexpr int kStages = kFit < 6 ? kFit / 2 * 2 : 6;
    static_assert(kStages >= 2, "ring");
    static constexpr int kDs = kStages * 2 * kHalf;  // the descales
    static constexpr int kScratch = kDs + kStages * kDescale;
    static constexpr int kBar = kScratch + kScratchBytes;
    static constexpr int kSmem = kBar + 1024;
};

struct TreeBars {
    uint64_t full[6], empty[6];
    TreeRange range;
    int abort;
    float m[kConsumers][kMaxRows], l[kConsumers][kMaxRows], x[kConsumers][kMaxRows];
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
// 8x8 transposition of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// Power of two 2^e (e in [-126, 127]; 128: infinite).
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

// The producer warp: lane 0 runs the ring, and each of the first lanes copies
// the tile's box of its own number (with its page looked up one tile ahead).
template <int D, bool F8, int NT>
__device__ __forceinline__ void produce(const CUtensorMap* tk, const CUtensorMap* tv, uint8_t* smem,
                                        TreeBars* bars, const TreeParams& p) {
    using C = TreeCfg<D, F8, NT>;
    const int lane = threadIdx.x & 31;
    const volatile int* abort_flag = &bars->abort;
    TreeWalk walk;
    walk.start(bars->range);
    TreePiece w;
    long long issued = 0;
    bool ok = true;
    const int boxes = kTileKeys / p.box_keys;
    while (ok && walk.next(p, w)) {
        int off = 0, page = lane < boxes ? tree_page(p, w.b, w.k0 * kTileKeys + lane * p.box_keys, w.keys, off) : -1;
        for (int kt = w.k0; kt < w.k1; ++kt, ++issued) {
            const int slot = (int)(issued % C::kStages);
            const long long round = issued / C::kStages;
            const int my_page = page, my_off = off;
            if (kt + 1 < w.k1 && lane < boxes)
                page = tree_page(p, w.b, (kt + 1) * kTileKeys + lane * p.box_keys, w.keys, off);
            if (round > 0) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&bars->empty[slot]), (uint32_t)((round - 1) & 1),
                                                       abort_flag));
                if (!ok) break;
            }
            const uint32_t bar = smem_u32(&bars->full[slot]);
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * C::kHalf + C::kDescale);
            __syncwarp();
            if (lane < boxes) {
                const uint32_t dk = smem_u32(smem + slot * 2 * C::kHalf);
                const uint32_t dv = dk + C::kHalf;
#pragma unroll
                for (int c = 0; c < C::kBoxes; ++c) {
                    const uint32_t to = c * (kTileKeys * 128) + lane * p.box_keys * 128;
                    tma_load_4d(dk + to, tk, bar, (F8 ? 128 : 64) * c, w.h, my_off, my_page);
                    tma_load_4d(dv + to, tv, bar, (F8 ? 128 : 64) * c, w.h, my_off, my_page);
                }
                if constexpr (F8) {
                    const long long at = ((long long)my_page * p.Hkv + w.h) * p.page_size + my_off;
                    const uint32_t ds = smem_u32(smem + C::kDs + slot * C::kDescale) + lane * p.box_keys * 4;
                    bulk_load(ds, my_page < 0 ? kTreeNoDescale : p.k_descale + at, p.box_keys * 4, bar);
                    bulk_load(ds + kTileKeys * 4, my_page < 0 ? kTreeNoDescale : p.v_descale + at, p.box_keys * 4, bar);
                }
            }
            __syncwarp();
        }
    }
    if (!ok && lane == 0) {
        atomicOr(p.err, kErrTimeout);
        *((volatile int*)&bars->abort) = 1;
    }
    // every issued copy lands before the CTA may leave
    for (int slot = 0; slot < C::kStages && slot < issued; ++slot) {
        const long long n = (issued - slot + C::kStages - 1) / C::kStages;
        mbar_wait(smem_u32(&bars->full[slot]), (uint32_t)((n - 1) & 1), nullptr);
    }
}

template <int D, bool F8, int NT>
__global__ void __launch_bounds__(kTreeThreads, TreeCfg<D, F8, NT>::kCtas)
attn_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ TreeParams p) {
    using C = TreeCfg<D, F8, NT>;
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
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the merge waits by itself)
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&bars->full[i]), 1);
            mbar_init(smem_u32(&bars->empty[i]), 2);
        }
        bars->abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (warp == kConsumers) {
        produce<D, F8, NT>(&tk, &tv, smem, bars, p);
        return;
    }

    const volatile int* abort_flag = &bars->abort;
    const int qr = lane >> 2, qc = lane & 3;
    const int mi = lane >> 3, ri = lane & 7;
    const int pair = warp >> 1, wk0 = (warp & 1) * 32;
    // this lane's keys of the warp's 32 are k_lane + 8 i, i < 4 (E4M3: an order that
    // keeps a quarter-warp's 16-byte loads on different banks)
    const int k_lane = F8 ? (qr >> 1) + 4 * (qr & 1) : qr;
    const int v_chunk = (qr >> 1) + 4 * (qr & 1);  // E4M3: 16-byte chunk of a V row's 128 columns
    // column of an accumulator element: MMA row qr + 8 hi of tile mt
    auto col_of = [&](int mt, int hi) {
        return F8 ? (mt >> 3) * 128 + 16 * v_chunk + 2 * (mt & 7) + hi : mt * 16 + qr + 8 * hi;
    };
    float* so = reinterpret_cast<float*>(smem + C::kScratch);
    TreeWalk walk;
    walk.start(bars->range);
    TreePiece w;
    long long used = 0;
    bool ok = true, first_piece = true;
    while (ok && walk.next(p, w)) {
        const int rows = min(C::kRows, w.drafted * p.G - w.rt * C::kRows);  // >= 1
        const int prefix = w.keys - w.drafted;
        // ---- Q operand: lane (qr, qc) holds columns of row qr + 8 nt (rows past
        // the last repeat it; never written)
        uint32_t qb[NT][D / 16][2];
        float qs[NT][2];  // what a product is multiplied with, rows 8 nt + 2 qc + {0, 1}
        int tok[NT][2];   // drafted token of those rows
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = w.rt * C::kRows + min(qr + 8 * nt, rows - 1);
            const int t = row / p.G;
            const __nv_bfloat16* q =
                p.q + (((size_t)w.b * p.Hq + (size_t)w.h * p.G + (row - t * p.G)) * p.T + t) * p.dh;
            float scale = p.c;
            if constexpr (!F8) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int c0 = ks * 16 + 2 * qc + 8 * hf;
                        qb[nt][ks][hf] = c0 < p.dh ? *reinterpret_cast<const uint32_t*>(q + c0) : 0u;
                    }
            } else {
                // fp16, each row scaled by a power of two that puts its largest value
                // in [2^14, 2^15): exact down to 2^-31 of it (8 bits above 2^-24), and off by
                // at most half a step, 2^-39 of it, below that
                float mx = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const int c0 = (ks >> 2) * 64 + 16 * qc + 4 * (ks & 3);
                    const uint2 v = c0 < p.dh ? *reinterpret_cast<const uint2*>(q + c0) : make_uint2(0u, 0u);
                    qb[nt][ks][0] = v.x;
                    qb[nt][ks][1] = v.y;
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(bf16lo_to_f32(v.x)), fabsf(bf16hi_to_f32(v.x))),
                                         fmaxf(fabsf(bf16lo_to_f32(v.y)), fabsf(bf16hi_to_f32(v.y)))));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                int e = (int)(__float_as_uint(mx) >> 23) - 127;
                e = e < -100 ? -100 : (e > 126 ? 126 : e);
                const float up = pow2i(14 - e);
                scale *= pow2i(e - 14);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                        qb[nt][ks][hf] =
                            pack_f16x2(bf16lo_to_f32(qb[nt][ks][hf]) * up, bf16hi_to_f32(qb[nt][ks][hf]) * up);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                qs[nt][r] = __shfl_sync(0xFFFFFFFFu, scale, 4 * (2 * qc + r));
                tok[nt][r] = __shfl_sync(0xFFFFFFFFu, t, 4 * (2 * qc + r));
            }
        }
        float acc[D / 16][NT][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[i][nt][0] = acc[i][nt][1] = acc[i][nt][2] = acc[i][nt][3] = 0.f;
        float m[NT][2], l[NT][2], xs[NT][2];
        // E4M3: a row's F = 2^fexp, 2^-100 (2^15 / F is finite where no key counts) to 2^128 (above every
        // finite descale); it is used together with 2^15 alone, so that each factor is in range
        int fexp[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                m[nt][r] = -INFINITY;
                l[nt][r] = 0.f;   // this lane's part of the sum that normalises O
                xs[nt][r] = 0.f;  // ... of the unrounded P (the LSE's)
                fexp[nt][r] = -100;
            }

        for (int kt = w.k0; kt < w.k1; ++kt, ++used) {
            if ((int)(used & 1) != pair) continue;  // the other pair's tile
            const int slot = (int)(used % C::kStages);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&bars->full[slot]),
                                                   (uint32_t)((used / C::kStages) & 1), abort_flag));
            if (!ok) break;
            const int key0 = kt * kTileKeys + wk0;  // this warp's first key
            const int nvalid = min(32, w.keys - key0);
            const uint32_t sK = smem_u32(smem + slot * 2 * C::kHalf);
            const uint32_t sV = sK + C::kHalf;
            const uint32_t sD = smem_u32(smem + C::kDs + slot * C::kDescale);
            bool wrote = false;
            if (nvalid > 0) {
                const bool plain = key0 + 32 <= prefix;  // every row sees all 32 keys
                // ---- S^T: sf[i >> 1][.][2 (i & 1) + r] is key k_lane + 8 i, row 8 nt + 2 qc + r
                float sf[2][NT][4];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float s2[NT][4];  // (two chains of products)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sf[g][nt][e] = s2[nt][e] = 0.f;
                    if constexpr (!F8) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            uint32_t a[4];
                            ldsm4(sK + tile_off(wk0 + 16 * g + (mi & 1) * 8 + ri, ks * 2 + (mi >> 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<false>(ks & 1 ? s2[nt] : sf[g][nt], a, qb[nt][ks][0], qb[nt][ks][1]);
                        }
                    } else {
#pragma unroll
                        for (int blk = 0; blk < D / 64; ++blk) {
                            const uint4 x = lds128(sK + tile_off(wk0 + 16 * g + k_lane, blk * 4 + qc));
                            const uint4 y = lds128(sK + tile_off(wk0 + 16 * g + k_lane + 8, blk * 4 + qc));
                            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t a[4] = {e4m3_lo(xw[k]), e4m3_lo(yw[k]), e4m3_hi(xw[k]), e4m3_hi(yw[k])};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816<true>(k & 1 ? s2[nt] : sf[g][nt], a, qb[nt][4 * blk + k][0],
                                                   qb[nt][4 * blk + k][1]);
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sf[g][nt][e] += s2[nt][e];
                }
                // ---- scale, mask
                float wv[4];  // E4M3: V's descale of this lane's keys
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float kd = 1.f;
                    wv[i] = 1.f;
                    if constexpr (F8) {
                        kd = lds32f(sD + (wk0 + k_lane + 8 * i) * 4);
                        wv[i] = lds32f(sD + (kTileKeys + wk0 + k_lane + 8 * i) * 4);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            sf[i >> 1][nt][2 * (i & 1) + r] *= F8 ? qs[nt][r] * kd : qs[nt][r];
                }
                unsigned bad = 0u;  // of the 32 keys: drafted rows of V with a NaN or an infinity
                if (!plain) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int kk = k_lane + 8 * i;
                        if (kk >= nvalid) wv[i] = 0.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                if (kk >= nvalid ||
                                    (key0 + kk >= prefix && !tree_sees(p, w.b, tok[nt][r], key0 + kk - prefix)))
                                    sf[i >> 1][nt][2 * (i & 1) + r] = -INFINITY;
                    }
                    for (int i = lane; i < 32 * (F8 ? D / 16 : D / 8); i += 32) {
                        const int kk = i & 31;
                        if (kk < nvalid && key0 + kk >= prefix &&
                            not_finite<F8>(lds128(sV + tile_off(wk0 + kk, i >> 5))))
                            bad |= 1u << kk;
                    }
                    if constexpr (F8) {
                        if (lane < nvalid && key0 + lane >= prefix &&
                            !isfinite(lds32f(sD + (kTileKeys + wk0 + lane) * 4)))
                            bad |= 1u << lane;
                    }
                    bad = __reduce_or_sync(0xFFFFFFFFu, bad);
                    if constexpr (F8) {  // (a finite descale still counts for F)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (bad >> (k_lane + 8 * i) & 1u && !isfinite(wv[i])) wv[i] = 0.f;
                    }
                }
                // ---- running maximum
                float mx[NT][2];
                bool moved = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float x = fmaxf(fmaxf(sf[0][nt][r], sf[0][nt][2 + r]), fmaxf(sf[1][nt][r], sf[1][nt][2 + r]));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                        mx[nt][r] = x;
                        moved |= x > m[nt][r];
                    }
                if constexpr (F8) {
                    int least = min(fexp[0][0], fexp[0][1]);
                    if constexpr (NT == 2) least = min(least, min(fexp[1][0], fexp[1][1]));
                    const float top_here = fmaxf(fmaxf(fabsf(wv[0]), fabsf(wv[1])), fmaxf(fabsf(wv[2]), fabsf(wv[3])));
                    if (__any_sync(0xFFFFFFFFu, top_here > pow2i(least))) {  // (2^128: infinite, above every finite descale)
                        // ---- F: the power of two above the largest descale of V of the keys that a row sees
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float top = 0.f;
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (sf[i >> 1][nt][2 * (i & 1) + r] != -INFINITY) top = fmaxf(top, fabsf(wv[i]));
#pragma unroll
                                for (int off = 4; off < 32; off <<= 1)
                                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
                                const int old = fexp[nt][r];
                                // 2^need > top
                                const int need = max(min((int)(__float_as_uint(top) >> 23) - 126, 128), old);
                                const float grow = old - need < -126 ? 0.f : pow2i(old - need);  // F_old / F_new
                                fexp[nt][r] = need;
#pragma unroll
                                for (int i = 0; i < D / 16; ++i) {
                                    acc[i][nt][r] *= grow;
                                    acc[i][nt][2 + r] *= grow;
                                }
                            }
                    }
                }
                if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float mn = fmaxf(m[nt][r], mx[nt][r]);
                            const float al = ex2(m[nt][r] - (mn == -INFINITY ? 0.f : mn));  // (no key yet: 0)
                            m[nt][r] = mn;
                            xs[nt][r] *= al;
                            l[nt][r] *= al;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                acc[i][nt][r] *= al;
                                acc[i][nt][2 + r] *= al;
                            }
                        }
                }
                // ---- P^T
                if constexpr (F8) {  // (rows that are added apart)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (bad >> (k_lane + 8 * i) & 1u) wv[i] = 0.f;
                }
                uint32_t pb[2][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
                    const float f0 = F8 ? pow2i(kPFrame - fexp[nt][0]) : 1.f, f1 = F8 ? pow2i(kPFrame - fexp[nt][1]) : 1.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p0 = ex2(sf[i >> 1][nt][2 * (i & 1)] - m0);
                        const float p1 = ex2(sf[i >> 1][nt][2 * (i & 1) + 1] - m1);
                        xs[nt][0] += p0;
                        xs[nt][1] += p1;
                        uint32_t pk;
                        if constexpr (F8) {
                            // (O over the sum of unrounded P; an unseen key's 0 before F, which may be far below it)
                            pk = pack_f16x2(p0 * wv[i] * f0, p1 * wv[i] * f1);
                        } else {
                            pk = pack_bf16x2(p0, p1);
                            l[nt][0] += bf16lo_to_f32(pk);
                            l[nt][1] += bf16hi_to_f32(pk);
                        }
                        pb[i >> 1][nt][i & 1] = transpose8x8(pk);
                    }
                }
                // ---- rows past the sequence, and rows with a NaN or an infinity:
                // the latter are added to the rows that see them, both are zeroed
                if (bad) {
                    for (unsigned left = bad; left; left &= left - 1) {
                        const int kk = __ffs(left) - 1;
                        const int qr_of = F8 ? 2 * (kk & 3) + ((kk >> 2) & 1) : kk & 7;  // who holds its scores
                        float pk[NT][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float own = kk < 16 ? (kk < 8 ? sf[0][nt][r] : sf[0][nt][2 + r])
                                                          : (kk < 24 ? sf[1][nt][r] : sf[1][nt][2 + r]);
                                const float sv = __shfl_sync(0xFFFFFFFFu, own, 4 * qr_of + qc);
                                // (-1: not seen)
                                pk[nt][r] = sv == -INFINITY ? -1.f : ex2(sv - (m[nt][r] == -INFINITY ? 0.f : m[nt][r]));
                                if constexpr (F8)
                                    if (sv != -INFINITY) pk[nt][r] *= pow2i(kPFrame - fexp[nt][r]);
                            }
                        float ds = 1.f;
                        if constexpr (F8) ds = lds32f(sD + (kTileKeys + wk0 + kk) * 4);
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
#pragma unroll
                            for (int hi = 0; hi < 2; ++hi) {
                                const int col = col_of(i, hi);
                                float v;
                                if constexpr (F8) {
                                    const uint32_t at = sV + tile_off(wk0 + kk, col >> 4) + (col & 15);
                                    uint32_t byte;
                                    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(at));
                                    v = e4m3_f32(byte) * ds;
                                } else {
                                    const uint32_t at = sV + tile_off(wk0 + kk, col >> 3) + 2 * (col & 7);
                                    uint32_t half;
                                    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(half) : "r"(at));
                                    v = __uint_as_float(half << 16);
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int r = 0; r < 2; ++r)
                                        if (pk[nt][r] != -1.f)
                                            acc[i][nt][2 * hi + r] = fmaf(pk[nt][r], v, acc[i][nt][2 * hi + r]);
                            }
                    }
                    __syncwarp();
                }
                const unsigned zero = bad | (nvalid < 32 ? 0xFFFFFFFFu << nvalid : 0u);
                if (zero) {
                    for (int i = lane; i < 32 * (F8 ? D / 16 : D / 8); i += 32)
                        if (zero >> (i & 31) & 1u) sts128(sV + tile_off(wk0 + (i & 31), i >> 5), 0u, 0u, 0u, 0u);
                    wrote = true;
                    __syncwarp();
                }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if constexpr (!F8) {
#pragma unroll
                        for (int mt = 0; mt < D / 16; ++mt) {
                            uint32_t a[4];
                            ldsm4_t(sV + tile_off(wk0 + 16 * g + (mi >> 1) * 8 + ri, mt * 2 + (mi & 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816<false>(acc[mt][nt], a, pb[g][nt][0], pb[g][nt][1]);
                        }
                    } else {
                        // P's k index 2 qc + {0, 1, 8, 9} is key qc + {0, 4, 8, 12}
#pragma unroll
                        for (int hf = 0; hf < D / 128; ++hf) {
                            const uint32_t at = sV + tile_off(wk0 + 16 * g + qc, hf * 8 + v_chunk);
                            const uint32_t at4 = sV + tile_off(wk0 + 16 * g + qc + 4, hf * 8 + v_chunk);
                            const uint4 r0 = lds128(at), r1 = lds128(at4), r2 = lds128(at + 1024), r3 = lds128(at4 + 1024);
                            const uint32_t a0[4] = {r0.x, r0.y, r0.z, r0.w}, a1[4] = {r1.x, r1.y, r1.z, r1.w};
                            const uint32_t a2[4] = {r2.x, r2.y, r2.z, r2.w}, a3[4] = {r3.x, r3.y, r3.z, r3.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t x01 = __byte_perm(a0[q], a1[q], 0x5140), y01 = __byte_perm(a0[q], a1[q], 0x7362);
                                const uint32_t x23 = __byte_perm(a2[q], a3[q], 0x5140), y23 = __byte_perm(a2[q], a3[q], 0x7362);
                                const uint32_t u[4] = {e4m3_lo(x01), e4m3_hi(x01), e4m3_lo(x23), e4m3_hi(x23)};
                                const uint32_t v[4] = {e4m3_lo(y01), e4m3_hi(y01), e4m3_lo(y23), e4m3_hi(y23)};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma16816<true>(acc[8 * hf + 2 * q][nt], u, pb[g][nt][0], pb[g][nt][1]);
                                    mma16816<true>(acc[8 * hf + 2 * q + 1][nt], v, pb[g][nt][0], pb[g][nt][1]);
                                }
                            }
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
        // ---- merge the four warps: sums over the keys' lanes, then the warps' maxima
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    l[nt][r] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][r], off);
                    xs[nt][r] += __shfl_xor_sync(0xFFFFFFFFu, xs[nt][r], off);
                }
                if (qr == 0) {
                    const int row = 8 * nt + 2 * qc + r;
                    bars->m[warp][row] = m[nt][r];
                    bars->l[warp][row] = F8 ? xs[nt][r] : l[nt][r];
                    bars->x[warp][row] = xs[nt][r];
                }
            }
        tree_consumers_sync();
        // this warp's O in the common frame and over the common sum
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 8 * nt + 2 * qc + r;
                const float M = fmaxf(fmaxf(bars->m[0][row], bars->m[1][row]), fmaxf(bars->m[2][row], bars->m[3][row]));
                const float Ms = M == -INFINITY ? 0.f : M;
                float sum = 0.f, sumx = 0.f;
#pragma unroll
                for (int x = 0; x < kConsumers; ++x) {
                    const float wt = ex2(bars->m[x][row] - Ms);
                    sum += wt * bars->l[x][row];
                    sumx += wt * bars->x[x][row];
                }
                const float mine =
                    sum == 0.f ? 0.f : ex2(m[nt][r] - Ms) * (F8 ? pow2i(fexp[nt][r] - kPFrame) : 1.f) / sum;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    acc[i][nt][r] *= mine;
                    acc[i][nt][2 + r] *= mine;
                }
                if (warp == 0 && qr == 0 && row < rows) {
                    const float lse2 = sumx == 0.f ? -INFINITY : M + log2f(sumx);
                    if (!w.whole) {
                        p.ws_lse[((size_t)blockIdx.x * 2 + (first_piece ? 0 : 1)) * C::kRows + row] = lse2;
                    } else if (p.lse) {
                        const int rr = w.rt * C::kRows + row;
                        p.lse[((size_t)w.b * p.Hq + (size_t)w.h * p.G + (rr - tok[nt][r] * p.G)) * p.T + tok[nt][r]] =
                            lse2 * kLn2t;
                    }
                }
            }
        // O of warps 2, 3 to warps 0, 1, then of warp 1 to warp 0 (lane by lane)
#pragma unroll 1
        for (int from = 2; from >= 1; from >>= 1) {
            float4* buf = reinterpret_cast<float4*>(so) + (warp & (from - 1)) * (C::kRows * D / 4) + lane;
            if (warp >= from && warp < 2 * from) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        buf[(i * NT + nt) * 32] = make_float4(acc[i][nt][0], acc[i][nt][1], acc[i][nt][2], acc[i][nt][3]);
            }
            tree_consumers_sync();
            if (warp < from) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float4 a = buf[(i * NT + nt) * 32];
                        acc[i][nt][0] += a.x;
                        acc[i][nt][1] += a.y;
                        acc[i][nt][2] += a.z;
                        acc[i][nt][3] += a.w;
                    }
            }
            if (from == 2) tree_consumers_sync();
        }
        if (!w.whole) {
            if (warp == 0) {
                float* out = p.ws_o + ((size_t)blockIdx.x * 2 + (first_piece ? 0 : 1)) * C::kRows * D;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int hi = 0; hi < 2; ++hi)
                            *reinterpret_cast<float2*>(out + col_of(i, hi) * C::kRows + 8 * nt + 2 * qc) =
                                make_float2(acc[i][nt][2 * hi], acc[i][nt][2 * hi + 1]);
            }
        } else {
            // rows [kRows][D] to shared memory (past warp 1's part), then out by all warps
            float* rows_s = so + C::kRows * D;
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            rows_s[(8 * nt + 2 * qc + (e & 1)) * D + col_of(i, e >> 1)] = acc[i][nt][e];
            }
            tree_consumers_sync();
            const int per = p.dh / 8;
            for (int i = threadIdx.x; i < rows * per; i += kConsumers * 32) {
                const int row = i / per, col = 8 * (i - row * per);
                const int rr = w.rt * C::kRows + row;
                const int t = rr / p.G;
                const size_t at =
                    (((size_t)w.b * p.Hq + (size_t)w.h * p.G + (rr - t * p.G)) * p.T + t) * p.dh + col;
                const float4 a = *reinterpret_cast<const float4*>(rows_s + row * D + col);
                const float4 b = *reinterpret_cast<const float4*>(rows_s + row * D + col + 4);
                if (p.out_f32) {
                    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.o) + at);
                    o[0] = a;
                    o[1] = b;
                } else {
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + at) =
                        make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                                   pack_bf16x2(b.z, b.w));
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

// A block takes the `group_rows` rows of a (sequence, KV head) that lie next to
// each other in a partial result, and merges the pieces of their item, if it was
// cut, by log-sum-exp in piece order: M = max lse_p, O = sum 2^(lse_p - M) o_p /
// sum 2^(lse_p - M).  Rows past the sequence's drafted tokens get O = 0, LSE =
// -inf.  A thread keeps to one row and CPT of its columns (blocks along y have
// other columns).  It is short and all latency (list, lse, partials, one after
// the other), so many loads of a thread are in flight, and it starts while the
// attention kernel ends (programmatic launch) and waits for it before it reads.
constexpr int kMergeThreads = 256;

template <int CPT>
__global__ void __launch_bounds__(kMergeThreads, 4)
attn_tree_merge_kernel(const __grid_constant__ TreeParams p) {
    // pieces whose loads are in flight together (16 columns: registers for one)
    constexpr int kPieces = CPT == 16 ? 1 : 32 / CPT;
    extern __shared__ float s_w[];     // [pieces][group_rows]: lse
    __shared__ __align__(16) float s_o[kMergeThreads * CPT + 32 * 4];  // rows 4 floats apart (banks)
    const int gr = p.group_rows;
    const int R = p.T * p.G;
    const int groups = (R + gr - 1) / gr;
    const int bh = blockIdx.x / groups;
    const int r0 = (blockIdx.x - bh * groups) * gr;
    const int b = bh / p.Hkv, h = bh - b * p.Hkv;
    const TreeSeq s = tree_seq(p, b);
    const int live = s.drafted * p.G;  // rows of the sequence
    int c0 = 0, c1 = -1, n = 1;        // CTAs that hold pieces of the item
    long long total = 1, start = 0;
    if (r0 < live) {
        total = tree_total_base(p, b, start);
        n = tree_ctas(p, total);
        start += ((long long)h * s.row_tiles + r0 / p.tile_rows) * (s.key_tiles + p.extra);
        const long long first = start + p.extra, last = first + s.key_tiles - 1;  // of its key tiles
        c0 = (int)tree_div(first * n, total);
        while (c0 + 1 < n && tree_first(total, n, c0 + 1) <= first) ++c0;
        c1 = (int)tree_div(last * n, total);
        while (c1 + 1 < n && tree_first(total, n, c1 + 1) <= last) ++c1;
    }
    const bool whole = c0 == c1;  // the attention kernel writes the live rows
    const int rows = min(gr, R - r0);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (every block: the grid may not end before the other)
    if (whole && r0 + rows <= live) return;
    const int row = threadIdx.x % gr, lane = threadIdx.x / gr, lanes = kMergeThreads / gr;
    const int in_tile = r0 % p.tile_rows;  // of the group's first row
    // only the first piece can be its CTA's last one (place 2c + 1): that CTA has
    // a key tile of the item before
    const int first_place = 2 * c0 + (start > tree_first(total, n, c0) ? 1 : 0);
    const int pieces = whole ? 0 : c1 - c0 + 1;
    auto place = [&](int i) { return (size_t)(i == 0 ? first_place : 2 * (c0 + i)); };
    const bool cut = pieces > 0 && r0 + row < live;
    // columns col0 + lane + k * lanes; the first pieces' loads do not wait for the lse
    const size_t stride = (size_t)p.tile_rows * p.dw;  // of a place
    const int col0 = blockIdx.y * lanes * CPT, cols = min(lanes * CPT, p.dw - col0);
    const float* src = p.ws_o + (size_t)in_tile * p.dw + (size_t)(col0 + lane) * gr + row;
    float v[kPieces][CPT], acc[CPT];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
#pragma unroll
            for (int k = 0; k < CPT; ++k)
                v[i][k] = cut && i0 + i < pieces && lane + k * lanes < cols
                              ? __ldcg(src + place(i0 + i) * stride + k * kMergeThreads)  // (lanes * gr)
                              : 0.f;
    };
    load(0);
    for (int i = lane; i < pieces; i += lanes)
        s_w[i * gr + row] = __ldcg(p.ws_lse + place(i) * p.tile_rows + in_tile + row);
    __syncthreads();
    float M = -INFINITY, sum = 0.f;
    if (cut)
        for (int i = 0; i < pieces; ++i) M = fmaxf(M, s_w[i * gr + row]);
    const float Ms = M == -INFINITY ? 0.f : M;
    // weights times 2^-shift, a sum of at most 1: pieces near fp32's largest value do not overflow
    const int shift = pieces > 1 ? 32 - __clz(pieces - 1) : 0;
    const float down = pow2i(-shift);
#pragma unroll
    for (int k = 0; k < CPT; ++k) acc[k] = 0.f;
    for (int i0 = 0; i0 < pieces; i0 += kPieces) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const float wt = cut && i0 + i < pieces ? ex2(s_w[(i0 + i) * gr + row] - Ms) * down : 0.f;
            sum += wt;
#pragma unroll
            for (int k = 0; k < CPT; ++k) acc[k] = fmaf(wt, v[i][k], acc[k]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    if (blockIdx.y == 0 && threadIdx.x < gr && row < rows && p.lse && (cut || r0 + row >= live)) {
        const int r = r0 + row, t = r / p.G;
        p.lse[((size_t)b * p.Hq + (size_t)h * p.G + (r - t * p.G)) * p.T + t] =
            sum == 0.f ? -INFINITY : (M + (shift + log2f(sum))) * kLn2t;
    }
#pragma unroll
    for (int k = 0; k < CPT; ++k)
        if (lane + k * lanes < cols) s_o[row * (cols + 4) + lane + k * lanes] = acc[k] * inv;
    __syncthreads();
    const int per = cols / 8;
    for (int i = threadIdx.x; i < rows * per; i += kMergeThreads) {
        const int ro = i / per, cc = 8 * (i - ro * per), col = col0 + cc;
        const int r = r0 + ro, t = r / p.G;
        if (col >= p.dh || (whole && r < live)) continue;
        const size_t at = (((size_t)b * p.Hq + (size_t)h * p.G + (r - t * p.G)) * p.T + t) * p.dh + col;
        const float4 x = *reinterpret_cast<const float4*>(&s_o[ro * (cols + 4) + cc]);
        const float4 y = *reinterpret_cast<const float4*>(&s_o[ro * (cols + 4) + cc + 4]);
        if (p.out_f32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.o) + at);
            o[0] = x;
            o[1] = y;
        } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + at) =
                make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y),
                           pack_bf16x2(y.z, y.w));
        }
    }
}

template <int D, bool F8, int NT>
attn_status_t launch_tree_t(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                            cudaStream_t stream, const DeviceInfo& dev) {
    using C = TreeCfg<D, F8, NT>;
    static int attr_set[64] = {0};
    if (dev.device >= 64 || !attr_set[dev.device]) {
        if (cudaFuncSetAttribute(attn_tree_kernel<D, F8, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem) != cudaSuccess)
            return ATTN_ERR_CUDA;
        if (dev.device < 64) attr_set[dev.device] = 1;
    }
    attn_tree_kernel<D, F8, NT><<<p.ctas, kTreeThreads, C::kSmem, stream>>>(tk, tv, p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Calls f<D, F8, NT>() for a cache of head dim d and `rows` query rows.
template <typename F>
auto tree_variant(int d, bool f8, int rows, F f) {
    using std::integral_constant;
    auto with_rows = [&](auto D, auto F8) {
        return rows <= 8 ? f(D, F8, integral_constant<int, 1>()) : f(D, F8, integral_constant<int, 2>());
    };
    integral_constant<bool, true> yes;
    integral_constant<bool, false> no;
    if (f8) return d <= 128 ? with_rows(integral_constant<int, 128>(), yes) : with_rows(integral_constant<int, 256>(), yes);
    if (d <= 64) return with_rows(integral_constant<int, 64>(), no);
    if (d <= 128) return f(integral_constant<int, 128>(), no, integral_constant<int, 1>());  // (more rows: tree_on_tc)
    return with_rows(integral_constant<int, 256>(), no);
}

size_t align16(size_t x) { return (x + 15) & ~size_t(15); }

}  // namespace

attn_status_t launch_tree_merge(const TreeParams& p, int num_sms, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)p.B * p.Hkv * ((p.T * p.G + p.group_rows - 1) / p.group_rows)));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = (size_t)p.ctas * p.group_rows * 4;  // (at most as many pieces as CTAs)
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // columns of a thread, of a row's share of 2 to 16: as few as leave one round
    // of blocks (four to an SM), since every block finds its item's pieces anew
    const int share = p.dw * p.group_rows / kMergeThreads;
    int cpt = 4;
    while (cpt < share && (long long)cfg.gridDim.x * (share / cpt) > 4ll * num_sms) cpt *= 2;
    cfg.gridDim.y = (unsigned)(share > cpt ? share / cpt : 1);
    const cudaError_t e = cpt == 4   ? cudaLaunchKernelEx(&cfg, attn_tree_merge_kernel<4>, p)
                          : cpt == 8 ? cudaLaunchKernelEx(&cfg, attn_tree_merge_kernel<8>, p)
                                     : cudaLaunchKernelEx(&cfg, attn_tree_merge_kernel<16>, p);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Whether a call runs on the tensor-core kernel of attn_tree_tc_sm103.cu, whose tile
// of 128 rows costs the same however few are live.  16 sequences of up to 32768 keys,
// 8 KV heads, this kernel / that one in us: bf16, d = 128, 8 rows 173 / 180, 12 rows
// 196 / 182, 16 rows 200 / 182, 20 rows 354 (two row tiles) / 186; bf16, d = 64, 16
// rows 114 / 136, 20 rows 195 / 136; E4M3, d = 128, 12 rows 148 / 204, 16 rows 149 / 205,
// 20 rows 269 / 205; E4M3, d = 64, 16 rows 148 / 205, 20 rows 266 / 205.  That kernel has
// no columns above 128: with d > 128 every 16 rows read the cache again here (bf16,
// d = 256, 4 KV heads: 8 rows 177 us, 32 rows 439, 256 rows 3300; E4M3 108, 335, 2530).
static bool tree_on_tc(int d, bool f8, int rows) {
    return d <= 128 && rows > (f8 || d <= 64 ? kMaxRows : kMaxRows / 2);
}

static void tree_shape(TreeParams& p, int rows, bool f8, int num_sms) {
    if (tree_on_tc(p.dh, f8, rows)) {
        tree_tc_shape(p, f8, num_sms);
        return;
    }
    p.tile_keys = kTileKeys;
    p.min_units = 2;
    p.extra = kExtraUnits;
    tree_variant(p.dh, f8, rows, [&](auto D, auto F8, auto NT) {
        using C = TreeCfg<decltype(D)::value, decltype(F8)::value, decltype(NT)::value>;
        p.tile_rows = p.group_rows = C::kRows;
        p.dw = D;
        p.ctas = num_sms * C::kCtas;
        return 0;
    });
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
    if (tree_on_tc(d, f8, rows_kv)) st = launch_tree_tc(tk, tv, p, f8, stream, dev);
    else
        st = tree_variant(d, f8, rows_kv, [&](auto D, auto F8, auto NT) {
            return launch_tree_t<decltype(D)::value, decltype(F8)::value, decltype(NT)::value>(tk, tv, p, stream, dev);
        });
    if (st != ATTN_OK) return st;
    return launch_tree_merge(p, dev.num_sms, stream);
}

}  // namespace gb300
