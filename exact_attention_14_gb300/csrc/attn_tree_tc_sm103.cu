// attn_tree_tc_sm103.cu -- tree attention (attn_tree_sm103.cu has the problem)
// for many query rows: up to 256 rows of one (sequence, KV head) at a time on
// the 5th-generation tensor cores.
//
// A persistent CTA per SM takes its range of the work list (tree_plan.h, items
// of 256 rows, 128-key tiles).  Two streams t = 0, 1 run side by side, each a
// 128-row tile with its own S, P and O in tensor memory and its own softmax
// warpgroup, so that one's exponentials overlap the other's products:
//   rows > 128 ("pair"):   the streams are the two row tiles and share every
//                          K and V tile;
//   rows <= 128 ("split"): both hold the same rows, stream t takes every second
//                          key tile, and the two are merged at the end.
// Roles (TcRoles): a TMA producer, an MMA issuer, two warpgroups of softmax (one a
// stream, a thread per row; they also lay Q out in shared memory, whose rows are not
// evenly spaced in a [B, Hq, T, d] tensor), and
//   bf16: a warp that prepares V in the tiles that hold drafted tokens or the end
//   of the sequence;
//   E4M3: warps that convert V's codes to fp16, times descale over F; the producer
//   lays the descales out.  K's codes and Q, as the sum of two E4M3 terms, go into
//   an 8-bit product as they are, so K is never converted.
// Calls of up to 128 rows (ONE) have an issuer for each stream, and in E4M3 a second
// producer and two more converters.
//
// A softmax warp takes 64 keys of S at a time (128 in registers at once spill: E4M3
// 368 -> 306 us), and the product of a half with V is issued while it works on the
// other: what stays between two tiles of a stream is half a product with V and S's.
//
// Masked places: see attn_tree_sm103.cu.  Here V rows past the sequence, and
// drafted tokens' V rows with a NaN or an infinity, are zeroed before the
// product; the latter are added again at the end of a piece to the rows that
// see them, with scores computed anew (a slow path that ordinary data never
// takes).  E4M3: so are keys of these tiles whose descales are far from the others'
// (tc_choose), which fp16 could not hold with them.
//
// Bound: HBM up to about 128 rows, then the tensor cores and the softmax.  256 rows
// by a 128-key tile: the four products take 2150 cycles of an SM's tensor cores, the
// tile (64 KiB in bf16) 2785 cycles of its share of HBM; measured, 16 sequences of
// 1024..32768 keys, 8 KV heads: bf16 about 3500 cycles (64 drafts, 4 heads a group,
// 250..262 us as a call, with the merge, 64% of the floor), E4M3 4600 (322 us on some
// cards, 347 on others), where S's multiplication with the descales (40 us) and fp16
// packing lengthen the softmax.  64 rows, bf16: 185..191 us, 87% of HBM's rate; E4M3
// 204 us, where both streams compute and convert for 128 rows.  d = 64 in E4M3 takes a
// 128-column tile half of zeros: 64 drafts 321..340 us.
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "tree_plan.h"

namespace gb300 {
namespace {

constexpr int kTcKeys = 128;
constexpr int kTcRows = 256;
constexpr float kTcTau = 8.0f;        // rescale threshold (log2 units)
// E4M3: P and its sums are held times 2^7, so that P, at most 2^(tau + 7), fits
// fp16 and weights down to 2^-21 of the largest keep its 11 bits
template <bool F8>
constexpr float kTcLift = F8 ? 7.0f : 0.0f;
// ... and V's descales over F times 2^7: with codes of at most 448 they fill fp16, and
// 2^7 / F and F / 2^7 are in fp32's range for every F from 2^-100 to 2^128
constexpr int kTcVLift = 7;
// E4M3, a special tile's keys are held with F when their descales are in (F / 2^12, F]: 2^7
// descale / F times a code, at least 2^-9, is then a normal fp16 number.  A drafted token
// raises the F of the keys before by up to 2^8.  Keys outside are added apart.
constexpr int kTcSpan = 12;
constexpr int kTcOver = 8;
constexpr float kTcLn2 = 0.69314718055994530942f;

// ONE: no item has more than 128 rows (every piece is split): the shared memory of a
// second Q tile holds more of K and V.
template <int D, bool F8, bool ONE>
struct TcCfg {
    static constexpr int kTile = 128 * D * 2;                  // 16-bit operand tile (Q's two terms)
    static constexpr int kStages = F8 ? 2 : (D == 128 ? (ONE ? 5 : 4) : 8);  // of K and V, E4M3: of V in fp16
    static constexpr int kCodes = 128 * 128;                   // E4M3 codes of a tile
    static constexpr int kKStages = F8 ? (ONE ? 4 : 3) : 0;                // K's codes, with K's and V's descales
    static constexpr int kVStages = F8 ? (ONE ? 3 : 2) : 0;                // V's codes
    static constexpr int kRing = (ONE ? 1 : 2) * kTile;         // after Q0, Q1
    static constexpr int kK = kRing + kStages * kTile;
    static constexpr int kV = kK + kKStages * kCodes;
    static constexpr int kDescale = kV + kVStages * kCodes;
    static constexpr int kBar = kDescale + kKStages * 1024;
    static constexpr int kSmem = kBar + 12 * 1024;
    static_assert(kSmem <= 232448, "shared memory budget");
};
template <bool F8, bool ONE>
struct TcRoles {
    static constexpr bool kMany = F8 && ONE;        // eight control warps
    static constexpr int kControl = kMany ? 8 : 4;  // the softmax warps come after them
    static constexpr int kThreads = 32 * (kControl + 8);
    static constexpr int kConverters = kMany ? 4 : 2;  // E4M3: the last control warps
    // registers of the control and the softmax warpgroups: their sum is the launch's
    static constexpr int kLaunch = kMany ? 128 : 168;
    static constexpr int kRegsControl = kMany ? 80 : 104, kRegsSoftmax = kMany ? 176 : 200;
    static_assert(32 * kControl * kRegsControl + 256 * kRegsSoftmax <= kThreads * kLaunch, "register split");
};

// Marks of the V rows that were taken out of the product: for each of the last pieces, for
// each of its special tiles (1024 drafted tokens reach over 10 at most), a bit
// per key.  A writer is at most 4 pieces ahead of the readers (a piece takes two
// of at most 8 ring slots), so 8 buffers need no hand-shake.
constexpr int kBadBufs = 8;
constexpr int kBadTiles = 10;
constexpr int kDs = 4;

struct TcBars {
    uint64_t q_full[2], s_full[2], o_half[2], o_full[2];
    uint64_t p_full[2][2];            // [stream][half of the tile's keys]
    uint64_t full[8], empty[8];       // tiles of K and V; E4M3: of V in fp16
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];  // E4M3 codes
    uint64_t ds_full[kDs], ds_empty[kDs];
    uint64_t fix_ask[2], fix_done[2];  // V of a special tile (of a stream; a pair's: [0]) is there / is prepared
    uint64_t stat, done, drain[2];
    TreeRange range;
    uint32_t tmem_base;
    int abort;
    uint32_t bad[kBadBufs][kBadTiles][4];
    float qs[2][128];                   // E4M3: what a row's products are multiplied with
    float m[2][128], l[2][128], lx[2][128];
    float fin[2];                       // E4M3: F / 2^7 of a stream at the end
    alignas(16) float kf[kDs][128];     // E4M3: K's descales of a tile
    alignas(16) float wv[kDs][128];     // E4M3: V's descales times 2^7 over F
    int fexp[kDs];
    uint32_t skip[kDs][4];              // E4M3: keys of a special tile that are added apart, by their descales
};
static_assert(sizeof(TcBars) <= 12 * 1024, "barrier block");

__device__ __forceinline__ void tc_abort(TcBars* bars, unsigned int* err) {
    atomicOr(err, kErrTimeout);
    *((volatile int*)&bars->abort) = 1;
}
__device__ __forceinline__ float tc_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ uint32_t tc_pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void tc_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ float2 tc_f16x2_f32(uint32_t h) {
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}
__device__ __forceinline__ void tc_sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ uint4 tc_lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag,
                                          int polls = 0) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(bar), parity & 1u, abort_flag, polls));
}

// A piece's streams.  Tile s of stream t is key tile k0 + (pair ? s : 2 s + t).
// Q lies in shared-memory tile t of a pair, in tile 0 of a split piece.
struct TcPiece {
    TreePiece w;
    int rows, n, prefix;
    bool pair;
    __device__ __forceinline__ void set(const TreeParams& p) {
        rows = min(kTcRows, w.drafted * p.G - w.rt * kTcRows);
        n = w.k1 - w.k0;
        prefix = w.keys - w.drafted;
        pair = rows > 128;
    }
    __device__ __forceinline__ int tile(int s, int t) const { return pair ? s : 2 * s + t; }
    __device__ __forceinline__ bool has(int s, int t) const { return tile(s, t) < n; }
    // a tile with drafted tokens or past the sequence's end
    __device__ __forceinline__ bool special(int j) const { return (w.k0 + j + 1) * kTcKeys > prefix; }
    // Where K and V of tile j lie in the order of a piece's 2 n bf16 loads: K of the
    // first tile of each stream, then per tile its V and the K of the stream's next.
    __device__ __forceinline__ int place_k(int j) const {
        const int ahead = pair ? 1 : 2;
        return j < ahead ? j : 2 * j - ahead + 1;
    }
    __device__ __forceinline__ int place_v(int j) const { return j + min(j + (pair ? 1 : 2), n); }
    __device__ __forceinline__ int first_special() const { return max(0, prefix / kTcKeys - w.k0); }
};

// ------------------------------------------------------------------ producer
// A ring of tiles that one warp fills.
struct TcRing {
    uint64_t *full, *empty;
    int slots, slot;
    uint32_t round;
    // The next slot once it is free, with `bytes` announced; -1: given up.
    __device__ __forceinline__ int take(int bytes, int lane, const volatile int* abort_flag) {
        if (round > 0 && !warp_wait(&empty[slot], round - 1u, abort_flag)) return -1;
        if (lane == 0) mbar_arrive_expect_tx(smem_u32(&full[slot]), bytes);
        __syncwarp();
        return slot;
    }
    __device__ __forceinline__ void next() {
        __syncwarp();
        if (++slot == slots) {
            slot = 0;
            ++round;
        }
    }
    __device__ __forceinline__ void land() {  // every copy lands
        for (int i = 0; i < slots; ++i) {
            const uint32_t n = round + (i < slot ? 1u : 0u);
            if (n > 0) mbar_wait(smem_u32(&full[i]), (n - 1u) & 1u, nullptr);
        }
        __syncwarp();
    }
};

// The F = 2^x of a special tile and the keys that are added apart, marked in `skip`; bit i
// of y: key 32 i + lane is one, or past the sequence.  vd: the tile's descales of V; keys
// below `prefix` come before the drafted ones, those from `keys` on are past the sequence.
// (Out of line: inside the producer's loop it took 64 drafts from 340 to 364 us.)
__device__ __noinline__ int2 tc_choose(const float* vd, int prefix, int keys, int fexp, uint32_t* skip) {
    constexpr int kNone = INT_MIN;
    const int lane = threadIdx.x & 31;
    int e[4], base = kNone, hi = kNone, lo = INT_MAX;  // 2^e above a descale
    bool lost[4];                                      // not finite
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = 32 * i + lane < keys ? fabsf(vd[32 * i + lane]) : 0.f;
        lost[i] = !(a < INFINITY);
        e[i] = a > 0.f && a < INFINITY ? max((int)(__float_as_uint(a) >> 23) - 126, -100) : kNone;
        if (e[i] == kNone) continue;
        if (32 * i + lane < prefix) base = max(base, e[i]);
        hi = max(hi, e[i]);
        lo = min(lo, e[i]);
    }
    base = max(__reduce_max_sync(0xFFFFFFFFu, base), fexp);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    if (base > -100) {  // there are keys before: F is theirs
        int top = base;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e[i] <= base + kTcOver) top = max(top, e[i]);
        fexp = __reduce_max_sync(0xFFFFFFFFu, top);
    } else if (hi != kNone) {  // the first keys of the piece: F for the largest or for the smallest, whichever are more
        int many = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            many += __popc(__ballot_sync(0xFFFFFFFFu, e[i] > hi - kTcSpan)) -
                    __popc(__ballot_sync(0xFFFFFFFFu, e[i] != kNone && e[i] < lo + kTcSpan));
        fexp = many >= 0 ? hi : lo + kTcSpan - 1;
    }
    int apart = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool out = lost[i] || (e[i] != kNone && (e[i] > fexp || e[i] <= fexp - kTcSpan));
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, out);
        if (lane == 0) skip[i] = votes;
        apart |= (int)(out || 32 * i + lane >= keys) << i;
    }
    return make_int2(fexp, apart);
}

// E4M3, a warp lays out the next tile's descales once its K is there: K's for the
// softmax, V's over F for the converters, F = 2^fexp above every one of the piece so
// far.  (K's codes go into the product as they are: rounded descales would enter the
// exponent.)  A drafted token that a row does not see may not cost it bits, so F and
// the keys that fit it are chosen anew in each special tile (tc_choose).
template <class C>
struct TcDescales {
    uint32_t tiles, kslot, kround;
    int fexp;
    __device__ __forceinline__ bool tile(uint8_t* smem, TcBars* bars, const TreePiece& w, int kt, int lane,
                                         const volatile int* abort_flag) {
        const uint32_t slot = tiles % kDs;
        if (!warp_wait(&bars->k_full[kslot], kround, abort_flag)) return false;
        if (tiles >= kDs && !warp_wait(&bars->ds_empty[slot], tiles / kDs - 1u, abort_flag)) return false;
        const float* raw = reinterpret_cast<const float*>(smem + C::kDescale + kslot * 1024);
        const int key0 = kt * kTcKeys + lane;
        float kd[4], vd[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kd[i] = raw[32 * i + lane];
            vd[i] = raw[128 + 32 * i + lane];
        }
        if ((kt + 1) * kTcKeys > w.keys - w.drafted) {
            const int2 c = tc_choose(raw + 128, w.keys - w.drafted - kt * kTcKeys, w.keys - kt * kTcKeys, fexp, bars->skip[slot]);
            fexp = c.x;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c.y >> i & 1) vd[i] = 0.f;  // (past the sequence too)
        } else {
            float top = fmaxf(fmaxf(fabsf(vd[0]), fabsf(vd[1])), fmaxf(fabsf(vd[2]), fabsf(vd[3])));
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
            fexp = max(fexp, min((int)(__float_as_uint(top) >> 23) - 126, 128));
        }
        const float fr = tc_pow2(kTcVLift - fexp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bars->kf[slot][32 * i + lane] = kd[i];
            bars->wv[slot][32 * i + lane] = vd[i] * fr;
        }
        if (lane == 0) bars->fexp[slot] = fexp;
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&bars->ds_full[slot]));
            mbar_arrive(smem_u32(&bars->k_empty[kslot]));
        }
        ++tiles;
        if (++kslot == C::kKStages) {
            kslot = 0;
            ++kround;
        }
        return true;
    }
};
// A lane's box of K's codes, with both descales.
template <class C>
__device__ __forceinline__ void tc_copy_k_codes(const CUtensorMap* map, uint8_t* smem, uint32_t bar, int slot, int lane,
                                                const TreeParams& p, int h, int page, int off) {
    tma_load_4d(smem_u32(smem + C::kK) + slot * C::kCodes + lane * p.box_keys * 128, map, bar, 0, h, off, page);
    const long long at = ((long long)page * p.Hkv + h) * p.page_size + off;
    const uint32_t ds = smem_u32(smem + C::kDescale) + slot * 1024 + lane * p.box_keys * 4;
    bulk_load(ds, page < 0 ? kTreeNoDescale : p.k_descale + at, p.box_keys * 4, bar);
    bulk_load(ds + 512, page < 0 ? kTreeNoDescale : p.v_descale + at, p.box_keys * 4, bar);
}

// A warp; each of its first lanes copies the tile's box of its own number.  The
// loads of a piece come in the order the products take them: K of the first
// tile of each stream, then per tile its V and the K of the stream's next tile.
template <int D, bool F8, bool ONE>
__device__ void tc_produce(const CUtensorMap* tk, const CUtensorMap* tv, uint8_t* smem, TcBars* bars,
                           const TreeParams& p) {
    using C = TcCfg<D, F8, ONE>;
    const int lane = threadIdx.x & 31;
    const uint32_t mine = lane * p.box_keys * 128;
    const volatile int* abort_flag = &bars->abort;
    const bool copies = lane < kTcKeys / p.box_keys;
    TcRing ring_k = {F8 ? bars->k_full : bars->full, F8 ? bars->k_empty : bars->empty, F8 ? C::kKStages : C::kStages, 0, 0u};
    TcRing ring_v = {bars->v_full, bars->v_empty, C::kVStages, 0, 0u};  // (bf16: K and V share the other)
    TcDescales<C> descales = {0u, 0u, 0u, 0};
    bool ok = true;
    TreeWalk walk;
    walk.start(bars->range);
    TcPiece x;
    while (ok && walk.next(p, x.w)) {
        x.set(p);
        auto load = [&](auto IsV, int page, int off) {
            constexpr bool is_v = decltype(IsV)::value;
            TcRing& r = F8 && is_v ? ring_v : ring_k;
            const int slot = r.take(!F8 ? C::kTile : (is_v ? C::kCodes : C::kCodes + 1024), lane, abort_flag);
            ok = slot >= 0;
            if (!ok) return;
            const uint32_t bar = smem_u32(&r.full[slot]);
            if (copies) {
                if constexpr (!F8) {
                    const uint32_t to = smem_u32(smem + C::kRing) + slot * C::kTile + mine;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_4d(to + c * 16384, is_v ? tv : tk, bar, 64 * c, x.w.h, off, page);
                } else if constexpr (is_v) {
                    tma_load_4d(smem_u32(smem + C::kV) + slot * C::kCodes + mine, tv, bar, 0, x.w.h, off, page);
                } else {
                    tc_copy_k_codes<C>(tk, smem, bar, slot, lane, p, x.w.h, page, off);
                }
            }
            r.next();
        };
        std::false_type K;
        std::true_type V;
        // pages of the tiles whose K has been loaded and whose V has not, and of
        // the next one (looked up before the wait that precedes its loads)
        int page[3], off[3];
        auto look = [&](int i, int j) {
            page[i] = -1;
            off[i] = 0;
            if (copies && j < x.n)
                page[i] = tree_page(p, x.w.b, (x.w.k0 + j) * kTcKeys + lane * p.box_keys, x.w.keys, off[i]);
        };
        look(0, 0);
        look(1, 1);
        look(2, 2);
        descales.fexp = -100;
        load(K, page[0], off[0]);
        if (!x.pair && x.n > 1 && ok) load(K, page[1], off[1]);
        for (int j = 0; j < x.n && ok; ++j) {
            load(V, page[0], off[0]);
            if (x.pair) {
                if (ok && j + 1 < x.n) load(K, page[1], off[1]);
            } else {
                if (ok && j + 2 < x.n) load(K, page[2], off[2]);
            }
            if constexpr (F8) ok = ok && descales.tile(smem, bars, x.w, x.w.k0 + j, lane, abort_flag);
            page[0] = page[1]; off[0] = off[1];
            page[1] = page[2]; off[1] = off[2];
            look(2, j + 3);
        }
    }
    if (!ok && lane == 0) tc_abort(bars, p.err);
    ring_k.land();
    if constexpr (F8) ring_v.land();
}

// E4M3 with eight control warps: a warp for K's codes and descales, another for V's
// codes that also lays the descales out (all of it in one warp takes longer than the
// copies themselves).
template <bool V, class C>
__device__ void tc_produce_codes(const CUtensorMap* map, uint8_t* smem, TcBars* bars, const TreeParams& p) {
    const int lane = threadIdx.x & 31;
    const volatile int* abort_flag = &bars->abort;
    const bool copies = lane < kTcKeys / p.box_keys;
    TcRing ring = {V ? bars->v_full : bars->k_full, V ? bars->v_empty : bars->k_empty, V ? C::kVStages : C::kKStages, 0, 0u};
    TcDescales<C> descales = {0u, 0u, 0u, 0};
    bool ok = true;
    TreeWalk walk;
    walk.start(bars->range);
    TreePiece w;
    while (ok && walk.next(p, w)) {
        descales.fexp = -100;
        // pages of this lane's box in the next two tiles
        int page[2], off[2];
        auto look = [&](int i, int kt) {
            page[i] = -1;
            off[i] = 0;
            if (copies && kt < w.k1) page[i] = tree_page(p, w.b, kt * kTcKeys + lane * p.box_keys, w.keys, off[i]);
        };
        look(0, w.k0);
        look(1, w.k0 + 1);
        for (int kt = w.k0; kt < w.k1; ++kt) {
            const int slot = ring.take(V ? C::kCodes : C::kCodes + 1024, lane, abort_flag);
            ok = slot >= 0;
            if (!ok) break;
            if (copies) {
                const uint32_t bar = smem_u32(&ring.full[slot]);
                if constexpr (V)
                    tma_load_4d(smem_u32(smem + C::kV) + slot * C::kCodes + lane * p.box_keys * 128, map, bar, 0, w.h,
                                off[0], page[0]);
                else
                    tc_copy_k_codes<C>(map, smem, bar, slot, lane, p, w.h, page[0], off[0]);
            }
            ring.next();
            page[0] = page[1];
            off[0] = off[1];
            look(1, kt + 2);
            if constexpr (V) {
                ok = descales.tile(smem, bars, w, kt, lane, abort_flag);
                if (!ok) break;
            }
        }
    }
    if (!ok && lane == 0) tc_abort(bars, p.err);
    ring.land();
}

// ----------------------------------------------------------------- MMA issuer
constexpr uint32_t kTcDescHi = sdesc_hi_sw128(1024);

// One warp for both streams, a stream after the other: while one's products run the
// other's softmax does, and two warps here let them fall into step (bf16, 64 drafts
// 246 -> 270 us, E4M3 320 -> 355).
template <int D, bool F8, bool ONE>
__device__ void tc_mma(uint8_t* smem, TcBars* bars, uint32_t tmem, const TreeParams& p) {
    using C = TcCfg<D, F8, ONE>;
    const volatile int* abort_flag = &bars->abort;
    constexpr uint32_t idS = F8 ? make_idesc_e4m3(128, kTcKeys) : make_idesc_bf16(128, kTcKeys, 0, 0);
    // (E4M3: P and V both fp16, format code 0)
    constexpr uint32_t idO = make_idesc_bf16(128, D, 0, 1) & ~(F8 ? (1u << 7) | (1u << 10) : 0u);
    const uint32_t q_lo[2] = {sdesc_lo(smem_u32(smem), 16), sdesc_lo(smem_u32(smem + C::kTile), 16)};
    const uint32_t ring = smem_u32(smem + C::kRing);
    uint32_t slot = 0, round = 0;  // of the next operand tile
    uint32_t cnt_q[2] = {0u, 0u}, cnt_p[2] = {0u, 0u}, cnt_fix[2] = {0u, 0u};
    bool ok = true;
    auto take = [&]() {
        const uint32_t mine = slot;
        ok = warp_wait(&bars->full[mine], round, abort_flag);
        if (++slot == C::kStages) {
            slot = 0;
            ++round;
        }
        tc_fence_after();
        return mine;
    };
    uint32_t kslot = 0, kround = 0;
    auto take_k = [&]() {
        if constexpr (!F8) {
            return take();
        } else {
            const uint32_t mine = kslot;
            ok = warp_wait(&bars->k_full[mine], kround, abort_flag);
            if (++kslot == C::kKStages) {
                kslot = 0;
                ++kround;
            }
            tc_fence_after();
            return mine;
        }
    };
    TreeWalk walk;
    walk.start(bars->range);
    TcPiece x;
    while (ok && walk.next(p, x.w)) {
        x.set(p);
        const bool pair = x.pair;
        const int n0 = pair ? x.n : (x.n + 1) / 2, n1 = pair ? x.n : x.n / 2;  // tiles of each stream
        uint32_t slot_k[2] = {0u, 0u}, slot_v[2] = {0u, 0u};  // (a pair's: [0])
        auto scores = [&](auto T) {  // of stream T's next tile
            constexpr int t = decltype(T)::value;
            const uint32_t slot = slot_k[pair ? 0 : t];
            const uint32_t a_lo = pair ? q_lo[t] : q_lo[0];
            const uint32_t to = tmem + t * 128;
            if constexpr (F8) {
                // both of Q's terms times K's codes
                const uint32_t k_lo = sdesc_lo(smem_u32(smem + C::kK) + slot * C::kCodes, 16);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss_f8_warp(to, sdesc_join(a_lo + (kk >> 2) * (16384 >> 4) + (kk & 3) * (32 >> 4), kTcDescHi),
                                   sdesc_join(k_lo + (kk & 3) * (32 >> 4), kTcDescHi), idS, kk > 0 ? 1u : 0u);
            } else {
                const uint32_t k_lo = sdesc_lo(ring + slot * C::kTile, 16);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t step = (kk >> 2) * (16384 >> 4) + (kk & 3) * (32 >> 4);
                    mma_ss_warp(to, sdesc_join(a_lo + step, kTcDescHi), sdesc_join(k_lo + step, kTcDescHi), idS,
                                kk > 0 ? 1u : 0u);
                }
            }
            mma_commit_warp(smem_u32(&bars->s_full[t]));
            if (!pair || t == 1) mma_commit_warp(smem_u32(F8 ? &bars->k_empty[slot] : &bars->empty[slot]));
        };
        std::integral_constant<int, 0> I0;
        std::integral_constant<int, 1> I1;
        auto begin = [&](auto T) {
            constexpr int t = decltype(T)::value;
            if ((t == 0 ? n0 : n1) == 0 || !ok) return;
            if (pair || t == 0) {
                ok = warp_wait(&bars->q_full[t], cnt_q[t]++, abort_flag);
                if (!ok) return;
                tc_fence_after();
            }
            if (!pair || t == 0) slot_k[t] = take_k();
            if (ok) scores(T);
        };
        // half H of the product with V of stream T's tile s; after the second the next scores
        auto step = [&](auto T, auto H, int s) {
            constexpr int t = decltype(T)::value, h = decltype(H)::value;
            const int n = t == 0 ? n0 : n1;
            if (s >= n || !ok) return;
            if (h == 0 && (!pair || t == 0)) {
                slot_v[t] = take();
                if (!F8 && ok && x.special(x.tile(s, t))) {
                    // the fixer works on it while this stream's softmax still runs
                    if (elect_one()) mbar_arrive(smem_u32(&bars->fix_ask[t]));
                    __syncwarp();
                    ok = warp_wait(&bars->fix_done[t], cnt_fix[t]++, abort_flag);
                }
                if (!ok) return;
            }
            ok = warp_wait(&bars->p_full[t][h], cnt_p[t], abort_flag, 32);
            if (!ok) return;
            tc_fence_after();
            const uint32_t slot = slot_v[pair ? 0 : t];
            const uint32_t v_lo = sdesc_lo(ring + slot * C::kTile, 16384);
#pragma unroll
            for (int kk = 0; kk < kTcKeys / 32; ++kk)
                mma_ts_warp(tmem + 256 + t * 128, tmem + t * 128 + h * 64 + kk * 8,
                            sdesc_join(v_lo + (4 * h + kk) * (2048 >> 4), kTcDescHi), idO,
                            (s > 0 || h > 0 || kk > 0) ? 1u : 0u);
            if (h == 0) {
                mma_commit_warp(smem_u32(&bars->o_half[t]));
                return;
            }
            ++cnt_p[t];
            if (!pair || t == 1) mma_commit_warp(smem_u32(&bars->empty[slot]));
            if (s + 1 < n) {
                if (!pair || t == 0) slot_k[t] = take_k();
                if (ok) scores(T);  // in order after the products that read P over it
            } else {
                mma_commit_warp(smem_u32(&bars->o_full[t]));
            }
        };
        begin(I0);
        begin(I1);
        for (int s = 0; s < n0 && ok; ++s) {
            step(I0, I0, s);
            step(I0, I1, s);
            step(I1, I0, s);
            step(I1, I1, s);
        }
        if (n1 == 0) mma_commit_warp(smem_u32(&bars->o_full[1]));
    }
    if (!ok && elect_one()) tc_abort(bars, p.err);
    mma_commit_warp(smem_u32(&bars->drain[0]));  // every product is done before TMEM goes
    mbar_wait(smem_u32(&bars->drain[0]), 0, nullptr);
    __syncwarp();
}

// Split pieces only: a warp per stream, so that neither waits for the other's softmax
// (E4M3, 16 drafts 242 -> 200 us, bf16 186 -> 183).
template <int D, bool F8, bool ONE>
__device__ void tc_mma_stream(int t, uint8_t* smem, TcBars* bars, uint32_t tmem, const TreeParams& p) {
    using C = TcCfg<D, F8, ONE>;
    const volatile int* abort_flag = &bars->abort;
    constexpr uint32_t idS = F8 ? make_idesc_e4m3(128, kTcKeys) : make_idesc_bf16(128, kTcKeys, 0, 0);
    // (E4M3: P and V both fp16, format code 0)
    constexpr uint32_t idO = make_idesc_bf16(128, D, 0, 1) & ~(F8 ? (1u << 7) | (1u << 10) : 0u);
    const uint32_t ring = smem_u32(smem + C::kRing);
    const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * 128;
    uint32_t loads = 0;  // tiles (E4M3), loads (bf16) of the pieces before
    uint32_t cnt_p = 0, cnt_fix = 0;
    const uint32_t q_lo = sdesc_lo(smem_u32(smem), 16);
    bool ok = true;
    // A ring's tiles are waited for one after another, the other stream's too, and
    // those are let go of at once: a slot is free when its reader is done with it and
    // the other has passed it, so that neither ever misses a phase of its barrier.
    struct Seen {
        uint64_t *full, *empty;
        uint32_t slot, round, at;
    };
    Seen seen_k = {F8 ? bars->k_full : bars->full, F8 ? bars->k_empty : bars->empty, 0u, 0u, 0u};
    Seen seen_v = {bars->full, bars->empty, 0u, 0u, 0u};  // (bf16: K and V share one ring)
    auto see = [&](Seen& s, auto Slots, uint32_t upto, bool mine) {  // `mine`: the last of them
        while (ok && s.at < upto) {
            ok = warp_wait(&s.full[s.slot], s.round, abort_flag);
            ++s.at;
            if (!(mine && s.at == upto) && elect_one()) mbar_arrive(smem_u32(&s.empty[s.slot]));
            __syncwarp();
            if (++s.slot == decltype(Slots)::value) {
                s.slot = 0;
                ++s.round;
            }
        }
    };
    std::integral_constant<uint32_t, F8 ? C::kKStages : C::kStages> SlotsK;
    std::integral_constant<uint32_t, C::kStages> SlotsV;
    auto see_k = [&](uint32_t upto, bool mine) { see(seen_k, SlotsK, upto, mine); };
    auto see_v = [&](uint32_t upto, bool mine) {
        if constexpr (F8) see(seen_v, SlotsV, upto, mine);
        else see(seen_k, SlotsK, upto, mine);
    };
    TreeWalk walk;
    walk.start(bars->range);
    TcPiece x;
    for (uint32_t piece = 0; ok && walk.next(p, x.w); ++piece) {
        x.set(p);
        // (also without a tile: this keeps step with the softmax warps)
        ok = warp_wait(&bars->q_full[0], piece, abort_flag);
        if (!ok) break;
        tc_fence_after();
        auto scores = [&](int j) {
            const uint32_t at = F8 ? loads + j : loads + x.place_k(j);
            const uint32_t slot = at % (F8 ? C::kKStages : C::kStages);
            see_k(at + 1u, true);
            if (!ok) return;
            tc_fence_after();
            if constexpr (F8) {
                // both of Q's terms times K's codes
                const uint32_t k_lo = sdesc_lo(smem_u32(smem + C::kK) + slot * C::kCodes, 16);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ss_f8_warp(tS, sdesc_join(q_lo + (kk >> 2) * (16384 >> 4) + (kk & 3) * (32 >> 4), kTcDescHi),
                                   sdesc_join(k_lo + (kk & 3) * (32 >> 4), kTcDescHi), idS, kk > 0 ? 1u : 0u);
            } else {
                const uint32_t k_lo = sdesc_lo(ring + slot * C::kTile, 16);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t step = (kk >> 2) * (16384 >> 4) + (kk & 3) * (32 >> 4);
                    mma_ss_warp(tS, sdesc_join(q_lo + step, kTcDescHi), sdesc_join(k_lo + step, kTcDescHi), idS,
                                kk > 0 ? 1u : 0u);
                }
            }
            mma_commit_warp(smem_u32(&bars->s_full[t]));
            mma_commit_warp(smem_u32(F8 ? &bars->k_empty[slot] : &bars->empty[slot]));
        };
        if (x.has(0, t)) scores(x.tile(0, t));
        for (int s = 0; x.has(s, t) && ok; ++s) {
            const int j = x.tile(s, t);
            const uint32_t at = F8 ? loads + j : loads + x.place_v(j);
            const uint32_t slot = at % C::kStages;
            see_v(at + 1u, true);
            if (!F8 && ok && x.special(j)) {
                // the fixer works on it while this stream's softmax still runs
                if (elect_one()) mbar_arrive(smem_u32(&bars->fix_ask[t]));
                __syncwarp();
                ok = warp_wait(&bars->fix_done[t], cnt_fix++, abort_flag);
            }
            const uint32_t v_lo = sdesc_lo(ring + slot * C::kTile, 16384);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ok = ok && warp_wait(&bars->p_full[t][h], cnt_p, abort_flag, 32);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kTcKeys / 32; ++kk)
                    mma_ts_warp(tO, tS + h * 64 + kk * 8, sdesc_join(v_lo + (4 * h + kk) * (2048 >> 4), kTcDescHi), idO,
                                (s > 0 || h > 0 || kk > 0) ? 1u : 0u);
                if (h == 0) mma_commit_warp(smem_u32(&bars->o_half[t]));
            }
            if (!ok) break;
            ++cnt_p;
            mma_commit_warp(smem_u32(&bars->empty[slot]));
            if (x.has(s + 1, t)) scores(x.tile(s + 1, t));  // in order after the products that read P over it
        }
        loads += F8 ? x.n : 2 * x.n;
        see_k(loads, false);
        if (F8) see_v(loads, false);
        mma_commit_warp(smem_u32(&bars->o_full[t]));  // (also without a tile)
    }
    if (!ok && elect_one()) tc_abort(bars, p.err);
    mma_commit_warp(smem_u32(&bars->drain[t]));  // every product is done before TMEM goes
    mbar_wait(smem_u32(&bars->drain[t]), 0, nullptr);
    __syncwarp();
}

// --------------------------------------------------- V of special tiles, bf16
// A warp, four keys a thread: rows past the sequence are zeroed, drafted
// tokens' rows with a NaN or an infinity are noted and zeroed.
template <int D, bool ONE>
__device__ void tc_fix(uint8_t* smem, TcBars* bars, const TreeParams& p) {
    using C = TcCfg<D, false, ONE>;
    const int lane = threadIdx.x & 31;
    const volatile int* abort_flag = &bars->abort;
    uint32_t fixed[2] = {0u, 0u}, loads = 0;
    bool ok = true;
    TreeWalk walk;
    walk.start(bars->range);
    TcPiece x;
    for (int piece = 0; ok && walk.next(p, x.w); ++piece) {
        x.set(p);
        for (int j = x.first_special(); j < x.n && ok; ++j) {
            if (!x.special(j)) continue;
            // (whoever asks has seen the tile's V arrive, and waits for this)
            const int b = x.pair ? 0 : j & 1;
            ok = warp_wait(&bars->fix_ask[b], fixed[b]++, abort_flag);
            if (!ok) break;
            const uint32_t tile = smem_u32(smem + C::kRing) + (loads + x.place_v(j)) % C::kStages * C::kTile;
            uint32_t* marks = bars->bad[piece % kBadBufs][j - x.first_special()];
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int row = i * 32 + lane;
                const int key = (x.w.k0 + j) * kTcKeys + row;
                const uint32_t at = tile + row * 128;
                bool bad = false;
                if (key >= x.prefix && key < x.w.keys) {
#pragma unroll 4
                    for (int c = 0; c < p.dh / 8; ++c) {
                        const uint4 v = tc_lds128(at + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4));
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            bad |= (u[e] & 0x7F80u) == 0x7F80u || (u[e] & 0x7F800000u) == 0x7F800000u;
                    }
                }
                const uint32_t votes = __ballot_sync(0xFFFFFFFFu, bad);
                if (lane == 0) marks[i] = votes;
                if (bad || key >= x.w.keys)
                    for (int c = 0; c < D / 8; ++c)
                        sts128(at + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4), 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->fix_done[b]));
        }
        loads += 2 * x.n;
    }
    if (!ok && lane == 0) tc_abort(bars, p.err);
}

// ------------------------------------------------------- V's codes to fp16, E4M3
// NC warps, 128 / NC keys each.  A lane takes 16 of a row's 128 codes, times the row's
// descale over F: two fp16 roundings, of the factor and of the product, less than
// P's and far less than O's.
template <int NC, class C>
__device__ void tc_convert(int wc, uint8_t* smem, TcBars* bars, const TreeParams& p) {
    constexpr int kRows = 128 / NC;
    const int lane = threadIdx.x & 31;
    const volatile int* abort_flag = &bars->abort;
    uint32_t raw_slot = 0, raw_round = 0, out_slot = 0, out_round = 0, tiles = 0;
    bool ok = true;
    TreeWalk walk;
    walk.start(bars->range);
    TcPiece x;
    const int c = lane & 7;
    // lane's row of four, plus 4 i: the lanes of the upper columns take the
    // neighbour's row, whose swizzle puts their stores on the other banks
    const int row_in = (lane >> 3) ^ (c >> 2);
    for (int piece = 0; ok && walk.next(p, x.w); ++piece) {
        x.set(p);
        for (int j = 0; j < x.n; ++j) {
            const uint32_t ds = tiles % kDs;
            ok = warp_wait(&bars->ds_full[ds], tiles / kDs, abort_flag) &&
                 warp_wait(&bars->v_full[raw_slot], raw_round, abort_flag);
            if (ok && out_round > 0) ok = warp_wait(&bars->empty[out_slot], out_round - 1u, abort_flag);
            if (!ok) break;
            const uint32_t raw = smem_u32(smem + C::kV + raw_slot * C::kCodes);
            const uint32_t out = smem_u32(smem + C::kRing + out_slot * C::kTile) + (c >> 2) * 16384;
            if (x.special(j)) {
                // rows that must not enter the product become zeros where they lie
                uint32_t marks = 0u;
#pragma unroll 1
                for (int i = 0; i < kRows / 4; ++i) {
                    const int row = kRows * wc + (lane >> 3) + 4 * i;
                    const int key = (x.w.k0 + j) * kTcKeys + row;
                    const uint32_t piece_at = raw + row * 128 + ((c ^ (row & 7)) << 4);
                    bool hit = false;
                    if (key >= x.prefix && key < x.w.keys) {
                        const uint4 v = tc_lds128(piece_at);
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 16; ++e) hit |= ((u[e >> 2] >> (8 * (e & 3))) & 0x7Fu) == 0x7Fu;
                    }
                    if (c == 0) hit |= (*((volatile uint32_t*)&bars->skip[ds][row >> 5]) >> (row & 31)) & 1u;
                    const unsigned votes = __ballot_sync(0xFFFFFFFFu, hit);
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        if ((votes >> (8 * g)) & 0xFFu) marks |= 1u << (4 * (i & 7) + g);
                    if (key >= x.w.keys || ((votes >> (lane & 24)) & 0xFFu)) sts128(piece_at, 0u, 0u, 0u, 0u);
                    if ((i & 7) == 7) {
                        if (lane == 0) bars->bad[piece % kBadBufs][j - x.first_special()][kRows / 32 * wc + (i >> 3)] = marks;
                        marks = 0u;
                    }
                }
                __syncwarp();  // (other lanes read the rows below)
            }
            // this lane's rows: row0 + 4 i; row & 7 = row_in + 4 (i & 1), so the
            // swizzle has two patterns
            const int row0 = kRows * wc + row_in;
            const uint32_t src[2] = {raw + row0 * 128 + ((c ^ row_in) << 4), raw + row0 * 128 + ((c ^ row_in ^ 4) << 4)};
            const int ch = 2 * (c & 3);
            const uint32_t dst[2] = {out + row0 * 128 + ((ch ^ row_in) << 4), out + row0 * 128 + ((ch ^ row_in ^ 4) << 4)};
            const uint32_t odd = 16 - ((row_in & 1) << 5);  // from an even chunk to its odd neighbour
            const float* fv = &bars->wv[ds][row0];
#pragma unroll 1
            for (int i0 = 0; i0 < kRows / 4; i0 += 4) {
                uint4 w[4];
                float d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = tc_lds128(src[i & 1] + 512 * (i0 + i));
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = fv[4 * (i0 + i)];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t h[8];
                    tc_e4m3x4(w[i].x, h[0], h[1]);
                    tc_e4m3x4(w[i].y, h[2], h[3]);
                    tc_e4m3x4(w[i].z, h[4], h[5]);
                    tc_e4m3x4(w[i].w, h[6], h[7]);
                    const uint32_t f = tc_pack_f16(d[i], d[i]);  // its descale over F
#pragma unroll
                    for (int e = 0; e < 8; ++e) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[e]) : "r"(f));
                    sts128(dst[i & 1] + 512 * (i0 + i), h[0], h[1], h[2], h[3]);
                    sts128(dst[i & 1] + 512 * (i0 + i) + odd, h[4], h[5], h[6], h[7]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&bars->full[out_slot]));
                mbar_arrive(smem_u32(&bars->v_empty[raw_slot]));
                mbar_arrive(smem_u32(&bars->ds_empty[ds]));
            }
            ++tiles;
            if (++raw_slot == C::kVStages) {
                raw_slot = 0;
                ++raw_round;
            }
            if (++out_slot == C::kStages) {
                out_slot = 0;
                ++out_round;
            }
        }
    }
    if (!ok && lane == 0) tc_abort(bars, p.err);
}

// -------------------------------------------------------------------- softmax
// A row's mask over 64 keys: bit i of word w is key u0 + 32 w + i,
// counted from the first drafted token (negative: before it).  `mask`: the row's
// words where T <= 64.
__device__ __forceinline__ void tc_allow(const TreeParams& p, int b, int t, int drafted, int u0,
                                         uint2 mask, uint32_t (&allow)[2]) {
    const int seen = p.mask ? drafted : min(t + 1, drafted);
    uint32_t bits[3];
    const int first = u0 >> 5;  // (floor) 32-bit word of the row's mask that u0 falls in
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int at = first + i;
        bits[i] = 0xFFFFFFFFu;  // before the drafted tokens, or no mask
        if (p.mask && at >= 0) {
            if (p.W == 1) {
                bits[i] = at == 0 ? mask.x : mask.y;
            } else {
                const int last = 2 * p.W - 1;
                bits[i] = __ldg(reinterpret_cast<const uint32_t*>(p.mask + ((size_t)b * p.T + t) * p.W) + min(at, last));
            }
        }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int n = seen - (u0 + 32 * w);  // keys below `seen`
        const uint32_t range = n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
        allow[w] = __funnelshift_r(bits[w], bits[w + 1], u0 & 31) & range;
    }
}

__device__ __forceinline__ void tc_ld16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}

struct TcRow {
    float m, l, lx;  // running maximum (log2 units), sums of rounded and of unrounded P (times 2^lift)
    int fexp;        // E4M3: F of what O holds
};

// Half a tile of a row, 64 keys: the maximum over all of it, O rescaled if that
// moved by more than tau (or, E4M3, if F grew), then P over S's first 32 columns.
// The scores stay in registers between the two; E4M3 multiplies them with K's
// descales, which every lane reads from the same shared address (a wavefront for
// four bytes: read once, not once for each use).  `stable()`: waits until no product
// is adding to O.
template <bool F8, class Stable>
__device__ __forceinline__ void tc_softmax_half(uint32_t tS, uint32_t tO, const float* kf, int fexp, bool special,
                                                const uint32_t (&allow)[2], bool first, float c, int ncols,
                                                TcRow& r, Stable stable) {
    uint32_t sr[64];
    tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
    tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
    tmem_wait_ld();
    if constexpr (F8) {
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
            const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(kf + i);
            float u, v;
            f2_split(f2_mul(f2(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])), k.x), u, v);
            sr[i] = __float_as_uint(u);
            sr[i + 1] = __float_as_uint(v);
            f2_split(f2_mul(f2(__uint_as_float(sr[i + 2]), __uint_as_float(sr[i + 3])), k.y), u, v);
            sr[i + 2] = __float_as_uint(u);
            sr[i + 3] = __float_as_uint(v);
        }
    }
    if (special) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (!(allow[i >> 5] >> (i & 31) & 1u)) sr[i] = 0xFF800000u;
    }
    float mx;
    {
        float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 64; i += 8) {
            m0 = fmax3(m0, __uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
            m1 = fmax3(m1, __uint_as_float(sr[i + 2]), __uint_as_float(sr[i + 3]));
            m2 = fmax3(m2, __uint_as_float(sr[i + 4]), __uint_as_float(sr[i + 5]));
            m3 = fmax3(m3, __uint_as_float(sr[i + 6]), __uint_as_float(sr[i + 7]));
        }
        mx = fmax3(fmaxf(m0, m1), m2, m3);
    }
    const float mt = mx * c;  // (c > 0)
    const bool need = mt > r.m + kTcTau;
    bool grow = false;
    if constexpr (F8) grow = !first && fexp != r.fexp;
    if (__any_sync(0xFFFFFFFFu, need) || grow) {
        const float m_new = need ? mt : r.m;
        float alpha = need ? ex2(r.m - m_new) : 1.f;
        r.l *= alpha;
        r.lx *= alpha;
        r.m = m_new;
        if constexpr (F8)
            if (grow) alpha = r.fexp - fexp < -126 ? 0.f : alpha * tc_pow2(r.fexp - fexp);
        if (!first) {
            stable();
            const uint64_t a2 = f2(alpha, alpha);
#pragma unroll 1
            for (int cc = 0; cc < ncols; cc += 16) {
                uint32_t o[16];
                tc_ld16(tO + cc, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    float u, v;
                    f2_split(f2_mul(f2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), a2), u, v);
                    o[i] = __float_as_uint(u);
                    o[i + 1] = __float_as_uint(v);
                }
                tmem_st16(tO + cc, o);
            }
        }
    }
    if constexpr (F8) r.fexp = fexp;
    const float m = (r.m == -INFINITY ? 0.f : r.m) - kTcLift<F8>;
    if constexpr (!F8) {
        // the largest weight is its rounded P: its error enters l too
        const float pm = mx == -INFINITY ? 0.f : ex2(fmaf(mx, c, -m));
        r.l += bf16lo_to_f32(pack_bf16x2(pm, 0.f)) - pm;
    }
    const uint64_t c2 = f2(c, c), nm2 = f2(-m, -m);
    uint64_t s0 = 0, s1 = 0, s2 = 0, s3 = 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int col = 32 * g + 2 * i;
            float a, b;
            f2_split(f2_fma(f2(__uint_as_float(sr[col]), __uint_as_float(sr[col + 1])), c2, nm2), a, b);
            const float p0 = ex2(a), p1 = ex2(b);
            switch (i & 3) {
                case 0: s0 = f2_add(s0, f2(p0, p1)); break;
                case 1: s1 = f2_add(s1, f2(p0, p1)); break;
                case 2: s2 = f2_add(s2, f2(p0, p1)); break;
                default: s3 = f2_add(s3, f2(p0, p1)); break;
            }
            pk[i] = F8 ? tc_pack_f16(p0, p1) : pack_bf16x2(p0, p1);
        }
        tmem_st16(tS + 16 * g, pk);
    }
    float u, v;
    f2_split(f2_add(f2_add(s0, s1), f2_add(s2, s3)), u, v);
    r.l += u + v;
    r.lx += u + v;
}

// Q rows of a stream's tile into shared memory: this warp's 32 rows, D / 8 lanes
// a row (rows past the last repeat it), 128-byte swizzled 64-column halves.
// `row_at`: where this lane's own row starts in Q.
template <int D, bool F8>
__device__ __forceinline__ void tc_load_q(const TreeParams& p, size_t row_at, int wq, int lane, uint32_t tile,
                                          float* qs) {
    constexpr int kLanes = D / 8;      // lanes of a row
    constexpr int kPer = 32 / kLanes;  // rows of an instruction
    const int c = lane % kLanes;
    const bool in = 8 * c < p.dh;
    const __nv_bfloat16* q = p.q + (in ? 8 * c : 0);
#pragma unroll 1
    for (int i0 = 0; i0 < 32 / kPer; i0 += 8) {  // eight loads of a lane in flight
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const size_t at = __shfl_sync(0xFFFFFFFFu, (unsigned long long)row_at, (i0 + i) * kPer + lane / kLanes);
            v[i] = __ldg(reinterpret_cast<const uint4*>(q + at));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = wq * 32 + (i0 + i) * kPer + lane / kLanes;
            uint32_t w[4] = {in ? v[i].x : 0u, in ? v[i].y : 0u, in ? v[i].z : 0u, in ? v[i].w : 0u};
            if constexpr (F8) {
                float mx = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mx = fmaxf(mx, fmaxf(fabsf(bf16lo_to_f32(w[e])), fabsf(bf16hi_to_f32(w[e]))));
#pragma unroll
                for (int off = kLanes / 2; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
                // a power of two that puts the row's largest value in [2^7, 2^8).  A bf16
                // value is then the sum of two E4M3 ones, exactly down to 2^-9 of the
                // largest, and to 2^-17 of the largest below that.
                int e = (int)(__float_as_uint(mx) >> 23) - 127;
                const bool inf = e > 127;
                e = e < -100 ? -100 : (e > 126 ? 126 : e);
                const float up = inf ? __uint_as_float(0x7FFFFFFFu) : tc_pow2(7 - e);  // (an infinity: the row is NaN)
                if (c == 0) qs[row] = p.c * tc_pow2(e - 7);
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float f[4] = {bf16lo_to_f32(w[2 * k]) * up, bf16hi_to_f32(w[2 * k]) * up,
                                        bf16lo_to_f32(w[2 * k + 1]) * up, bf16hi_to_f32(w[2 * k + 1]) * up};
                    hi[k] = pack_e4m3x2(f[0], f[1]) | pack_e4m3x2(f[2], f[3]) << 16;
                    uint32_t a, b;
                    tc_e4m3x4(hi[k], a, b);
                    const float2 g0 = tc_f16x2_f32(a), g1 = tc_f16x2_f32(b);
                    lo[k] = pack_e4m3x2(f[0] - g0.x, f[1] - g0.y) | pack_e4m3x2(f[2] - g1.x, f[3] - g1.y) << 16;
                }
                const uint32_t at = tile + row * 128 + (((c >> 1) ^ (row & 7)) << 4) + 8 * (c & 1);
                tc_sts64(at, hi[0], hi[1]);
                tc_sts64(at + 16384, lo[0], lo[1]);
            } else {
                sts128(tile + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// A thread's row of a piece: `row` of the item, drafted token `tok`, row `bht` of
// Q and O; `rows` of the warpgroup's tile are live.
struct TcMine {
    int rows, row, tok;
    size_t bht;
};
__device__ __forceinline__ TcMine tc_mine(const TreeParams& p, const TcPiece& x, int t, int me) {
    TcMine a;
    const int row0 = x.pair ? 128 * t : 0;
    a.rows = min(128, x.rows - row0);
    a.row = row0 + min(me, a.rows - 1);
    const int r = x.w.rt * kTcRows + a.row;
    a.tok = r / p.G;
    a.bht = ((size_t)x.w.b * p.Hq + (size_t)x.w.h * p.G + (r - a.tok * p.G)) * p.T + a.tok;
    return a;
}
// What a thread needs to write its row.
struct TcOut {
    int row, tok;      // row of the item, its drafted token
    bool live, two;    // inside the item; both streams hold a part
    float inv0, inv1;  // factors of stream 0's and 1's O
    float m, inv;      // maximum and 1 / sum of the row (for rows added apart)
    size_t bht, place;
};

// Columns [col0, col1) of the row: a partial result goes out a column at a time
// (32 rows side by side), a whole one 32 or 64 bytes of the row at a time.
__device__ __forceinline__ void tc_write(const TreeParams& p, const TcPiece& x, const TcOut& o, uint32_t tA, int col0,
                                         int col1) {
    float* part = p.ws_o + (o.place * kTcRows + (o.row & ~31)) * p.dw + (threadIdx.x & 31);
    const size_t at = o.bht * p.dh;
#pragma unroll 1
    for (int cc = col0; cc < col1; cc += 16) {
        uint32_t a[16], b[16];
        tc_ld16(tA + cc, a);
        if (o.two) tc_ld16(tA + 128 + cc, b);
        tmem_wait_ld();
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            v[i] = __uint_as_float(a[i]) * o.inv0;
            if (o.two) v[i] = fmaf(__uint_as_float(b[i]), o.inv1, v[i]);
        }
        if (!x.w.whole) {
            if (o.live) {
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(cc + i) * 32] = v[i];
            }
        } else if (o.live && p.out_f32) {
            float* out = static_cast<float*>(p.o) + at + cc;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (cc + 4 * i < p.dh)
                    reinterpret_cast<float4*>(out)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else if (o.live) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + at + cc;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (cc + 8 * i < p.dh)
                    reinterpret_cast<uint4*>(out)[i] =
                        make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                   pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
        }
    }
}

// Eight bf16 values; eight E4M3 ones.
__device__ __forceinline__ void tc_values(uint4 v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16lo_to_f32(u[i]);
        f[2 * i + 1] = bf16hi_to_f32(u[i]);
    }
}
__device__ __forceinline__ void tc_values(uint32_t a, uint32_t b, float (&f)[8]) {
    uint32_t h[4];
    tc_e4m3x4(a, h[0], h[1]);
    tc_e4m3x4(b, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = tc_f16x2_f32(h[i]);
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}

// The same with the keys whose V rows were taken out of the product: O scaled (and the
// streams' added), then those keys that the row sees, with their scores computed anew in
// fp32 from the row of Q in shared memory.  Rare, so out of line.
template <int D, bool F8, bool ONE>
__device__ __noinline__ void tc_write_apart(const TreeParams& p, TcPiece x, TcOut o, uint32_t tA, int col0, int col1,
                                            const uint32_t* bad, const TcBars* bars, int tile) {
    const int me = threadIdx.x & 127;
    const uint32_t q = smem_u32(bars) - TcCfg<D, F8, ONE>::kBar + tile * TcCfg<D, F8, ONE>::kTile + me * 128;
    const float c = fmaxf(F8 ? bars->qs[tile][me] : p.c, 1e-37f);
#pragma unroll 1
    for (int cc = col0; cc < col1; cc += 16) {
        uint32_t a[16], b[16];
        tc_ld16(tA + cc, a);
        if (o.two) tc_ld16(tA + 128 + cc, b);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = __uint_as_float(a[i]) * o.inv0;
            if (o.two) v = fmaf(__uint_as_float(b[i]), o.inv1, v);
            a[i] = __float_as_uint(v);
        }
        tmem_st16(tA + cc, a);
    }
    tmem_wait_st();
    o.inv0 = 1.0f;
    o.two = false;
    const int key0 = (x.w.k0 + x.first_special()) * kTcKeys;
    const int end = min(x.w.k1 * kTcKeys, x.w.keys);
#pragma unroll 1
    for (int key = key0; key < end; ++key) {
        const int i = key - key0;
        if (!(*((const volatile uint32_t*)bad + (i >> 5)) >> (i & 31) & 1u)) continue;
        const bool sees = key < x.prefix || tree_sees(p, x.w.b, o.tok, key - x.prefix);
        if (!__any_sync(0xFFFFFFFFu, sees)) continue;
        int off;
        const int page = tree_page(p, x.w.b, key, x.w.keys, off);
        if (page < 0) continue;  // (zeros)
        const long long row = (((long long)page * p.page_size + off) * p.Hkv + x.w.h) * p.dh;
        const uint8_t* k = p.k_pages + row * (F8 ? 1 : 2);
        const uint8_t* v = p.v_pages + row * (F8 ? 1 : 2);
        float s = 0.f, vd = 1.f;
        if constexpr (F8) {
            const long long ds = ((long long)page * p.Hkv + x.w.h) * p.page_size + off;
#pragma unroll 1
            for (int ch = 0; ch < p.dh / 16; ++ch) {
                const uint32_t at = q + ((ch ^ (me & 7)) << 4);
                const uint4 a = tc_lds128(at), b = tc_lds128(at + 16384);
                const uint4 kc = __ldg(reinterpret_cast<const uint4*>(k) + ch);
                const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
                const uint32_t kw[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float fa[8], fb[8], fk[8];
                    tc_values(aw[2 * g], aw[2 * g + 1], fa);
                    tc_values(bw[2 * g], bw[2 * g + 1], fb);
                    tc_values(kw[2 * g], kw[2 * g + 1], fk);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s = fmaf(fa[e] + fb[e], fk[e], s);
                }
            }
            s *= __ldg(p.k_descale + ds);
            vd = __ldg(p.v_descale + ds);
        } else {
#pragma unroll 1
            for (int ch = 0; ch < p.dh / 8; ++ch) {
                float fq[8], fk[8];
                tc_values(tc_lds128(q + (ch >> 3) * 16384 + (((ch & 7) ^ (me & 7)) << 4)), fq);
                tc_values(__ldg(reinterpret_cast<const uint4*>(k) + ch), fk);
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(fq[e], fk[e], s);
            }
        }
        const float w = ex2(s * c - o.m + kTcLift<F8>) * o.inv;
#pragma unroll 1
        for (int cc = col0; cc < col1; cc += 16) {
            uint32_t a[16];
            tc_ld16(tA + cc, a);
            float f[2][8] = {};
            if constexpr (F8) {
                const uint4 vc = __ldg(reinterpret_cast<const uint4*>(v + cc));
                tc_values(vc.x, vc.y, f[0]);
                tc_values(vc.z, vc.w, f[1]);
            } else {
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    if (cc + 8 * g < p.dh) tc_values(__ldg(reinterpret_cast<const uint4*>(v + 2 * (cc + 8 * g))), f[g]);
            }
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (sees) a[e] = __float_as_uint(fmaf(w, f[e >> 3][e & 7] * vd, __uint_as_float(a[e])));
            tmem_st16(tA + cc, a);
        }
        tmem_wait_st();
    }
    tc_write(p, x, o, tA, col0, col1);
}

template <int D, bool F8, bool ONE>
__device__ void tc_softmax(int t, int wq, int lane, uint8_t* smem, TcBars* bars, uint32_t tmem, const TreeParams& p) {
    using C = TcCfg<D, F8, ONE>;
    const volatile int* abort_flag = &bars->abort;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lanes;
    const uint32_t tO = tmem + 256 + lanes;  // of stream 0; stream 1: + 128
    const int ncols = (p.dh + 15) / 16 * 16;
    const int me = wq * 32 + lane;
    uint32_t cnt_s = 0, cnt_x = 0, tiles = 0;
    bool ok = true;
    TreeWalk walk;
    walk.start(bars->range);
    TcPiece x;
    for (int piece = 0; ok && walk.next(p, x.w); ++piece) {
        x.set(p);
        const TcMine my = tc_mine(p, x, t, me);
        const bool active = wq * 32 < my.rows;  // (warp-uniform)
        if (x.pair || t == 0) {  // (stream 0's warps lay out a split piece's Q)
            if (active) tc_load_q<D, F8>(p, my.bht * p.dh, wq, lane, smem_u32(smem + t * C::kTile), bars->qs[t]);
            if (lane == 0) mbar_arrive(smem_u32(&bars->q_full[t]));
        }
        if constexpr (F8) {
            // a split piece's stream 1 reads the factors that stream 0's warps wrote
            if (!x.pair && t == 1) {
                ok = warp_wait(&bars->q_full[0], (uint32_t)piece, abort_flag);
                if (!ok) break;
            }
        }
        // (above zero, so that a masked -inf stays one)
        const float c = fmaxf(F8 ? *((volatile float*)&bars->qs[x.pair ? t : 0][me]) : p.c, 1e-37f);
        // the row's mask, if it fits in 64 bits (used at the piece's last tiles)
        uint2 mask = make_uint2(0xFFFFFFFFu, 0xFFFFFFFFu);
        if (p.mask && p.W == 1 && x.w.k1 * kTcKeys > x.prefix)
            mask = __ldg(reinterpret_cast<const uint2*>(p.mask + (size_t)x.w.b * p.T + my.tok));
        TcRow st;
        st.m = -INFINITY;
        st.l = st.lx = 0.f;
        st.fexp = -100;
        int s = 0;
        for (; x.has(s, t) && ok; ++s) {
            const int j = x.tile(s, t);
            // (descales are laid out in order, and this stream, or with `done` both, has used
            // those of the tile before: the place's last phase is over)
            const float* kf = nullptr;
            int fexp = 0;
            if constexpr (F8) {
                const uint32_t g = tiles + (uint32_t)j;
                const int slot = (int)(g % kDs);
                ok = warp_wait(&bars->ds_full[slot], g / kDs, abort_flag);
                if (!ok) break;
                kf = bars->kf[slot];
                fexp = *((volatile int*)&bars->fexp[slot]);
            }
            const bool special = x.special(j);
            ok = warp_wait(&bars->s_full[t], cnt_s, abort_flag, 32);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (active) {
                    uint32_t allow[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                    if (special)
                        tc_allow(p, x.w.b, my.tok, x.w.drafted, (x.w.k0 + j) * kTcKeys + 64 * h - x.prefix, mask,
                                 allow);
                    // (S was issued after the tile before; of this one the first half's product)
                    auto stable = [&]() {
                        if (h == 0) return;
                        ok = warp_wait(&bars->o_half[t], cnt_s, abort_flag);
                        tc_fence_after();
                    };
                    tc_softmax_half<F8>(tS + 64 * h, tO + 128 * t, F8 ? kf + 64 * h : nullptr, fexp, special, allow,
                                        s == 0 && h == 0, c, ncols, st, stable);
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[t][h]));
            }
            if (!ok) break;
            ++cnt_s;
            if constexpr (F8) {
                if (lane == 0) {
                    const uint32_t e = smem_u32(&bars->ds_empty[(tiles + (uint32_t)j) % kDs]);
                    mbar_arrive(e);
                    if (!x.pair) mbar_arrive(e);  // (the barrier counts both streams' warps)
                }
            }
        }
        if (!ok) break;
        tiles += (uint32_t)x.n;
        ok = warp_wait(&bars->o_full[t], (uint32_t)piece, abort_flag);
        if (!ok) break;
        tc_fence_after();
        // ---- epilogue
        float inv0, inv1 = 0.f, m = st.m, lx = st.lx, inv_l;  // factors of stream 0's and 1's O
        int col0 = 0, col1 = ncols;
        uint32_t tA = tO + 128 * t;
        if (x.pair) {
            inv_l = st.l == 0.f ? 0.f : 1.0f / st.l;
            inv0 = F8 ? inv_l * tc_pow2(st.fexp - kTcVLift) : inv_l;
        } else {
            // the streams' statistics meet in shared memory; each warpgroup
            // then merges half of the columns, both O's being in its lanes
            bars->m[t][me] = st.m;
            bars->l[t][me] = st.l;
            bars->lx[t][me] = st.lx;
            if (wq == 0 && lane == 0) bars->fin[t] = F8 ? tc_pow2(st.fexp - kTcVLift) : 1.f;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->stat));
            ok = warp_wait(&bars->stat, cnt_x, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const float m0 = bars->m[0][me], m1 = bars->m[1][me];
            m = fmaxf(m0, m1);
            const float ms = m == -INFINITY ? 0.f : m;
            const float a0 = ex2(m0 - ms), a1 = ex2(m1 - ms);
            const float l = a0 * bars->l[0][me] + a1 * bars->l[1][me];
            lx = a0 * bars->lx[0][me] + a1 * bars->lx[1][me];
            inv_l = l == 0.f ? 0.f : 1.0f / l;
            inv0 = a0 * inv_l * bars->fin[0];
            inv1 = a1 * inv_l * bars->fin[1];
            const int half = (ncols / 2 + 15) / 16 * 16;
            col0 = t == 0 ? 0 : half;
            col1 = t == 0 ? half : ncols;
            tA = tO;
        }
        const uint32_t* bad = &bars->bad[piece % kBadBufs][0][0];
        uint32_t any_bad = 0u;
        for (int i = 0; i < 4 * (x.n - x.first_special()); ++i) any_bad |= *((const volatile uint32_t*)bad + i);
        if (active) {
            TcOut o;
            o.row = my.row;
            o.live = me < my.rows;
            o.two = !x.pair && x.n > 1;
            o.inv0 = inv0;
            o.inv1 = inv1;
            o.m = m;
            o.inv = inv_l;
            o.tok = my.tok;
            o.bht = my.bht;
            o.place = (size_t)blockIdx.x * 2 + (piece == 0 ? 0 : 1);
            if (any_bad) tc_write_apart<D, F8, ONE>(p, x, o, tA, col0, col1, bad, bars, x.pair ? t : 0);
            else tc_write(p, x, o, tA, col0, col1);
            if (o.live && (x.pair || t == 0)) {
                const float lse2 = lx == 0.f ? -INFINITY : m - kTcLift<F8> + log2f(lx);
                if (!x.w.whole) p.ws_lse[o.place * kTcRows + my.row] = lse2;
                else if (p.lse) p.lse[my.bht] = lse2 * kTcLn2;
            }
        }
        // O, the statistics and the marks are read: the next piece may write them
        tc_fence_before();
        __syncwarp();
        if (!x.pair) {
            if (lane == 0) mbar_arrive(smem_u32(&bars->done));
            ok = warp_wait(&bars->done, cnt_x, abort_flag);
            ++cnt_x;
            tc_fence_after();
        }
    }
    if (!ok && lane == 0) tc_abort(bars, p.err);
}

template <int D, bool F8, bool ONE>
__global__ void __launch_bounds__((TcRoles<F8, ONE>::kThreads), 1)
attn_tree_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const __grid_constant__ TreeParams p) {
    using C = TcCfg<D, F8, ONE>;
    using Roles = TcRoles<F8, ONE>;
    constexpr int kIssuers = ONE ? 2 : 1;
    extern __shared__ __align__(1024) uint8_t smem[];
    TcBars* bars = reinterpret_cast<TcBars*>(smem + C::kBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {  // the swizzled boxes need 1024-byte bases
        if (threadIdx.x == 0) atomicOr(p.err, kErrLayout);
        return;
    }
    if (threadIdx.x == 64) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the merge waits by itself)
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bars->q_full[t]), 4);
            for (int h = 0; h < 2; ++h) {
                mbar_init(smem_u32(&bars->p_full[t][h]), 4);
            }
            mbar_init(smem_u32(&bars->s_full[t]), 1);
            mbar_init(smem_u32(&bars->o_half[t]), 1);
            mbar_init(smem_u32(&bars->o_full[t]), 1);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(smem_u32(&bars->full[i]), F8 ? Roles::kConverters : 1);
            mbar_init(smem_u32(&bars->empty[i]), kIssuers);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(&bars->k_full[i]), 1);
            mbar_init(smem_u32(&bars->k_empty[i]), kIssuers + 1);  // (and the descales)
            mbar_init(smem_u32(&bars->v_full[i]), 1);
            mbar_init(smem_u32(&bars->v_empty[i]), Roles::kConverters);
        }
        for (int i = 0; i < kDs; ++i) {
            mbar_init(smem_u32(&bars->ds_full[i]), 1);
            mbar_init(smem_u32(&bars->ds_empty[i]), 8 + Roles::kConverters);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bars->fix_ask[t]), 1);
            mbar_init(smem_u32(&bars->fix_done[t]), 1);
            mbar_init(smem_u32(&bars->drain[t]), 1);
        }
        mbar_init(smem_u32(&bars->stat), 8);
        mbar_init(smem_u32(&bars->done), 8);
        bars->abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        const TreeRange r = tree_range(p, blockIdx.x);
        if (lane == 0) bars->range = r;
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    if (warp < Roles::kControl) {
        reg_dealloc<Roles::kRegsControl>();
        constexpr int kFirstConverter = Roles::kControl - Roles::kConverters;
        if (warp == 1 || (ONE && warp == 2)) {
            if constexpr (ONE) tc_mma_stream<D, F8, ONE>(warp - 1, smem, bars, tmem, p);
            else tc_mma<D, F8, ONE>(smem, bars, tmem, p);
        } else if constexpr (Roles::kMany) {
            if (warp == 0) tc_produce_codes<false, C>(&tk, smem, bars, p);
            if (warp == 3) tc_produce_codes<true, C>(&tv, smem, bars, p);
        } else {
            if (warp == 0) tc_produce<D, F8, ONE>(&tk, &tv, smem, bars, p);
        }
        if constexpr (F8) {
            if (warp >= kFirstConverter) tc_convert<Roles::kConverters, C>(warp - kFirstConverter, smem, bars, p);
        } else {
            if (warp == 3) tc_fix<D, ONE>(smem, bars, p);
        }
    } else {
        reg_alloc<Roles::kRegsSoftmax>();
        tc_softmax<D, F8, ONE>((warp - Roles::kControl) >> 2, warp & 3, lane, smem, bars, tmem, p);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool F8, bool ONE>
attn_status_t launch_tc_t(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream,
                          const DeviceInfo& dev) {
    using C = TcCfg<D, F8, ONE>;
    static int attr_set[64] = {0};
    if (dev.device >= 64 || !attr_set[dev.device]) {
        if (cudaFuncSetAttribute(attn_tree_tc_kernel<D, F8, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem) != cudaSuccess)
            return ATTN_ERR_CUDA;
        if (dev.device < 64) attr_set[dev.device] = 1;
    }
    attn_tree_tc_kernel<D, F8, ONE><<<p.ctas, TcRoles<F8, ONE>::kThreads, C::kSmem, stream>>>(tk, tv, p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

void tree_tc_shape(TreeParams& p, bool f8, int num_sms) {
    p.tile_rows = kTcRows;
    p.tile_keys = kTcKeys;
    p.dw = p.dh <= 64 && !f8 ? 64 : 128;
    p.ctas = num_sms;
    p.min_units = 2;
    p.extra = 6;  // Q's layout, the first copies, O's way out (64 drafts: 245 us; 0: 308, 4: 250, 8: 247, 10: 250)
    p.group_rows = 32;
}

attn_status_t launch_tree_tc(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, bool f8,
                             cudaStream_t stream, const DeviceInfo& dev) {
    if (p.T * p.G <= 128) {
        if (f8) return launch_tc_t<128, true, true>(tk, tv, p, stream, dev);
        if (p.dw == 128) return launch_tc_t<128, false, true>(tk, tv, p, stream, dev);
        return launch_tc_t<64, false, true>(tk, tv, p, stream, dev);
    }
    if (f8) return launch_tc_t<128, true, false>(tk, tv, p, stream, dev);
    if (p.dw == 128) return launch_tc_t<128, false, false>(tk, tv, p, stream, dev);
    return launch_tc_t<64, false, false>(tk, tv, p, stream, dev);
}

}  // namespace gb300
