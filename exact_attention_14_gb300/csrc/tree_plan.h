// tree_plan.h -- how the tree-attention kernels share out their work.
//
// An item is (sequence b, KV head h, tile of query rows rt); the rows of a
// (sequence, KV head) are its drafted tokens times the group's heads, row
// t * G + g.  An item's units are its key tiles, after `extra` units that stand
// for the time its start and end take.  Items lie one after another
// (b, then h, then rt) and CTA c of n takes the units [c * total / n,
// (c + 1) * total / n): every CTA has the same number of key tiles to read,
// whatever the lengths are, and an item is cut only where a CTA's range ends.
// The lengths live on the device, so each CTA works the ranges out itself.  An item
// has all key tiles of its sequence, those that no row of its tile sees too: a chain of
// 1024 tokens (4 sequences, 32 / 8 heads of 128, bf16) takes 217 us without a prefix and
// 608 us after 8192 keys, where its visible products need 18 and 307 us.
// A piece that is not a whole item leaves a partial result in the workspace:
// a CTA has at most two such pieces, its first (place 2c) and its last
// (2c + 1), so the workspace does not grow with the batch.  The merge kernel
// redoes the same arithmetic to find an item's pieces.
#pragma once

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {

struct TreeParams {
    int B, Hq, Hkv, G, T, W;   // W: mask words of a row
    int max_blocks, page_size;
    int box_keys;              // keys of one copy: the largest of 16, 32, 64, 128 that divides the page and the tile
    long long num_blocks;
    int dh;                    // head dim of the tensors
    int ctas;                  // grid size of the attention kernel
    int min_units;             // units of a CTA, at least: 2 (3 sequences of 2000..4000 keys, 7 drafts: 1 22.6, 2 18.9, 4 20.3 us)
    int extra;                 // an item's start and end, in key tiles
    int tile_keys, tile_rows;
    float c;                   // scale * log2(e)
    const int* block_table;
    const int* seqlens;
    const int* q_lens;         // NULL: T everywhere
    const unsigned long long* mask;  // NULL: drafted token t sees tokens 0..t
    const float* k_descale;
    const float* v_descale;
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const __nv_bfloat16* q;
    void* o;
    float* lse;
    float* ws_o;               // [2 * ctas][tile_rows / group_rows][dw][group_rows]
    float* ws_lse;             // [2 * ctas][tile_rows], base 2
    int dw;                    // columns of a partial row
    int group_rows;            // 8, 16 or 32: rows that lie next to each other in a partial
    int out_f32;
    unsigned int* err;
};

// A sequence of the batch: keys, drafted tokens, row tiles and key tiles of
// its items.  Lengths out of range count as no drafted tokens at all.
struct TreeSeq {
    int keys, drafted, row_tiles, key_tiles;
    bool bad;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
    TreeSeq s;
    s.keys = __ldg(p.seqlens + b);
    s.drafted = p.q_lens ? __ldg(p.q_lens + b) : p.T;
    s.bad = s.keys < 0 || (long long)s.keys > (long long)p.max_blocks * p.page_size || s.drafted < 0 ||
            s.drafted > p.T || s.drafted > s.keys;
    if (s.bad) s.keys = s.drafted = 0;
    s.row_tiles = (s.drafted * p.G + p.tile_rows - 1) / p.tile_rows;
    s.key_tiles = (s.keys + p.tile_keys - 1) / p.tile_keys;
    return s;
}
__device__ __forceinline__ long long tree_units(const TreeParams& p, const TreeSeq& s) {
    return s.key_tiles == 0 ? 0 : (long long)p.Hkv * s.row_tiles * (s.key_tiles + p.extra);
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// Units of the whole batch, and of the sequences before b (a full warp calls).
__device__ __forceinline__ long long tree_total_base(const TreeParams& p, int b, long long& base) {
    const int lane = threadIdx.x & 31;
    long long n = 0, before = 0;
    for (int i = lane; i < p.B; i += 32) {
        const long long units = tree_units(p, tree_seq(p, i));
        n += units;
        if (i < b) before += units;
    }
    base = warp_sum(before);
    return warp_sum(n);
}

// CTAs that take part, and the first unit of CTA c of them.
__device__ __forceinline__ int tree_ctas(const TreeParams& p, long long total) {
    const long long want = (total + p.min_units - 1) / p.min_units;
    return (int)(want < p.ctas ? (want < 1 ? 1 : want) : p.ctas);
}
__device__ __forceinline__ long long tree_div(long long a, long long b) {  // (64-bit divisions take hundreds of cycles)
    return (a | b) <= 0xFFFFFFFFll ? (long long)((unsigned)a / (unsigned)b) : a / b;  // (neither below 0)
}
__device__ __forceinline__ long long tree_first(long long total, int n, int c) { return tree_div(total * c, n); }

// A CTA's place in the list of units: its range, and the sequence that holds
// its first unit (`base`: units before that sequence).
struct TreeRange {
    long long u0, u1, base;
    int b;
};

// Found by a full warp; the same in every lane.
__device__ __forceinline__ TreeRange tree_range(const TreeParams& p, int cta) {
    const int lane = threadIdx.x & 31;
    TreeRange r;
    r.u0 = r.u1 = r.base = 0;
    r.b = 0;
    // the first 32 sequences' units stay in registers for the second look
    long long first = 0, sum = 0;
    for (int b = lane; b < p.B; b += 32) {
        const TreeSeq s = tree_seq(p, b);
        if (s.bad && cta == 0) atomicOr(p.err, kErrBadSeqlen);
        const long long units = tree_units(p, s);
        if (b < 32) first = units;
        sum += units;
    }
    const long long total = warp_sum(sum);
    const int n = tree_ctas(p, total);
    if (cta >= n || total == 0) return r;
    r.u0 = tree_first(total, n, cta);
    r.u1 = tree_first(total, n, cta + 1);
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const long long mine = b0 == 0 ? first : (b < p.B ? tree_units(p, tree_seq(p, b)) : 0);
        long long upto = mine;  // inclusive prefix sum over the lanes
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, off);
            if (lane >= off) upto += v;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, base + upto > r.u0);
        if (hit) {
            const int l = __ffs(hit) - 1;
            r.b = b0 + l;
            r.base = base + __shfl_sync(0xFFFFFFFFu, upto - mine, l);
            break;
        }
        base += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    return r;
}

// A piece of work: key tiles [k0, k1) of item (b, h, rt).
struct TreePiece {
    int b, h, rt, k0, k1;
    int keys, drafted;   // of the sequence
    bool whole;          // all of the item's key tiles
};

// Walks a range piece by piece; every role of a CTA walks its own copy.
struct TreeWalk {
    long long u, u1, base;
    int b;
    __device__ __forceinline__ void start(const TreeRange& r) {
        u = r.u0; u1 = r.u1; base = r.base; b = r.b;
    }
    __device__ __forceinline__ bool next(const TreeParams& p, TreePiece& w) {
        while (u < u1) {
            TreeSeq s = tree_seq(p, b);
            long long n = tree_units(p, s);
            while (u >= base + n) {  // ends: the units sum up to the total
                base += n;
                s = tree_seq(p, ++b);
                n = tree_units(p, s);
            }
            const long long at = u - base;
            const unsigned len = (unsigned)(s.key_tiles + p.extra);  // units of an item
            int from, item;
            if (at <= 0x7FFFFFFFll) {  // (64-bit divisions take hundreds of cycles)
                item = (int)((unsigned)at / len);
                from = (int)((unsigned)at - (unsigned)item * len);
            } else {
                item = (int)(at / len);
                from = (int)(at - (long long)item * len);
            }
            const long long left = u1 - u;
            const int to = left < (long long)len - from ? from + (int)left : (int)len;
            u += to - from;
            w.k0 = from < p.extra ? 0 : from - p.extra;
            w.k1 = to < p.extra ? 0 : to - p.extra;
            if (w.k1 <= w.k0) continue;  // nothing but the item's extra units
            w.h = (int)((unsigned)item / (unsigned)s.row_tiles);
            w.rt = item - w.h * s.row_tiles;
            w.b = b;
            w.keys = s.keys;
            w.drafted = s.drafted;
            w.whole = w.k0 == 0 && w.k1 == s.key_tiles;
            return true;
        }
        return false;
    }
};

// The page of the cache that holds key `key` of sequence b, -1 (reads as
// zeros) for keys past the sequence and for entries that name no page.
__device__ __forceinline__ int tree_page(const TreeParams& p, int b, int key, int keys, int& off) {
    const int blk = key / p.page_size;
    off = key - blk * p.page_size;
    if (key >= keys) return -1;
    const int page = __ldg(p.block_table + (size_t)b * p.max_blocks + blk);
    return page >= 0 && (long long)page < p.num_blocks ? page : -1;
}

// The descales of keys that have no page (their codes are zeros): up to 128.
static __device__ __align__(128) float kTreeNoDescale[128] = {};

// Whether row (drafted token t of sequence b) sees drafted token u.
__device__ __forceinline__ bool tree_sees(const TreeParams& p, int b, int t, int u) {
    if (!p.mask) return u <= t;
    const unsigned long long w = __ldg(p.mask + ((size_t)b * p.T + t) * p.W + (u >> 6));
    return (w >> (u & 63)) & 1ull;
}

// The kernel for many rows (attn_tree_tc_sm103.cu): its part of the
// parameters, and its launch.
void tree_tc_shape(TreeParams& p, bool f8, int num_sms);
attn_status_t launch_tree_tc(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, bool f8,
                             cudaStream_t stream, const DeviceInfo& dev);

// Merges the pieces of the items that were cut, and writes the rows past each
// sequence's drafted tokens (O = 0, LSE = -inf).
attn_status_t launch_tree_merge(const TreeParams& p, int num_sms, cudaStream_t stream);

}  // namespace gb300
