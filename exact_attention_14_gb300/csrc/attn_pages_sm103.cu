// attn_pages_sm103.cu -- block tables, cache slots and positions of a step's new
// tokens, built on the GPU from the requests' lengths; and pages taken back.
//
// The free pages are a stack in device memory.  With need_b = ceil((len_b + new_b) /
// page) - ceil(len_b / page) pages wanted by request b and P_b the sum of need over
// the requests before it, page i of the request's (i < need_b) is the stack's entry
// count - 1 - (P_b + i): a prefix sum over the requests decides everything, and no
// two threads compete for a page.  A request whose pages end past the stack
// (P_b + need_b > count) gets none; every later one that needs a page does not
// either, so the pages given are the first max(P_b + need_b) of the stack.
//
// Each block takes the prefix sums itself (at most 4096 requests, two loads each for the
// sums, and again where they go to shared memory: cheaper than a second launch), then a
// share of the tokens and pages; which request a token or page belongs to is a binary
// search in shared memory.  The lengths and the stack's count change only when every
// block has read them: the last to arrive, counted in the pool's second word, writes
// them.  Bound by latency (12 bytes a token leave): in a graph an extend and a trim take
// 9.4 us together for 16 requests of a token, 20.3 for 512 prompts of 17..4096 tokens, a
// million in all.
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kPagesThreads = 256;
constexpr int kPagesMaxRequests = 4096;
constexpr int kPoolHeader = 4;       // count, blocks arrived, two words unused
constexpr int kTokensPerThread = 4;  // two 16-byte stores of slots, one of positions

__device__ __forceinline__ int sat_add(int a, int b) {   // of numbers >= 0
    const unsigned s = (unsigned)a + (unsigned)b;
    return s > 0x7FFFFFFFu ? 0x7FFFFFFF : (int)s;
}

__device__ __forceinline__ int pages_of(int len, int page_size) {
    return (int)(((unsigned)len + (unsigned)page_size - 1u) / (unsigned)page_size);
}

// Exclusive prefix sum over the block's threads; `all`: the whole sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, s);
        if (lane >= s) x = sat_add(x, y);
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kPagesThreads / 32; ++w) {
        if (w == warp) before = all;
        all = sat_add(all, warp_sums[w]);
    }
    __syncthreads();
    const int up = __shfl_up_sync(0xFFFFFFFFu, x, 1);
    return sat_add(before, lane ? up : 0);
}

// The last index b with prefix[b] <= i, for prefix[0] = 0 and i < prefix[n].
__device__ __forceinline__ int find(const int* prefix, int n, int i) {
    int lo = 0, hi = n;   // prefix[lo] <= i < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// Whether this block is the launch's last to get here (uniform over its threads; at most
// 65535 blocks).  `flag`, of all threads alike: set on return if a block came with it set.
// Called behind a barrier of the block: what it read before is not read after, so the
// last one may overwrite it.
__device__ __forceinline__ bool last_block(int* pool, bool& flag) {
    __shared__ unsigned int seen;   // blocks before this one, and above them how many had it set
    if (threadIdx.x == 0) {
        const unsigned int mine = flag ? 1u << 16 : 0u;
        seen = mine;
        if (gridDim.x > 1) {
            __threadfence();
            seen = atomicAdd(reinterpret_cast<unsigned int*>(pool) + 1, 1u + mine) + mine;
            __threadfence();
        }
    }
    __syncthreads();
    flag = seen >> 16;
    return (seen & 0xFFFFu) == gridDim.x - 1;
}

struct ExtendArgs {
    int* pool;
    int num_blocks;
    int* block_table;
    int* seqlens;
    const int* new_lens;
    long long* slots;
    int* positions;    // may be NULL
    int* cu_seqlens;   // packed rows, or NULL
    int* granted;      // may be NULL
    int B, max_blocks, page_size;
    int width;         // > 0: rows [B, width]; 0: packed
    int total;         // rows
};

// Request b's length and new tokens; a request that cannot be (a negative length,
// more tokens than its row of the table holds or its padded row has) has none.
__device__ __forceinline__ bool request(const ExtendArgs& a, int b, int& len, int& add) {
    len = a.seqlens[b];
    add = __ldg(a.new_lens + b);
    const long long room = (long long)a.max_blocks * a.page_size;
    const bool good = len >= 0 && add >= 0 && (long long)len + add <= room && (a.width == 0 || add <= a.width);
    if (!good) add = 0;
    if (len < 0 || len > room) len = 0;
    return good;
}

__global__ void __launch_bounds__(kPagesThreads)
attn_pages_extend_kernel(const ExtendArgs a, unsigned int* err) {
    __shared__ int rows[kPagesMaxRequests + 1];   // prefix sums: token rows,
    __shared__ int want[kPagesMaxRequests + 1];   // pages wanted
    __shared__ int warp_sums[kPagesThreads / 32];
    const int tid = threadIdx.x;
    int count = *reinterpret_cast<volatile int*>(a.pool);
    const bool count_ok = count >= 0 && count <= a.num_blocks;
    if (!count_ok) count = 0;
    bool bad = !count_ok;
    const int per = (a.B + kPagesThreads - 1) / kPagesThreads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    int r = 0, w = 0;
    for (int b = b0; b < b1; ++b) {
        int len, add;
        bad |= !request(a, b, len, add);
        r = sat_add(r, add);
        w = sat_add(w, pages_of(len + add, a.page_size) - pages_of(len, a.page_size));
    }
    int all_rows, all_want;
    r = block_scan(r, warp_sums, all_rows);
    w = block_scan(w, warp_sums, all_want);
    // packed rows for fewer tokens: from the first request whose tokens end past them on,
    // new tokens count as none (`at`: the sum with them, which says which requests these are)
    const int limit = a.width > 0 ? 0x7FFFFFFF : a.total;
    int at = r;
    if (all_rows > limit) {
        bad = true;
        r = w = 0;
        int end = at;
        for (int b = b0; b < b1; ++b) {
            int len, add;
            request(a, b, len, add);
            end = sat_add(end, add);
            if (end > limit) add = 0;
            r += add;
            w = sat_add(w, pages_of(len + add, a.page_size) - pages_of(len, a.page_size));
        }
        r = block_scan(r, warp_sums, all_rows);
        w = block_scan(w, warp_sums, all_want);
    }
    for (int b = b0; b < b1; ++b) {
        int len, add;
        request(a, b, len, add);
        at = sat_add(at, add);
        if (at > limit) add = 0;
        rows[b] = r;
        want[b] = w;
        r = sat_add(r, add);
        w = sat_add(w, pages_of(len + add, a.page_size) - pages_of(len, a.page_size));
    }
    if (tid == 0) {
        rows[a.B] = all_rows;
        want[a.B] = all_want;
    }
    __syncthreads();
    auto given = [&](int b) { return want[b + 1] == want[b] || want[b + 1] <= count; };
    const int* stack = a.pool + kPoolHeader;

    // slots and positions, kTokensPerThread rows at a time
    const int step = gridDim.x * kPagesThreads * kTokensPerThread;
    for (int n0 = (blockIdx.x * kPagesThreads + tid) * kTokensPerThread; n0 < a.total; n0 += step) {
        long long slot[kTokensPerThread];
        int pos[kTokensPerThread];
        int b = -1, len = 0, add = 0, first = 0, have = 0, page = -1, page_at = -1;
        bool ok = false;
#pragma unroll
        for (int i = 0; i < kTokensPerThread; ++i) {
            const int n = n0 + i;
            slot[i] = -1;
            pos[i] = 0;
            const bool row = n < a.total && (a.width > 0 || n < all_rows);
            if (!row) continue;
            if (b < 0 || (a.width > 0 ? n >= first + a.width : n >= rows[b + 1])) {
                b = a.width > 0 ? n / a.width : find(rows, a.B, n);
                first = a.width > 0 ? b * a.width : rows[b];
                request(a, b, len, add);
                have = pages_of(len, a.page_size);
                ok = given(b);
                page_at = -1;
            }
            const int t = n - first;
            if (t >= add) continue;
            const int p = len + t;
            pos[i] = p;
            if (!ok) continue;
            const int blk = (int)((unsigned)p / (unsigned)a.page_size);
            if (blk != page_at) {
                page_at = blk;
                page = blk < have ? __ldg(a.block_table + (size_t)b * a.max_blocks + blk)
                                  : __ldg(stack + (count - 1 - (want[b] + blk - have)));
            }
            if ((unsigned)page < (unsigned)a.num_blocks)
                slot[i] = (long long)page * a.page_size + (p - blk * a.page_size);
            else
                bad = true;
        }
        if (n0 + kTokensPerThread <= a.total) {   // (16-byte aligned arrays)
            longlong2* s = reinterpret_cast<longlong2*>(a.slots + n0);
            s[0] = make_longlong2(slot[0], slot[1]);
            s[1] = make_longlong2(slot[2], slot[3]);
            if (a.positions) *reinterpret_cast<int4*>(a.positions + n0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kTokensPerThread; ++i)
                if (n0 + i < a.total) {
                    a.slots[n0 + i] = slot[i];
                    if (a.positions) a.positions[n0 + i] = pos[i];
                }
        }
    }
    // the pages into the table (they lie behind every entry read above)
    const int pages = min(all_want, count);
    for (int i = blockIdx.x * kPagesThreads + tid; i < pages; i += gridDim.x * kPagesThreads) {
        const int b = find(want, a.B, i);
        if (!given(b)) continue;
        const int len = a.seqlens[b];
        a.block_table[(size_t)b * a.max_blocks + pages_of(len, a.page_size) + (i - want[b])] =
            __ldg(stack + (count - 1 - i));
    }
    if (blockIdx.x == 0) {
        for (int b = tid; b < a.B; b += kPagesThreads)
            if (a.granted) a.granted[b] = given(b) ? rows[b + 1] - rows[b] : 0;
        if (a.cu_seqlens)
            for (int b = tid; b <= a.B; b += kPagesThreads) a.cu_seqlens[b] = rows[b];
    }
    if (bad) atomicOr(err, kErrBadSeqlen);
    bool no_flag = false;
    __syncthreads();
    if (!last_block(a.pool, no_flag)) return;
    int taken = 0;
    for (int b = tid; b < a.B; b += kPagesThreads) {
        if (!given(b)) continue;
        const int add = rows[b + 1] - rows[b];
        if (add > 0) a.seqlens[b] += add;
        if (want[b + 1] > want[b]) taken = max(taken, want[b + 1]);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) taken = max(taken, __shfl_xor_sync(0xFFFFFFFFu, taken, s));
    if ((tid & 31) == 0) warp_sums[tid >> 5] = taken;
    __syncthreads();
    if (tid == 0) {
        for (int x = 0; x < kPagesThreads / 32; ++x) taken = max(taken, warp_sums[x]);
        if (count_ok) a.pool[0] = count - taken;
        a.pool[1] = 0;
    }
}

// Request b gives back the pages past its first keep_b tokens.  Freed page i (in
// the order of the requests, and of each one's table) becomes entry count + F - 1 -
// i of the stack, F of them in all, so a step's pages given back go out again in the
// same order.  What lies past the stack's count means nothing, so the pages are
// written there while they are checked, and the last block counts them in, or, where
// one of them was no page of the cache, leaves the call without effect.
__global__ void __launch_bounds__(kPagesThreads)
attn_pages_trim_kernel(int* pool, int num_blocks, const int* block_table, int* seqlens, const int* keep_lens,
                       int B, int max_blocks, int page_size, unsigned int* err) {
    __shared__ int freed[kPagesMaxRequests + 1];
    __shared__ int warp_sums[kPagesThreads / 32];
    const int tid = threadIdx.x;
    const int count = *reinterpret_cast<volatile int*>(pool);
    const long long room = (long long)max_blocks * page_size;
    bool bad = count < 0 || count > num_blocks;
    // tokens held and kept; a request whose length cannot be keeps what it has
    auto lens = [&](int b, int& now, int& keep) {
        now = seqlens[b];
        keep = min(max(__ldg(keep_lens + b), 0), now);
        const bool good = now >= 0 && now <= room;
        if (!good) now = keep = 0;
        return good;
    };
    const int per = (B + kPagesThreads - 1) / kPagesThreads;
    const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
    int f = 0, now, keep;
    for (int b = b0; b < b1; ++b) {
        bad |= !lens(b, now, keep);
        f = sat_add(f, pages_of(now, page_size) - pages_of(keep, page_size));
    }
    int all;
    f = block_scan(f, warp_sums, all);
    for (int b = b0; b < b1; ++b) {
        freed[b] = f;
        lens(b, now, keep);
        f = sat_add(f, pages_of(now, page_size) - pages_of(keep, page_size));
    }
    if (tid == 0) freed[B] = all;
    __syncthreads();
    // more pages than the cache has: some were given back twice; nothing is done
    const bool fits = count >= 0 && count <= num_blocks && all <= num_blocks - count;
    bad |= !fits;
    bool no_page = false;
    if (fits) {
        int* stack = pool + kPoolHeader;
        for (int i = blockIdx.x * kPagesThreads + tid; i < all; i += gridDim.x * kPagesThreads) {
            const int b = find(freed, B, i);
            lens(b, now, keep);
            const int page = __ldg(block_table + (size_t)b * max_blocks + pages_of(keep, page_size) + (i - freed[b]));
            no_page |= (unsigned)page >= (unsigned)num_blocks;
            stack[count + all - 1 - i] = page;
        }
    }
    if (bad || no_page) atomicOr(err, kErrBadSeqlen);
    no_page = __syncthreads_or(no_page);
    if (!last_block(pool, no_page)) return;
    if (fits && !no_page) {
        for (int b = tid; b < B; b += kPagesThreads)
            if (lens(b, now, keep) && keep < now) seqlens[b] = keep;
        if (tid == 0) pool[0] = count + all;
    }
    if (tid == 0) pool[1] = 0;
}

__global__ void __launch_bounds__(kPagesThreads) attn_pages_init_kernel(int* pool, int num_blocks) {
    for (long long i = blockIdx.x * (long long)kPagesThreads + threadIdx.x; i < (long long)num_blocks + kPoolHeader;
         i += (long long)gridDim.x * kPagesThreads)
        pool[i] = i >= kPoolHeader ? num_blocks - 1 - (int)(i - kPoolHeader) : (i == 0 ? num_blocks : 0);
}

}  // namespace

attn_status_t launch_pages_init(int* pool, int num_blocks, cudaStream_t stream) {
    const long long blocks = ((long long)num_blocks + kPoolHeader + kPagesThreads - 1) / kPagesThreads;
    attn_pages_init_kernel<<<(unsigned)(blocks < 1024 ? blocks : 1024), kPagesThreads, 0, stream>>>(pool, num_blocks);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t launch_pages_extend(int* pool, int num_blocks, int* block_table, int* seqlens, const int* new_lens,
                                  long long* slots, int* positions, int* cu_seqlens, int* granted, int B,
                                  int max_blocks, int page_size, int width, long long total,
                                  cudaStream_t stream, const DeviceInfo& dev) {
    if (B > kPagesMaxRequests) return ATTN_ERR_UNSUPPORTED;
    const ExtendArgs a{pool,    num_blocks, block_table, seqlens,    new_lens,  slots, positions,
                       cu_seqlens, granted,    B,           max_blocks, page_size, width, (int)total};
    const long long share = kPagesThreads * kTokensPerThread;
    const long long blocks = (total + share - 1) / share;
    const int grid = (int)(blocks < 1 ? 1 : blocks < 2 * dev.num_sms ? blocks : 2 * dev.num_sms);
    attn_pages_extend_kernel<<<grid, kPagesThreads, 0, stream>>>(a, dev.err_word);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t launch_pages_trim(int* pool, int num_blocks, const int* block_table, int* seqlens,
                                const int* keep_lens, int B, int max_blocks, int page_size,
                                cudaStream_t stream, const DeviceInfo& dev) {
    if (B > kPagesMaxRequests) return ATTN_ERR_UNSUPPORTED;
    // (how many pages come back is known on the device; the tables' size bounds it)
    const long long blocks = ((long long)B * max_blocks + 4 * kPagesThreads - 1) / (4 * kPagesThreads);
    const int grid = (int)(blocks < 1 ? 1 : blocks < dev.num_sms ? blocks : dev.num_sms);
    attn_pages_trim_kernel<<<grid, kPagesThreads, 0, stream>>>(pool, num_blocks, block_table, seqlens, keep_lens, B,
                                                               max_blocks, page_size, dev.err_word);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace gb300
