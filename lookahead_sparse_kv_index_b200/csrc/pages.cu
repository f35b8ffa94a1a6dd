// The pages of a paged cache: growing, forking, freeing, packing and copying (lsa_page_*).
//
// The books are whole numbers, so every result is exact and the same from run to run: new pages are the free ones of
// the lowest index, handed out in the order of the call's rows, and the counts change by integer atomics.  Growing and
// forking are one CTA: it adds up what the call needs, counts free pages from index 0 until they suffice (nothing is
// written before that), and lists them, round by round, for a thread each to hand to its row; 1024 threads take 16
// counts each a round, so a pool of 64K pages is four rounds a pass.  Their latency is what they cost: a free, a fork of
// 20 rows and its copies take 11 us.  New pages are looked for from the pool's front, which a pool in use holds: of pools
// nine tenths held, 64 pages for as many rows take 7 us of 8,000 pages, 29 us of 100,000 and 206 us of a million; a call
// that needs no page takes 6 to 8 us whatever the pool.  The copy of whole pages is bound by HBM: 202 MB copied to other pages take 62 us,
// the copy rate.
#include "paged.cuh"

namespace lsa {
namespace {

using paged::CacheView;
using paged::Span;

constexpr int kBooks = 1024;            // threads of a books kernel
constexpr int kPer = 16;                // counts a thread and round
constexpr int kRound = kBooks * kPer;
constexpr int kMaxRows = 65536;
constexpr int64_t kMaxPages = int64_t(1) << 24;

struct Books {
    int32_t *table, *len, *refs;
    int32_t n_rows, max_pages, page_size;
    int64_t n_pages;
};

// Inclusive sum over the block of one value a thread; *total is the block's.  `part`: 33 values of shared memory, which
// calls may use one after the other.
template <typename V>
__device__ __forceinline__ V block_scan(V v, V *part, V *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    V s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V up = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += up;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        V w = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const V up = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += up;
        }
        part[lane] = w;
    }
    __syncthreads();
    const V before = warp ? part[warp - 1] : 0;
    *total = part[31];
    __syncthreads();
    return before + s;
}

// The counts of the 16 pages of this thread in round `r`, and which of them are free (0), as a mask.
struct Counts {
    int4 v[kPer / 4];
    __device__ __forceinline__ void load(const Books &bk, int64_t r) {
        const int64_t p0 = r * kRound + int64_t(threadIdx.x) * kPer;
        if (p0 + kPer <= bk.n_pages && (reinterpret_cast<uintptr_t>(bk.refs) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < kPer / 4; ++i) v[i] = reinterpret_cast<const int4 *>(bk.refs + p0)[i];
        } else {
            auto one = [&](int i) { return p0 + i < bk.n_pages ? bk.refs[p0 + i] : 1; };
#pragma unroll
            for (int i = 0; i < kPer / 4; ++i) v[i] = make_int4(one(4 * i), one(4 * i + 1), one(4 * i + 2), one(4 * i + 3));
        }
    }
    __device__ __forceinline__ uint32_t free() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i)
            m |= (uint32_t(v[i].x == 0) | uint32_t(v[i].y == 0) << 1 | uint32_t(v[i].z == 0) << 2 |
                  uint32_t(v[i].w == 0) << 3)
                 << (4 * i);
        return m;
    }
};

// The pool's free pages, round by round (whole block).  Round 0's counts are asked for before anything else and their sum
// is kept: most calls end there.
struct Free {
    Counts counts0;
    int upto0, total0;      // free pages of round 0 up to and with this thread's, all of its
};
__device__ __forceinline__ int free_of(const Books &bk, const Free &f, int64_t r, uint32_t *mask, int *total, int *part) {
    if (r == 0) {
        *mask = f.counts0.free();
        *total = f.total0;
        return f.upto0;
    }
    Counts c;
    c.load(bk, r);
    *mask = c.free();
    return block_scan(__popc(*mask), part, total);
}

// Whether the pool has `need` free pages.
__device__ bool enough_free(const Books &bk, int64_t need, Free &f, int *part) {
    f.upto0 = block_scan(__popc(f.counts0.free()), part, &f.total0);
    int64_t have = f.total0;
    for (int64_t r = 1; have < need && r * kRound < bk.n_pages; ++r) {
        uint32_t m;
        int total;
        free_of(bk, f, r, &m, &total, part);
        have += total;
    }
    return have >= need;
}

// Hands the `need` lowest free pages out: give(k, page) for the k-th, by one thread.  A round's pages are listed first, so
// that neighbouring ones go to different threads (each handing out the free ones of its own sixteen, a call of 20 pages
// took 10 us more).  give may write the page's own count.  `list`: kRound places of shared memory.
template <typename F>
__device__ void hand_out(const Books &bk, int64_t need, const Free &f, int *part, uint16_t *list, F give) {
    int64_t given = 0;
    for (int64_t r = 0; given < need && r * kRound < bk.n_pages; ++r) {
        uint32_t m;
        int total;
        int at = free_of(bk, f, r, &m, &total, part) - __popc(m);
        for (; m; m &= m - 1) list[at++] = uint16_t(threadIdx.x * kPer + __ffs(m) - 1);
        __syncthreads();
        const int64_t left = need - given;
        const int take = left < total ? int(left) : total;
        for (int k = threadIdx.x; k < take; k += kBooks) give(given + k, int32_t(r * kRound + list[k]));
        __syncthreads();
        given += total;
    }
}

// Entries that row r holds, and the pages of n entries (both below 2^31).
__device__ __forceinline__ uint32_t held_entries(const Books &bk, int r) {
    const int64_t n = bk.len[r], reach = int64_t(bk.max_pages) * bk.page_size;
    return uint32_t(n < 0 ? 0 : n > reach ? reach : n);
}
__device__ __forceinline__ uint32_t pages_of(const Books &bk, uint32_t n) {
    return (n + uint32_t(bk.page_size) - 1) / uint32_t(bk.page_size);
}

// What the threads' items need, summed up to each thread: first[t] in shared memory, the sum is returned.  (A sum that
// 32 bits do not hold is more than any pool has, and first is not used.)
__device__ __forceinline__ int64_t prefix(int64_t mine, int32_t *first, int64_t *part) {
    int64_t total;
    first[threadIdx.x + 1] = int32_t(block_scan(mine, part, &total));
    if (threadIdx.x == 0) first[0] = 0;
    __syncthreads();
    return total;
}

// The thread whose items hold the k-th page: first[t] <= k < first[t + 1].
__device__ __forceinline__ int thread_of(const int32_t *first, int64_t k) {
    int lo = 0, hi = kBooks - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= k) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kBooks) page_grow(Books bk, const int32_t *__restrict__ add, int32_t *err) {
    __shared__ int64_t part64[33];
    __shared__ int32_t first[kBooks + 1];
    __shared__ int part[33];
    __shared__ uint16_t list[kRound];
    pdl_launch_dependents();
    pdl_wait();
    Free free;
    free.counts0.load(bk, 0);
    const int per = (bk.n_rows + kBooks - 1) / kBooks;
    const int r0 = min(bk.n_rows, int(threadIdx.x) * per), r1 = min(bk.n_rows, r0 + per);
    const int64_t reach = int64_t(bk.max_pages) * bk.page_size;
    // pages that row r holds and pages that it needs besides (more than it may have counts as past the end)
    auto need_of = [&](int r, uint32_t *have, bool *past) {
        const uint32_t n = held_entries(bk, r), more = add[r] > 0 ? add[r] : 0;
        *past |= int64_t(n) + more > reach;
        *have = pages_of(bk, n);
        return *past ? 0u : pages_of(bk, n + more) - *have;
    };
    int64_t need = 0;
    uint32_t have;
    bool past = false;
    for (int r = r0; r < r1; ++r) need += need_of(r, &have, &past);
    past = __syncthreads_or(past);
    const int64_t total = prefix(need, first, part64);
    if (past || !enough_free(bk, total, free, part)) {
        if (threadIdx.x == 0) raise_err(err, LSA_ERR_CAPACITY);
        return;
    }
    hand_out(bk, total, free, part, list, [&](int64_t k, int32_t page) {
        const int t = thread_of(first, k);
        int64_t at = first[t];
        uint32_t have;
        bool past = false;
        for (int r = t * per;; ++r) {
            const uint32_t n = need_of(r, &have, &past);
            if (k < at + n) {
                bk.table[int64_t(r) * bk.max_pages + have + (k - at)] = page;
                bk.refs[page] = 1;
                return;
            }
            at += n;
        }
    });
    __syncthreads();
    for (int r = r0; r < r1; ++r)
        if (add[r] > 0) bk.len[r] = int32_t(held_entries(bk, r) + add[r]);
}

// First half of a fork: checks the call and takes the new last pages.  A call that is refused leaves copy_src = -2, which
// the second half turns into -1.
__global__ void __launch_bounds__(kBooks) page_fork_take(Books bk, const int32_t *__restrict__ src,
                                                         const int32_t *__restrict__ dst, int n, int32_t *copy_src,
                                                         int32_t *copy_dst, int32_t *err) {
    __shared__ int64_t part64[33];
    __shared__ int32_t first[kBooks + 1];
    __shared__ int part[33];
    __shared__ uint16_t list[kRound];
    __shared__ uint32_t named[kMaxRows / 32];
    pdl_launch_dependents();
    pdl_wait();
    Free free;
    free.counts0.load(bk, 0);
    const int per = (n + kBooks - 1) / kBooks;
    const int i0 = min(n, int(threadIdx.x) * per), i1 = min(n, i0 + per);
    auto part_filled = [&](int i) { return held_entries(bk, src[i]) % uint32_t(bk.page_size) > 0; };
    for (int i = threadIdx.x; i < (bk.n_rows + 31) / 32; i += kBooks) named[i] = 0;
    __syncthreads();
    bool bad = false;
    int64_t need = 0;
    for (int i = i0; i < i1; ++i) {
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= bk.n_rows || d < 0 || d >= bk.n_rows) {
            bad = true;
        } else {
            need += part_filled(i);
            bad |= bk.len[d] != 0;
            bad |= (atomicOr(&named[d >> 5], 1u << (d & 31)) >> (d & 31)) & 1u;
        }
    }
    bad = __syncthreads_or(bad);
    if (!bad)      // a row that becomes a copy cannot be copied in the same call
        for (int i = i0; i < i1; ++i) bad |= (named[src[i] >> 5] >> (src[i] & 31)) & 1u;
    bad = __syncthreads_or(bad);
    const int64_t total = prefix(need, first, part64);
    if (bad || !enough_free(bk, total, free, part)) {
        if (threadIdx.x == 0) raise_err(err, bad ? LSA_ERR_INVALID : LSA_ERR_CAPACITY);
        for (int i = threadIdx.x; i < n; i += kBooks) {
            copy_src[i] = -2;
            copy_dst[i] = -1;
        }
        return;
    }
    for (int i = i0; i < i1; ++i) {
        if (!part_filled(i)) copy_src[i] = copy_dst[i] = -1;
    }
    hand_out(bk, total, free, part, list, [&](int64_t k, int32_t page) {
        const int t = thread_of(first, k);
        int64_t at = first[t];
        for (int i = t * per;; ++i) {
            const bool one = part_filled(i);
            if (one && k == at) {
                const uint32_t full = held_entries(bk, src[i]) / uint32_t(bk.page_size);
                const int32_t from = bk.table[int64_t(src[i]) * bk.max_pages + full];
                bk.table[int64_t(dst[i]) * bk.max_pages + full] = page;
                bk.refs[page] = 1;
                copy_src[i] = from < 0 || from >= bk.n_pages ? -1 : from;
                copy_dst[i] = page;
                return;
            }
            at += one;
        }
    });
}

// Second half, one CTA a fork: shares the full pages.
constexpr int kFork = 256;
__global__ void __launch_bounds__(kFork) page_fork_share(Books bk, const int32_t *__restrict__ src,
                                                         const int32_t *__restrict__ dst, int32_t *copy_src) {
    const int i = blockIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    __shared__ bool refused;
    if (threadIdx.x == 0) refused = copy_src[i] == -2;
    __syncthreads();
    if (refused) {
        if (threadIdx.x == 0) copy_src[i] = -1;
        return;
    }
    const int64_t s = src[i], d = dst[i];
    const uint32_t n = held_entries(bk, int(s));
    const int64_t full = n / uint32_t(bk.page_size), held = pages_of(bk, n);
    for (int64_t c = threadIdx.x; c < bk.max_pages; c += kFork) {
        if (c < full) {
            const int32_t page = bk.table[s * bk.max_pages + c];
            bk.table[d * bk.max_pages + c] = page;
            if (page >= 0 && page < bk.n_pages) atomicAdd(&bk.refs[page], 1);
        } else if (c >= held) {
            bk.table[d * bk.max_pages + c] = -1;
        }
    }
    if (threadIdx.x == 0) bk.len[d] = int32_t(n);
}

// One CTA a row: whoever takes its length to 0 frees its pages, so a row named twice is freed once.
__global__ void __launch_bounds__(kFork) page_free(Books bk, const int32_t *__restrict__ rows, int32_t *err) {
    __shared__ int held_s;
    pdl_launch_dependents();
    pdl_wait();
    const int r = rows[blockIdx.x];
    if (r < 0 || r >= bk.n_rows) {
        if (threadIdx.x == 0) raise_err(err, LSA_ERR_INVALID);
        return;
    }
    if (threadIdx.x == 0) {
        const int64_t n = atomicExch(&bk.len[r], 0), reach = int64_t(bk.max_pages) * bk.page_size;
        held_s = int(pages_of(bk, uint32_t(n < 0 ? 0 : n > reach ? reach : n)));
    }
    __syncthreads();
    const int held = held_s;
    for (int c = threadIdx.x; c < held; c += kFork) {
        int32_t *e = &bk.table[int64_t(r) * bk.max_pages + c];
        const int32_t page = *e;
        *e = -1;
        if (page < 0 || page >= bk.n_pages) {
            raise_err(err, LSA_ERR_INVALID);
        } else if (atomicSub(&bk.refs[page], 1) <= 0) {
            atomicAdd(&bk.refs[page], 1);
            raise_err(err, LSA_ERR_INVALID);
        }
    }
}

// ------------------------------------------------------------------ packing
// With L held pages, held(p) the held ones below p, and M the held ones at or past L: page p >= L that is held is move
// held(p) - held(L), and free page p < L takes move p - held(p); both run over 0 .. M - 1.
constexpr int kPack = 1024, kPackPages = kPack * 4;

__device__ __forceinline__ int held_of4(const Books &bk, int64_t p0, uint32_t *mask) {
    uint32_t m = 0;
    if (p0 + 4 <= bk.n_pages && (reinterpret_cast<uintptr_t>(bk.refs) & 15) == 0) {
        const int4 v = *reinterpret_cast<const int4 *>(bk.refs + p0);
        m = uint32_t(v.x > 0) | uint32_t(v.y > 0) << 1 | uint32_t(v.z > 0) << 2 | uint32_t(v.w > 0) << 3;
    } else {
        for (int i = 0; i < 4; ++i)
            if (p0 + i < bk.n_pages && bk.refs[p0 + i] > 0) m |= 1u << i;
    }
    *mask = m;
    return __popc(m);
}

__global__ void __launch_bounds__(kPack) pack_count(Books bk, int32_t *cnt) {
    __shared__ int part[33];
    pdl_launch_dependents();
    pdl_wait();
    uint32_t m;
    int total;
    block_scan(held_of4(bk, int64_t(blockIdx.x) * kPackPages + threadIdx.x * 4, &m), part, &total);
    if (threadIdx.x == 0) cnt[blockIdx.x] = total;
}

// Three sums over the block at once (whole block; `part`: [3][32] of shared memory).
__device__ __forceinline__ void block_sum3(int (&v)[3], int (*part)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        v[i] = __reduce_add_sync(0xffffffffu, v[i]);
        if (lane == 0) part[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = __reduce_add_sync(0xffffffffu, part[i][lane]);
    __syncthreads();
}

// A pool of up to so many pages is counted by every block for itself, which takes less than a launch: 4096 pages 8.6 us
// against 9.9, 16384 pages 10.5 against 10.8, but 32768 pages 12.5 against 11.1.
constexpr int64_t kSmallPool = 4 * kPackPages;

__global__ void __launch_bounds__(kPack) pack_moves(Books bk, const int32_t *__restrict__ cnt, int blocks,
                                                    int32_t *__restrict__ rank, int32_t *move_src, int32_t *move_dst,
                                                    int32_t *n_moves) {
    __shared__ int part[33], part3[3][32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t p0 = int64_t(blockIdx.x) * kPackPages + threadIdx.x * 4;
    uint32_t m;
    const int mine = held_of4(bk, p0, &m);
    // all held pages, those of the blocks before this one
    int sum[3] = {0, 0, 0};
    if (bk.n_pages <= kSmallPool) {
        for (int64_t p = threadIdx.x * 4; p < bk.n_pages; p += kPackPages) {
            uint32_t any;
            const int c = held_of4(bk, p, &any);
            sum[0] += c;
            if (p < int64_t(blockIdx.x) * kPackPages) sum[1] += c;
        }
    } else {
        for (int i = threadIdx.x; i < blocks; i += kPack) {
            sum[0] += cnt[i];
            if (i < int(blockIdx.x)) sum[1] += cnt[i];
        }
    }
    block_sum3(sum, part3);
    const int L = sum[0], block_before = sum[1];
    // held(L): with the counts at hand, the blocks before L's and the pages of its block below L
    int front[3] = {0, 0, 0};
    const int lb = bk.n_pages <= kSmallPool ? 0 : L / kPackPages;
    for (int i = threadIdx.x; i < lb; i += kPack) front[0] += cnt[i];
    for (int64_t p = int64_t(lb) * kPackPages + threadIdx.x * 4; p < L; p += kPackPages) {
        uint32_t any;
        held_of4(bk, p, &any);
        if (p + 4 > L) any &= (1u << (L - p)) - 1u;
        front[0] += __popc(any);
    }
    block_sum3(front, part3);
    const int held_front = front[0], M = L - held_front;

    int all;
    int held = block_before + block_scan(mine, part, &all) - mine;
    for (int i = 0; i < 4; ++i) {
        const int64_t p = p0 + i;
        if (p >= bk.n_pages) break;
        const bool live = (m >> i) & 1u;
        int rk = -1;
        if (live && p >= L) {
            rk = held - held_front;
            move_src[rk] = int32_t(p);
        } else if (!live && p < L) {
            rk = int(p) - held;
            move_dst[rk] = int32_t(p);
        }
        rank[p] = rk;
        if (p >= M) move_src[p] = move_dst[p] = -1;
        held += live;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *n_moves = M;
}

// refs_out and table_out, which may be the books' own: a move's two counts are written by its dst's thread alone.
__global__ void __launch_bounds__(kFork) pack_apply(Books bk, const int32_t *__restrict__ rank,
                                                    const int32_t *__restrict__ move_src,
                                                    const int32_t *__restrict__ move_dst, int32_t *table_out,
                                                    int32_t *refs_out) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t step = int64_t(gridDim.x) * kFork, me = int64_t(blockIdx.x) * kFork + threadIdx.x;
    for (int64_t p = me; p < bk.n_pages; p += step) {
        const int32_t rk = rank[p];
        if (rk < 0) {
            refs_out[p] = bk.refs[p];
        } else if (move_dst[rk] == p) {
            const int32_t s = move_src[rk];
            refs_out[p] = bk.refs[s];
            refs_out[s] = 0;
        }
    }
    const int64_t entries = int64_t(bk.n_rows) * bk.max_pages;
    for (int64_t i = me; i < entries; i += step) {
        const int32_t e = bk.table[i];
        int32_t to = e;
        if (e >= 0 && e < bk.n_pages) {
            const int32_t rk = rank[e];
            if (rk >= 0 && move_src[rk] == e) to = move_dst[rk];
        }
        table_out[i] = to;
    }
}

// --------------------------------------------------------------------- copy
// A page of K (or V) is `rows` runs of `run` 16-byte pieces; a run is the page itself where its rows lie side by side.
struct CopyArgs {
    CacheView cache;
    const int32_t *src, *dst, *count;
    int32_t n, both, scaled;
    int64_t run;                 // 16-byte pieces of a run
    int32_t rows;                // runs of a page
    int32_t inner;               // runs along the inner of the page's two extents
    int64_t outer_stride, inner_stride;   // bytes
    int32_t parts;               // CTA-sized parts of a page (K, and V behind it)
    int32_t *err;
};
constexpr int kCopy = 256, kCopyUnroll = 8, kPart = kCopy * kCopyUnroll;   // 16-byte pieces of a part

__global__ void __launch_bounds__(kCopy) page_copy(CopyArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    int64_t n = a.n;
    if (a.count) {
        const int64_t c = *a.count;
        n = c < 0 ? 0 : c < n ? c : n;
    }
    const int64_t pieces = a.run * a.rows;      // of a page of K
    const int per = a.parts * (a.both ? 2 : 1);
    for (int64_t w = blockIdx.x; w < n * per; w += gridDim.x) {
        const int64_t i = w / per;
        int part = int(w - i * per);
        const int32_t s = a.src[i], d = a.dst[i];
        if (s < 0 || d < 0 || s == d) continue;
        if (s >= a.cache.n_pages || d >= a.cache.n_pages) {
            if (threadIdx.x == 0) raise_err(a.err, LSA_ERR_INVALID);
            continue;
        }
        const bool second = part >= a.parts;
        if (second) part -= a.parts;
        uint8_t *base = second ? a.cache.v : a.cache.k;
        const uint8_t *from = base + s * a.cache.page_stride;
        uint8_t *to = base + d * a.cache.page_stride;
        const int64_t p0 = int64_t(part) * kPart + threadIdx.x;
        uint4 v[kCopyUnroll];
        int64_t off[kCopyUnroll];
#pragma unroll
        for (int j = 0; j < kCopyUnroll; ++j) {
            const int64_t p = p0 + j * kCopy;
            off[j] = -1;
            if (p < pieces) {
                if (a.rows == 1) {
                    off[j] = p * 16;
                } else {
                    const int r = int(p / a.run), o = r / a.inner;
                    off[j] = o * a.outer_stride + (r - o * a.inner) * a.inner_stride + (p - r * a.run) * 16;
                }
                v[j] = *reinterpret_cast<const uint4 *>(from + off[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < kCopyUnroll; ++j)
            if (off[j] >= 0) *reinterpret_cast<uint4 *>(to + off[j]) = v[j];
        if (a.scaled && part == 0) {
            float *sc = second ? a.cache.vs : a.cache.ks;
            const int64_t m = int64_t(a.cache.page_size) * a.cache.Hkv;
            for (int64_t j = threadIdx.x; j < m; j += kCopy) sc[d * m + j] = sc[s * m + j];
        }
    }
}

lsa_status check_books(const lsa_page_table *pt, const char *who, Books *bk) {
    LSA_CHECK_ARG(pt, "%s: the pages' books are required", who);
    LSA_CHECK_ARG(pt->table && pt->len && pt->refs, "%s: table, len and refs are required", who);
    LSA_CHECK_ARG(pt->n_rows >= 1 && pt->max_pages >= 1 && pt->page_size >= 1 && pt->n_pages >= 1,
                  "%s: n_rows=%d max_pages=%d page_size=%d n_pages=%lld must be positive", who, pt->n_rows,
                  pt->max_pages, pt->page_size, (long long)pt->n_pages);
    LSA_CHECK_SUPPORTED(pt->n_rows <= kMaxRows, "%s: n_rows=%d > %d", who, pt->n_rows, kMaxRows);
    LSA_CHECK_SUPPORTED(pt->n_pages <= kMaxPages, "%s: n_pages=%lld > %lld", who, (long long)pt->n_pages,
                        (long long)kMaxPages);
    LSA_CHECK_ARG(int64_t(pt->max_pages) * pt->page_size < (int64_t(1) << 31),
                  "%s: a table row reaches 2^31 entries or more", who);
    *bk = Books{pt->table, pt->len, pt->refs, pt->n_rows, pt->max_pages, pt->page_size, pt->n_pages};
    return LSA_OK;
}

struct BookSpans {
    Span s[3];
};
BookSpans book_spans(const Books &bk) {
    return {{{bk.table, int64_t(bk.n_rows) * bk.max_pages * 4, "the table"},
             {bk.len, int64_t(bk.n_rows) * 4, "len"},
             {bk.refs, bk.n_pages * 4, "refs"}}};
}

// Refuses a call whose lists share bytes with each other (a call's inputs, the first `inputs` of them, may) or the books.
template <int N>
lsa_status check_apart(const Span (&x)[N], int inputs, const Books &bk, const char *who) {
    for (int i = 0; i < N; ++i) {
        for (const Span &b : book_spans(bk).s)
            LSA_CHECK_ARG(!meet(x[i], b), "%s: %s overlaps %s", who, x[i].name, b.name);
        for (int j = 0; j < i; ++j)
            LSA_CHECK_ARG(i < inputs || !meet(x[i], x[j]), "%s: %s overlaps %s", who, x[i].name, x[j].name);
    }
    return LSA_OK;
}

int64_t pack_blocks(int64_t n_pages) { return (n_pages + kPackPages - 1) / kPackPages; }

}  // namespace
}  // namespace lsa

using namespace lsa;

extern "C" lsa_status lsa_page_grow(const lsa_page_table *pt, const int32_t *add, int32_t *err, void *stream) {
    clear_error();
    Books bk;
    const lsa_status s = check_books(pt, "lsa_page_grow", &bk);
    if (s != LSA_OK) return s;
    LSA_CHECK_ARG(add, "lsa_page_grow: add is required");
    LSA_CUDA(launch_pdl(page_grow, dim3(1), dim3(kBooks), 0, as_stream(stream), bk, add, err));
    LSA_LAUNCHED("page_grow");
    return LSA_OK;
}

extern "C" lsa_status lsa_page_fork(const lsa_page_table *pt, const int32_t *src, const int32_t *dst, int32_t n,
                                    int32_t *copy_src, int32_t *copy_dst, int32_t *err, void *stream) {
    clear_error();
    Books bk;
    const lsa_status s = check_books(pt, "lsa_page_fork", &bk);
    if (s != LSA_OK) return s;
    LSA_CHECK_ARG(n >= 0 && n <= pt->n_rows, "lsa_page_fork: n=%d not in [0, n_rows]", n);
    if (n == 0) return LSA_OK;
    LSA_CHECK_ARG(src && dst && copy_src && copy_dst, "lsa_page_fork: src, dst, copy_src and copy_dst are required");
    const Span lists[] = {{src, int64_t(n) * 4, "src"}, {dst, int64_t(n) * 4, "dst"}, {copy_src, int64_t(n) * 4, "copy_src"},
                          {copy_dst, int64_t(n) * 4, "copy_dst"}};
    const lsa_status apart = check_apart(lists, 2, bk, "lsa_page_fork");
    if (apart != LSA_OK) return apart;
    cudaStream_t st = as_stream(stream);
    LSA_CUDA(launch_pdl(page_fork_take, dim3(1), dim3(kBooks), 0, st, bk, src, dst, int(n), copy_src, copy_dst, err));
    LSA_LAUNCHED("page_fork_take");
    LSA_CUDA(launch_pdl(page_fork_share, dim3(n), dim3(kFork), 0, st, bk, src, dst, copy_src));
    LSA_LAUNCHED("page_fork_share");
    return LSA_OK;
}

extern "C" lsa_status lsa_page_free(const lsa_page_table *pt, const int32_t *rows, int32_t n, int32_t *err,
                                    void *stream) {
    clear_error();
    Books bk;
    const lsa_status s = check_books(pt, "lsa_page_free", &bk);
    if (s != LSA_OK) return s;
    LSA_CHECK_ARG(n >= 0, "lsa_page_free: n=%d < 0", n);
    if (n == 0) return LSA_OK;
    LSA_CHECK_ARG(rows, "lsa_page_free: rows is required");
    const Span lists[] = {{rows, int64_t(n) * 4, "rows"}};
    const lsa_status apart = check_apart(lists, 1, bk, "lsa_page_free");
    if (apart != LSA_OK) return apart;
    LSA_CUDA(launch_pdl(page_free, dim3(n), dim3(kFork), 0, as_stream(stream), bk, rows, err));
    LSA_LAUNCHED("page_free");
    return LSA_OK;
}

extern "C" size_t lsa_page_compact_workspace_size(int64_t n_pages) {
    if (n_pages < 1 || n_pages > kMaxPages) return 0;
    return align_up(size_t(pack_blocks(n_pages)) * 4, 256) + align_up(size_t(n_pages) * 4, 256);
}

extern "C" lsa_status lsa_page_compact(const lsa_page_table *pt, int32_t *table_out, int32_t *refs_out,
                                       int32_t *move_src, int32_t *move_dst, int32_t *n_moves, void *workspace,
                                       size_t ws_bytes, void *stream) {
    clear_error();
    Books bk;
    const lsa_status s = check_books(pt, "lsa_page_compact", &bk);
    if (s != LSA_OK) return s;
    LSA_CHECK_ARG(table_out && refs_out && move_src && move_dst && n_moves && workspace,
                  "lsa_page_compact: table_out, refs_out, move_src, move_dst, n_moves and workspace are required");
    LSA_CHECK_ARG(ws_bytes >= lsa_page_compact_workspace_size(pt->n_pages) && aligned16(workspace),
                  "lsa_page_compact: workspace of %zu bytes < %zu", ws_bytes,
                  lsa_page_compact_workspace_size(pt->n_pages));
    // in place: the table and the counts as they are; anything else lies apart
    const int64_t table_bytes = int64_t(pt->n_rows) * pt->max_pages * 4, page_bytes = pt->n_pages * 4;
    const Span lists[] = {{table_out == pt->table ? nullptr : table_out, table_bytes, "table_out"},
                          {refs_out == pt->refs ? nullptr : refs_out, page_bytes, "refs_out"},
                          {move_src, page_bytes, "move_src"},
                          {move_dst, page_bytes, "move_dst"},
                          {n_moves, 4, "n_moves"},
                          {workspace, int64_t(lsa_page_compact_workspace_size(pt->n_pages)), "the workspace"}};
    const lsa_status apart = check_apart(lists, 0, bk, "lsa_page_compact");
    if (apart != LSA_OK) return apart;
    const int blocks = int(pack_blocks(pt->n_pages));
    int32_t *cnt = static_cast<int32_t *>(workspace);
    int32_t *rank = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + align_up(size_t(blocks) * 4, 256));
    cudaStream_t st = as_stream(stream);
    if (pt->n_pages > kSmallPool) {
        LSA_CUDA(launch_pdl(pack_count, dim3(blocks), dim3(kPack), 0, st, bk, cnt));
        LSA_LAUNCHED("pack_count");
    }
    LSA_CUDA(launch_pdl(pack_moves, dim3(blocks), dim3(kPack), 0, st, bk, static_cast<const int32_t *>(cnt), blocks,
                        rank, move_src, move_dst, n_moves));
    LSA_LAUNCHED("pack_moves");
    const int64_t most = int64_t(pt->n_rows) * pt->max_pages > pt->n_pages ? int64_t(pt->n_rows) * pt->max_pages
                                                                           : pt->n_pages;
    const int64_t want = (most + kFork - 1) / kFork;
    const int grid = int(want < int64_t(sm_count()) * 8 ? want : int64_t(sm_count()) * 8);
    LSA_CUDA(launch_pdl(pack_apply, dim3(grid), dim3(kFork), 0, st, bk, static_cast<const int32_t *>(rank),
                        static_cast<const int32_t *>(move_src), static_cast<const int32_t *>(move_dst), table_out,
                        refs_out));
    LSA_LAUNCHED("pack_apply");
    return LSA_OK;
}

extern "C" lsa_status lsa_page_copy(const lsa_page_cache *cache, const int32_t *src, const int32_t *dst, int32_t n,
                                    const int32_t *count, int32_t *err, void *stream) {
    clear_error();
    const lsa_status s = paged::check_cache(cache, "lsa_page_copy");
    if (s != LSA_OK) return s;
    LSA_CHECK_ARG(n >= 0, "lsa_page_copy: n=%d < 0", n);
    if (n == 0) return LSA_OK;
    LSA_CHECK_ARG(src && dst, "lsa_page_copy: src and dst are required");
    CopyArgs a = {};
    a.cache = paged::view_of(*cache);
    a.src = src;
    a.dst = dst;
    a.count = count;
    a.n = n;
    a.both = cache->v != cache->k;
    a.scaled = cache->dtype == LSA_E4M3;
    a.err = err;
    // rows of a page as a grid of two extents, the one of the smaller stride inside; runs grow over extents without gaps
    const int64_t row = int64_t(cache->D) * int64_t(elem_size(cache->dtype));
    int64_t in_n = cache->Hkv, in_s = a.cache.head_stride, out_n = cache->page_size, out_s = a.cache.slot_stride;
    if (out_n > 1 && (in_n == 1 || out_s < in_s)) {
        std::swap(in_n, out_n);
        std::swap(in_s, out_s);
    }
    a.run = row / 16;
    if (in_n == 1 || in_s == row) {
        a.run *= in_n;
        in_s = row * in_n;
        in_n = 1;
        if (out_n == 1 || out_s == in_s) {
            a.run *= out_n;
            out_n = 1;
        }
    }
    LSA_CHECK_SUPPORTED(int64_t(cache->page_size) * cache->Hkv < (int64_t(1) << 31),
                        "lsa_page_copy: a page of 2^31 rows or more");
    a.inner = int32_t(in_n);
    a.rows = int32_t(in_n * out_n);
    a.inner_stride = in_s;
    a.outer_stride = out_s;
    // (rows of up to 2 KB: at most 2^27 parts)
    a.parts = int32_t((a.run * a.rows + kPart - 1) / kPart);
    const int64_t work = int64_t(n) * a.parts * (a.both ? 2 : 1);
    const int64_t most = int64_t(sm_count()) * 8;
    LSA_CUDA(launch_pdl(page_copy, dim3(unsigned(work < most ? work : most)), dim3(kCopy), 0, as_stream(stream), a));
    LSA_LAUNCHED("page_copy");
    return LSA_OK;
}
