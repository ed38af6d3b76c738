// cache.cu -- the paged key/value cache around the verify step (sm_103a): reserving, forking and
// releasing pages, appending the new tokens' rows, committing a step.
//
// Everything here is bookkeeping on small arrays or a copy: no arithmetic on the values.  The
// bookkeeping is bound by latency (one launch each; reserve a second for its copies), append and
// the copies of commit and reserve by memory: 16-byte accesses, several in flight per thread.
#include <algorithm>

#include "cache.cuh"

namespace specrej {
namespace {

constexpr int kBookThreads = 1024;  // the one block of reserve

// Exclusive prefix sum over the block; *total is the block's sum.
template <int THREADS> __device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *total)
{
    __shared__ int64_t sums[THREADS / 32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, incl, d);
        incl += lane >= d ? y : 0;
    }
    __syncthreads();  // the sums of the scan before have been read
    if (lane == 31)
        sums[w] = incl;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        before += i < w ? sums[i] : 0;
        all += sums[i];
    }
    *total = all;
    return before + incl - x;
}

__global__ void __launch_bounds__(kCopyThreads) init_kernel(CacheView c)
{
    const int64_t n = (int64_t)gridDim.x * blockDim.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (int64_t i = t; i < c.num_pages; i += n) {
        c.free_pages[i] = (int32_t)i;
        c.ref[i] = 0;
    }
    for (int64_t i = t; i < c.num_requests; i += n)
        c.lens[i] = c.held[i] = 0;
    for (int64_t i = t; i < (int64_t)c.num_requests * c.max_pages; i += n)
        c.table[i / c.max_pages * c.table_stride + i % c.max_pages] = -1;
    if (t == 0) {
        *c.num_free = c.num_pages;
        c.error[0] = 0;
        c.error[1] = INT_MAX;
    }
}

// What request r asks of reserve: the pages it must hold in all (0: none, or a request that is
// skipped) and the page that it would write but shares (-1: none).
struct Ask {
    int need, shared;
};

__device__ __forceinline__ Ask reserve_ask(const CacheView &c, const int32_t *cu, int r)
{
    Ask a{0, -1};
    const int n = cu[r + 1] - cu[r];
    if (n <= 0)
        return a;
    const int64_t len = c.lens[r];
    const int held = c.held[r];
    if (len < 0 || held < 0 || held > c.max_pages || len > (int64_t)held * c.page_size ||
        len + n > (int64_t)c.max_pages * c.page_size) {
        cache_error(c.error, SPEC_DEVERR_LENGTH, r);
        return a;
    }
    if (len % c.page_size) {
        const int page = c.table[r * c.table_stride + len / c.page_size];
        if (page < 0 || page >= c.num_pages || c.ref[page] < 1) {
            cache_error(c.error, SPEC_DEVERR_PAGE, r);
            return a;
        }
        if (c.ref[page] > 1)
            a.shared = page;
    }
    a.need = pages_of(len + n, c.page_size);
    return a;
}

// Reserve is one block: it lists the requests that write to a shared page, decides which of them copy
// it (request order: each copies while others hold the page; the last of its holders keeps it), finds
// every request's place in the stack of free pages by a prefix sum, and hands the pages out.  It is
// bound by the chain of dependent loads (lengths, table, counts, stack), not by work.
//
// A thread per request, all of it in registers and shared memory; new pages are handed out a thread
// each, which finds its request by bisection.
__global__ void __launch_bounds__(kBookThreads) reserve_kernel(CacheView c, const int32_t *cu, int B)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the copies wait for the whole of this
    __shared__ int32_t held_of[kBookThreads], copies_of[kBookThreads], shared_of[kBookThreads];
    __shared__ int32_t free_of[kBookThreads];  // the top of the stack, read before it is known what is asked for
    __shared__ int64_t base_of[kBookThreads + 1];
    __shared__ int first_short, ncopy;
    const int r = threadIdx.x;
    const int32_t have = *c.num_free;
    int32_t here = 0, next = 0, len = 0, held = 0;
    if (r < B) {
        here = cu[r];
        next = cu[r + 1];
        len = c.lens[r];
        held = c.held[r];
    }
    if (r == 0) {
        first_short = INT_MAX;
        ncopy = 0;
    }
    if (__syncthreads_or(here > next || (r == 0 && here != 0))) {
        if (r == 0) {
            *c.ncopy = 0;
            cache_error(c.error, SPEC_DEVERR_LAYOUT, -1);
        }
        return;
    }
    free_of[r] = have <= c.num_pages && r < have ? c.free_pages[have - 1 - r] : -1;
    int need = 0, shared = -1, refs = 0;
    if (next > here) {
        const int n = next - here;
        if (len < 0 || held < 0 || held > c.max_pages || len > (int64_t)held * c.page_size ||
            (int64_t)len + n > (int64_t)c.max_pages * c.page_size) {
            cache_error(c.error, SPEC_DEVERR_LENGTH, r);
        } else {
            need = pages_of((int64_t)len + n, c.page_size);
            if (len % c.page_size) {
                const int page = c.table[r * c.table_stride + len / c.page_size];
                refs = page >= 0 && page < c.num_pages ? c.ref[page] : 0;
                if (refs < 1) {
                    cache_error(c.error, SPEC_DEVERR_PAGE, r);
                    need = 0;
                } else if (refs > 1) {
                    shared = page;
                }
            }
        }
    }
    bool copies = false;
    shared_of[r] = shared;
    if (__syncthreads_or(shared >= 0) && shared >= 0) {
        int before = 0;
#pragma unroll 8
        for (int j = 0; j < r; ++j)
            before += shared_of[j] == shared;
        copies = refs - before > 1;
    }
    const int fresh = (need > held ? need - held : 0) + copies;
    int64_t used;
    const int64_t at = block_scan<kBookThreads>(fresh, &used);
    held_of[r] = held;
    copies_of[r] = copies;
    base_of[r] = at;
    if (fresh && at + fresh > have)
        atomicMin(&first_short, r);
    __syncthreads();  // also: no count is changed before every thread has read its page's
    if (used > have || have > c.num_pages) {
        if (r == 0) {
            *c.ncopy = 0;
            cache_error(c.error, SPEC_DEVERR_CAPACITY, first_short);
        }
        return;
    }
    for (int64_t k = r; k < used; k += kBookThreads) {
        int lo = 0, hi = B;  // the last request with base <= k; those of no new page lie before it
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (base_of[mid] <= k)
                lo = mid;
            else
                hi = mid;
        }
        const int page = k < kBookThreads ? free_of[k] : c.free_pages[have - 1 - k];
        const int i = (int)(k - base_of[lo]) - copies_of[lo];  // -1: the copy of its last page
        if (page < 0 || page >= c.num_pages)
            cache_error(c.error, SPEC_DEVERR_PAGE, lo);
        else
            c.ref[page] = 1;
        if (i >= 0)
            c.table[lo * c.table_stride + held_of[lo] + i] = page;
    }
    if (copies) {
        const int page = at < kBookThreads ? free_of[at] : c.free_pages[have - 1 - at];
        c.table[r * c.table_stride + len / c.page_size] = page;
        atomicSub(&c.ref[shared], 1);
        if (page >= 0 && page < c.num_pages)
            c.copies[atomicAdd(&ncopy, 1)] = make_int4(shared, page, len % c.page_size, 0);
    }
    if (need > held)
        c.held[r] = need;
    __syncthreads();
    if (r == 0) {
        *c.ncopy = ncopy;
        *c.num_free = have - (int32_t)used;
    }
}

// The same for more requests than the block has threads, in turns, with its lists in the scratch.
__global__ void __launch_bounds__(kBookThreads) reserve_many_kernel(CacheView c, const int32_t *cu, int B)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    if (tid == 0)
        *c.ncopy = 0;
    if (!block_layout_ok(cu, B, INT_MAX)) {
        if (tid == 0)
            cache_error(c.error, SPEC_DEVERR_LAYOUT, -1);
        return;
    }
    int64_t nwriters = 0, total;
    for (int r0 = 0; r0 < B; r0 += kBookThreads) {
        const int r = r0 + tid;
        Ask a{0, -1};
        if (r < B) {
            a = reserve_ask(c, cu, r);
            c.flags[r] = a.need > 0 ? 0 : -1;  // -1: gets nothing, whatever the counts become
        }
        const int64_t at = nwriters + block_scan<kBookThreads>(a.shared >= 0, &total);
        if (a.shared >= 0)
            c.writers[at] = make_int2(r, a.shared);
        nwriters += total;
    }
    __syncthreads();
    // usually a handful: every writer looks at all of them
    for (int64_t i = tid; i < nwriters; i += kBookThreads) {
        const int2 me = c.writers[i];
        int before = 0;
        for (int64_t j = 0; j < i; ++j)
            before += c.writers[j].y == me.y;
        c.flags[me.x] = c.ref[me.y] - before > 1;
    }
    __syncthreads();
    const int32_t have = *c.num_free;
    __shared__ int first_short;
    if (tid == 0)
        first_short = INT_MAX;
    int64_t used = 0;
    for (int r0 = 0; r0 < B; r0 += kBookThreads) {
        const int r = r0 + tid;
        int64_t fresh = 0;
        const int copies = r < B ? c.flags[r] : -1;
        if (copies >= 0) {
            const int need = pages_of((int64_t)c.lens[r] + (cu[r + 1] - cu[r]), c.page_size), held = c.held[r];
            fresh = (need > held ? need - held : 0) + copies;
        }
        const int64_t at = used + block_scan<kBookThreads>(fresh, &total);
        if (r < B) {
            c.base[r] = at;
            if (fresh && at + fresh > have)
                atomicMin(&first_short, r);
        }
        used += total;
    }
    __syncthreads();
    if (used > have || have > c.num_pages) {
        if (tid == 0)
            cache_error(c.error, SPEC_DEVERR_CAPACITY, first_short);
        return;
    }
    // Hand out: a warp per request, as pages per request may be many.  Who gets pages and who copies was
    // settled above: counts change from here on.
    for (int r = w; r < B; r += kBookThreads / 32) {
        if (c.flags[r] < 0)
            continue;
        const int n = cu[r + 1] - cu[r];
        const int64_t len = c.lens[r];
        const int held = c.held[r];
        int32_t *row = c.table + r * c.table_stride;
        const bool copies = c.flags[r] != 0;
        const int need = pages_of(len + n, c.page_size);
        const int64_t top = have - 1 - c.base[r];
        for (int i = held + lane; i < need; i += 32) {
            const int page = c.free_pages[top - copies - (i - held)];
            row[i] = page;
            if (page >= 0 && page < c.num_pages)
                c.ref[page] = 1;
            else
                cache_error(c.error, SPEC_DEVERR_PAGE, r);
        }
        __syncwarp();
        if (lane == 0) {
            if (copies) {
                const int64_t col = len / c.page_size;
                const int old = row[col], page = c.free_pages[top];
                row[col] = page;
                if (page >= 0 && page < c.num_pages) {
                    c.ref[page] = 1;
                    atomicSub(&c.ref[old], 1);
                    c.copies[atomicAdd(c.ncopy, 1)] = make_int4(old, page, (int)(len % c.page_size), 0);
                } else {
                    cache_error(c.error, SPEC_DEVERR_PAGE, r);
                }
            }
            if (need > held)
                c.held[r] = need;
        }
    }
    if (tid == 0)
        *c.num_free = have - (int32_t)used;
}

// The rows of the copy list, in every layer, in parts of a page's keys or values in one layer: four
// 16-byte vectors a thread, all loaded before any is stored.
__global__ void __launch_bounds__(kCopyThreads) copy_rows_kernel(CacheView c)
{
    constexpr int U = 4;
    const int vecs = c.dim / 8;
    const int parts = (c.page_size * c.heads * vecs + U * kCopyThreads - 1) / (U * kCopyThreads);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t units = (int64_t)*c.ncopy * c.num_layers * 2 * parts;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t unit = u / parts;
        const int part = (int)(u - unit * parts);
        const int4 pair = c.copies[unit / (c.num_layers * 2)];
        const int which = (int)(unit % (c.num_layers * 2));
        const int count = pair.z * c.heads * vecs, i0 = part * U * kCopyThreads + threadIdx.x;
        if (i0 >= count)
            continue;
        char *base = (which & 1 ? c.v : c.k) + 2 * ((which >> 1) * c.layer_stride);
        const char *src = base + 2 * (pair.x * c.page_stride);
        char *dst = base + 2 * (pair.y * c.page_stride);
        int64_t offset[U];
        uint4 x[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + j * kCopyThreads, row = i / vecs;
            offset[j] = 2 * (row / c.heads * c.token_stride + row % c.heads * c.head_stride + (i - row * vecs) * 8);
            if (i < count)
                x[j] = *reinterpret_cast<const uint4 *>(src + offset[j]);
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i0 + j * kCopyThreads < count)
                *reinterpret_cast<uint4 *>(dst + offset[j]) = x[j];
    }
}

struct NewRows {
    const char *k, *v;
    int64_t k_token, k_head, v_token, v_head;  // elements
};

// A warp per new token: the loads of its rows are started before its place is looked up.
__global__ void __launch_bounds__(kCopyThreads) append_kernel(CacheView c, NewRows in, int64_t layer_offset,
                                                              const int32_t *cu, int B, int64_t N)
{
    const int lane = threadIdx.x & 31;
    const bool ok = block_layout_ok(cu, B, N);
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            cache_error(c.error, SPEC_DEVERR_LAYOUT, -1);
        return;
    }
    const int64_t t = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    if (t >= cu[B])
        return;
    const int vecs = c.dim / 8, count = c.heads * vecs;
    auto source = [&](int i, uint4 &a, uint4 &b) {
        const int head = i / vecs, e = i % vecs * 8;
        a = ld_stream(in.k + 2 * (t * in.k_token + head * in.k_head + e));
        b = ld_stream(in.v + 2 * (t * in.v_token + head * in.v_head + e));
    };
    constexpr int U = 4;
    uint4 a[U], b[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
        if (lane + 32 * j < count)
            source(lane + 32 * j, a[j], b[j]);
    const int r = warp_find_request(cu, B, t, lane);
    const int64_t len = c.lens[r];
    const int64_t pos = len + (t - cu[r]);
    if (len < 0 || pos >= (int64_t)c.max_pages * c.page_size) {
        if (lane == 0)
            cache_error(c.error, SPEC_DEVERR_LENGTH, r);
        return;
    }
    const int col = (int)(pos / c.page_size);
    const int page = c.table[r * c.table_stride + col];
    if (col >= c.held[r] || page < 0 || page >= c.num_pages || c.ref[page] != 1) {
        if (lane == 0)
            cache_error(c.error, SPEC_DEVERR_PAGE, r);
        return;
    }
    const int64_t at = layer_offset + page * c.page_stride + pos % c.page_size * c.token_stride;
    for (int i0 = lane; i0 < count; i0 += 32 * U) {
        if (i0 != lane) {
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (i0 + 32 * j < count)
                    source(i0 + 32 * j, a[j], b[j]);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + 32 * j;
            if (i < count) {
                const int64_t o = 2 * (at + i / vecs * c.head_stride + i % vecs * 8);
                *reinterpret_cast<uint4 *>(c.k + o) = a[j];
                *reinterpret_cast<uint4 *>(c.v + o) = b[j];
            }
        }
    }
}

// The new length of request r, or -1 with an error recorded.
__device__ __forceinline__ int64_t commit_length(const CacheView &c, const int32_t *cu, const int32_t *accepted,
                                                 int r, bool report)
{
    const int n = cu[r + 1] - cu[r], a = accepted[r], held = c.held[r];
    const int64_t len = c.lens[r];
    if (n == 0 || a == -1)
        return len;
    if (a < -1 || a >= n || !holds(c, held, (int)len, n)) {
        if (report)
            cache_error(c.error, SPEC_DEVERR_LENGTH, r);
        return -1;
    }
    return len + a + 1;
}

__global__ void __launch_bounds__(kCopyThreads) commit_chain_kernel(CacheView c, const int32_t *cu, int B, int64_t N,
                                                                    const int32_t *accepted, int32_t *out_lens)
{
    if (!block_layout_ok(cu, B, N)) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            cache_error(c.error, SPEC_DEVERR_LAYOUT, -1);
        return;
    }
    const int r = blockIdx.x * kCopyThreads + threadIdx.x;
    if (r < B) {
        const int64_t len = commit_length(c, cu, accepted, r, true);
        out_lens[r] = len < 0 ? c.lens[r] : (int32_t)len;
    }
}

// Trees: blocks (request, share of the cache's columns).  A block walks its request's path in
// shared memory, then each thread carries one 16-byte column (of one layer, keys or values, head)
// down the path.  Node indices ascend along a path and each is at least its depth, so a row is
// read before a later level's row is written over it: destination d is the source of a level below
// d at most, and those were read earlier.
__global__ void __launch_bounds__(kCopyThreads) commit_tree_kernel(CacheView c, const int32_t *cu, int B, int64_t N,
                                                                   const int32_t *accepted, const int32_t *parent,
                                                                   const int32_t *last_node, int32_t *out_lens)
{
    __shared__ int32_t par[kMaxTree], path[kMaxTree];
    __shared__ int64_t from[kMaxTree], to[kMaxTree];
    __shared__ int bad, moves;
    const int tid = threadIdx.x, r = blockIdx.x;
    const bool ok = block_layout_ok(cu, B, N);
    if (!ok && r == 0 && blockIdx.y == 0 && tid == 0)
        cache_error(c.error, SPEC_DEVERR_LAYOUT, -1);
    if (ok) {
        const bool report = blockIdx.y == 0 && tid == 0;
        const int first = cu[r], n = cu[r + 1] - first;
        const int64_t len = c.lens[r];
        int64_t after = commit_length(c, cu, accepted, r, report);
        if (tid == 0)
            bad = moves = 0;
        if (after > len) {  // accepted >= 0
            const int depth = accepted[r];
            for (int i = tid; i < n && i < kMaxTree; i += kCopyThreads)
                par[i] = parent[first + i];
            __syncthreads();
            if (tid == 0) {
                int at = last_node[r];
                bad = n > kMaxTree || at < 0 || at >= n ? SPEC_DEVERR_TREE : 0;
                for (int d = depth; d >= 0 && !bad; --d) {
                    path[d] = at;
                    const int up = par[at];
                    if (d == 0 ? at != 0 || up != -1 : up < 0 || up >= at)
                        bad = SPEC_DEVERR_TREE;
                    at = up;
                }
            }
            __syncthreads();
            if (!bad) {
                // the first level that moves: from there on every level does
                for (int d = tid; d <= depth; d += kCopyThreads) {
                    const int64_t src = len + path[d], dst = len + d;
                    const int64_t scol = src / c.page_size, dcol = dst / c.page_size;
                    const int sp = c.table[r * c.table_stride + scol], dp = c.table[r * c.table_stride + dcol];
                    const int held = c.held[r];
                    if (path[d] != d) {
                        if (scol >= held || sp < 0 || sp >= c.num_pages || dcol >= held || dp < 0 ||
                            dp >= c.num_pages || c.ref[dp] != 1)
                            atomicOr(&bad, SPEC_DEVERR_PAGE);
                        atomicAdd(&moves, 1);
                    }
                    from[d] = sp * c.page_stride + src % c.page_size * c.token_stride;
                    to[d] = dp * c.page_stride + dst % c.page_size * c.token_stride;
                }
            }
            __syncthreads();
            if (bad) {
                if (report)
                    cache_error(c.error, bad, r);
                after = -1;
            } else if (moves > 0) {
                const int d0 = depth + 1 - moves;
                const int vecs = c.dim / 8;
                const int64_t columns = (int64_t)c.num_layers * 2 * c.heads * vecs;
                for (int64_t i = (int64_t)blockIdx.y * kCopyThreads + tid; i < columns;
                     i += (int64_t)gridDim.y * kCopyThreads) {
                    const int e = (int)(i % vecs) * 8;
                    int64_t x = i / vecs;
                    const int head = (int)(x % c.heads);
                    x /= c.heads;
                    char *base = (x & 1 ? c.v : c.k) + 2 * ((x >> 1) * c.layer_stride + head * c.head_stride + e);
                    constexpr int U = 8;
                    for (int d = d0; d <= depth; d += U) {
                        uint4 val[U];
#pragma unroll
                        for (int j = 0; j < U; ++j)
                            if (d + j <= depth)
                                val[j] = *reinterpret_cast<const uint4 *>(base + 2 * from[d + j]);
#pragma unroll
                        for (int j = 0; j < U; ++j)
                            if (d + j <= depth)
                                *reinterpret_cast<uint4 *>(base + 2 * to[d + j]) = val[j];
                    }
                }
            }
        }
        if (report)
            c.flags[r] = after < 0 ? (int32_t)len : (int32_t)after;
    }
    // Lengths last, when no block reads the old ones any more.
    if (last_block(c.ticket, gridDim.x * gridDim.y) && ok)
        for (int i = tid; i < B; i += kCopyThreads)
            out_lens[i] = __ldcg(&c.flags[i]);
}

// A block per fork.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(CacheView c, const int32_t *src, const int32_t *dst, int F)
{
    const int f = blockIdx.x, tid = threadIdx.x;
    const int s = src[f], d = dst[f];
    bool bad = s < 0 || s >= c.num_requests || d < 0 || d >= c.num_requests || s == d;
    // (what the checks need is asked for at once: the kernel is a chain of loads)
    int len = 0, held = 0, taken = 0, mine = -1;
    if (!bad) {
        len = c.lens[s];
        held = c.held[s];
        taken = c.held[d];
        if (tid < c.max_pages)
            mine = c.table[s * c.table_stride + tid];
    }
    for (int g = tid; g < F; g += kCopyThreads)
        bad |= (g != f && dst[g] == d) || dst[g] == s || src[g] == d;
    bad |= taken != 0;
    if (__syncthreads_or(bad)) {
        if (tid == 0)
            cache_error(c.error, SPEC_DEVERR_FORK, d >= 0 && d < c.num_requests ? d : -1);
        return;
    }
    const int count = len < 0 ? -1 : pages_of(len, c.page_size);
    if (count < 0 || count > held || count > c.max_pages) {
        if (tid == 0)
            cache_error(c.error, SPEC_DEVERR_LENGTH, d);
        return;
    }
    const int32_t *from = c.table + s * c.table_stride;
    int32_t *to = c.table + d * c.table_stride;
    bool lost = false;
    for (int i = tid; i < count; i += kCopyThreads) {
        const int page = i == tid ? mine : from[i];
        lost |= page < 0 || page >= c.num_pages || c.ref[page] < 1;
    }
    if (__syncthreads_or(lost)) {
        if (tid == 0)
            cache_error(c.error, SPEC_DEVERR_PAGE, d);
        return;
    }
    for (int i = tid; i < count; i += kCopyThreads) {
        const int page = i == tid ? mine : from[i];
        to[i] = page;
        atomicAdd(&c.ref[page], 1);
    }
    if (tid == 0) {
        c.lens[d] = len;
        c.held[d] = count;
    }
}

constexpr int kReleaseThreads = 512;

// Blocks take requests in turn and count their pages down; pages at zero are marked in a bitmap,
// which the last block reads in ascending order: the list does not depend on the order of atomics.
__global__ void __launch_bounds__(kReleaseThreads) release_kernel(CacheView c, const int32_t *keep, int B)
{
    const int tid = threadIdx.x;
    for (int r = blockIdx.x; r < B; r += gridDim.x) {
        const int len = c.lens[r], held = c.held[r];
        const int want = keep ? keep[r] : len;
        if (len < 0 || want < 0 || held < 0 || held > c.max_pages) {
            if (tid == 0)
                cache_error(c.error, SPEC_DEVERR_LENGTH, r);
            continue;
        }
        const int now = want < len ? want : len;
        const int kept = pages_of(now, c.page_size);
        __syncthreads();  // every thread has read the request's length and pages
        for (int i = kept + tid; i < held; i += kReleaseThreads) {
            int32_t *entry = &c.table[r * c.table_stride + i];
            const int page = *entry;
            *entry = -1;
            if (page < 0 || page >= c.num_pages) {
                cache_error(c.error, SPEC_DEVERR_PAGE, r);
                continue;
            }
            const int old = atomicSub(&c.ref[page], 1);
            if (old == 1) {
                atomicOr(&c.freed[page >> 5], 1u << (page & 31));
            } else if (old < 1) {
                atomicAdd(&c.ref[page], 1);
                cache_error(c.error, SPEC_DEVERR_PAGE, r);
            }
        }
        if (tid == 0) {
            c.lens[r] = now;
            if (kept < held)
                c.held[r] = kept;
        }
    }
    if (!last_block(c.ticket, gridDim.x))
        return;
    const int words = (c.num_pages + 31) / 32;
    const int per = (words + kReleaseThreads - 1) / kReleaseThreads;
    const int w0 = tid * per < words ? tid * per : words, w1 = w0 + per < words ? w0 + per : words;
    int64_t mine = 0, total;
    for (int i = w0; i < w1; ++i)
        mine += __popc(__ldcg(&c.freed[i]));
    const int have = *c.num_free;
    int64_t at = have + block_scan<kReleaseThreads>(mine, &total);
    const bool room = have >= 0 && have + total <= c.num_pages;
    if (mine)
        for (int i = w0; i < w1; ++i) {
            uint32_t bits = __ldcg(&c.freed[i]);
            if (!bits)
                continue;
            c.freed[i] = 0;
            for (; bits; bits &= bits - 1)
                if (room)
                    c.free_pages[at++] = i * 32 + __ffs(bits) - 1;
        }
    __syncthreads();
    if (tid == 0) {
        if (room)
            *c.num_free = have + (int32_t)total;
        else
            cache_error(c.error, SPEC_DEVERR_PAGE, -1);
    }
}

}  // namespace
}  // namespace specrej

using namespace specrej;

extern "C" {

size_t spec_cache_scratch_size(int32_t num_requests, int32_t num_pages)
{
    if (num_requests < 1 || num_pages < 1)
        return 0;
    return scratch_plan(num_requests, num_pages).total;
}

spec_status spec_cache_init(const spec_cache *cache, void *stream)
{
    CacheView c;
    spec_status s = view_cache(cache, &c);
    if (s != SPEC_OK)
        return s;
    if (pending())
        return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(cache->scratch, 0, spec_cache_scratch_size(cache->num_requests, cache->num_pages), st) !=
        cudaSuccess)
        return SPEC_ERR_CUDA;
    const int64_t most = std::max<int64_t>(c.num_pages, (int64_t)c.num_requests * c.max_pages);
    return launch(false, init_kernel, dim3((unsigned)std::min<int64_t>((most + kCopyThreads - 1) / kCopyThreads, 1024)),
                  kCopyThreads, st, c);
}

spec_status spec_cache_error(const spec_cache *cache, void *stream, int32_t *error_bits, int32_t *first_bad_request)
{
    if (!cache || !cache->error)
        return SPEC_ERR_INVALID_ARG;
    if (pending())
        return SPEC_ERR_CUDA;
    int32_t word[2] = {0, INT_MAX};
    const int32_t clear[2] = {0, INT_MAX};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(word, cache->error, sizeof word, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return SPEC_ERR_CUDA;
    if (word[0] && (cudaMemcpyAsync(cache->error, clear, sizeof clear, cudaMemcpyHostToDevice, s) != cudaSuccess ||
                    cudaStreamSynchronize(s) != cudaSuccess))
        return SPEC_ERR_CUDA;
    if (error_bits)
        *error_bits = word[0];
    if (first_bad_request)
        *first_bad_request = word[1] == INT_MAX ? -1 : word[1];
    return word[0] & SPEC_DEVERR_TIMEOUT ? SPEC_ERR_TIMEOUT : word[0] ? SPEC_ERR_DEVICE_INPUT : SPEC_OK;
}

spec_status spec_cache_reserve(const spec_cache *cache, const int32_t *cu_new, int32_t B, void *stream)
{
    CacheView c;
    spec_status s = view_cache(cache, &c);
    if (s != SPEC_OK)
        return s;
    if (!cu_new || !ptr_aligned(cu_new, 4) || B < 0 || B > c.num_requests)
        return SPEC_ERR_INVALID_ARG;
    int sms;
    if (pending() || current_sms(&sms) != cudaSuccess)
        return SPEC_ERR_CUDA;
    if (B == 0)
        return SPEC_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    s = launch(false, B <= kBookThreads ? reserve_kernel : reserve_many_kernel, dim3(1), kBookThreads, st, c, cu_new, B);
    if (s != SPEC_OK)
        return s;
    return launch(true, copy_rows_kernel, dim3(sms * 8), kCopyThreads, st, c);
}

spec_status spec_cache_append(const spec_cache *cache, int32_t layer, const void *k_new, int64_t k_token_stride,
                              int64_t k_head_stride, const void *v_new, int64_t v_token_stride,
                              int64_t v_head_stride, const int32_t *cu_new, int32_t B, int64_t N, void *stream)
{
    CacheView c;
    spec_status s = view_cache(cache, &c);
    if (s != SPEC_OK)
        return s;
    if (layer < 0 || layer >= c.num_layers || !cu_new || !ptr_aligned(cu_new, 4) || B < 0 || B > c.num_requests ||
        N < 0 || (N > 0 && (!k_new || !v_new)) || !ptr_aligned(k_new, 16) || !ptr_aligned(v_new, 16))
        return SPEC_ERR_INVALID_ARG;
    if (!good_stride(k_token_stride, N) || !good_stride(v_token_stride, N) ||
        !good_stride(k_head_stride, c.heads) || !good_stride(v_head_stride, c.heads))
        return SPEC_ERR_INVALID_ARG;
    if (N > INT32_MAX)
        return SPEC_ERR_UNSUPPORTED;
    if (pending())
        return SPEC_ERR_CUDA;
    if (B == 0 || N == 0)
        return SPEC_OK;
    const NewRows in{static_cast<const char *>(k_new), static_cast<const char *>(v_new),
                     N > 1 ? k_token_stride : 0, c.heads > 1 ? k_head_stride : 0,
                     N > 1 ? v_token_stride : 0, c.heads > 1 ? v_head_stride : 0};
    const int64_t blocks = (N + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    return launch(false, append_kernel, dim3((unsigned)blocks), kCopyThreads, static_cast<cudaStream_t>(stream), c, in,
                  layer * c.layer_stride, cu_new, B, N);
}

spec_status spec_cache_commit(const spec_cache *cache, const int32_t *cu_new, int32_t B, int64_t N,
                              const int32_t *num_accepted, const int32_t *parent, const int32_t *last_node,
                              int32_t *out_lens, void *stream)
{
    CacheView c;
    spec_status s = view_cache(cache, &c);
    if (s != SPEC_OK)
        return s;
    if (!cu_new || !ptr_aligned(cu_new, 4) || B < 0 || B > c.num_requests || N < 0 || (B > 0 && !num_accepted) ||
        !ptr_aligned(num_accepted, 4) || !ptr_aligned(parent, 4) || !ptr_aligned(last_node, 4) ||
        !ptr_aligned(out_lens, 4) || (parent == nullptr) != (last_node == nullptr))
        return SPEC_ERR_INVALID_ARG;
    if (N > INT32_MAX)
        return SPEC_ERR_UNSUPPORTED;
    int sms;
    if (pending() || current_sms(&sms) != cudaSuccess)
        return SPEC_ERR_CUDA;
    if (B == 0)
        return SPEC_OK;
    int32_t *out = out_lens ? out_lens : c.lens;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!parent) {
        return launch(false, commit_chain_kernel, dim3((B + kCopyThreads - 1) / kCopyThreads), kCopyThreads, st, c, cu_new, B,
                      N, num_accepted, out);
    }
    // Blocks for every column once, as far as the device holds them (8 blocks per SM).
    const int64_t columns = (int64_t)c.num_layers * 2 * c.heads * (c.dim / 8);
    const int64_t split = std::max<int64_t>(
        1, std::min<int64_t>((columns + kCopyThreads - 1) / kCopyThreads, (int64_t)sms * 8 / B));
    return launch(false, commit_tree_kernel, dim3((unsigned)B, (unsigned)split), kCopyThreads, st, c, cu_new, B, N,
                  num_accepted, parent, last_node, out);
}

spec_status spec_cache_fork(const spec_cache *cache, const int32_t *src, const int32_t *dst, int32_t num_forks,
                            void *stream)
{
    CacheView c;
    spec_status s = view_cache(cache, &c);
    if (s != SPEC_OK)
        return s;
    if (num_forks < 0 || (num_forks > 0 && (!src || !dst)) || !ptr_aligned(src, 4) || !ptr_aligned(dst, 4))
        return SPEC_ERR_INVALID_ARG;
    if (pending())
        return SPEC_ERR_CUDA;
    if (num_forks == 0)
        return SPEC_OK;
    return launch(false, fork_kernel, dim3(num_forks), kCopyThreads, static_cast<cudaStream_t>(stream), c, src, dst, num_forks);
}

spec_status spec_cache_release(const spec_cache *cache, const int32_t *keep_lens, int32_t B, void *stream)
{
    CacheView c;
    spec_status s = view_cache(cache, &c);
    if (s != SPEC_OK)
        return s;
    if (B < 0 || B > c.num_requests || !ptr_aligned(keep_lens, 4))
        return SPEC_ERR_INVALID_ARG;
    int sms;
    if (pending() || current_sms(&sms) != cudaSuccess)
        return SPEC_ERR_CUDA;
    if (B == 0)
        return SPEC_OK;
    return launch(false, release_kernel, dim3(std::min(B, sms * 2)), kReleaseThreads, static_cast<cudaStream_t>(stream), c,
                  keep_lens, B);
}

}  // extern "C"
