// share.cu -- which requests of a batch share the pages of a prefix, from the page table (sm_103a).
//
// Two neighbouring requests are linked when their first columns name the same pages, over pages full of committed
// tokens, for at least so many tokens; a group is a run of links, and shares what the shortest of them does.
// A block per request compares its row with the one before, 1024 columns at a time and no further than they agree; the
// last block to end finds the runs, by a scan forward (where each begins, its shortest link) and one backward (where it
// ends).  Bound by its launch and the chain of loads: 4.1 us of 9 requests, 6.8 of 512 whose prefixes are up to 1900
// pages long (4 MB of tables).
#include "cache.cuh"

namespace specrej {
namespace {

constexpr int kShareThreads = 256;

// Inclusive scans over the block of (link, value) pairs: `restart` entries take nothing from those before them.
__device__ __forceinline__ int2 scan_min(int2 x, int lane, int warp, int2 *sums, int2 carry)
{
    // x.x: the first index of the run (-1: before this scan), x.y: the least value in it so far
    auto after = [](int2 before, int2 x) { return x.x >= 0 ? x : make_int2(before.x, min(before.y, x.y)); };
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int2 y = make_int2(__shfl_up_sync(kFull, x.x, d), __shfl_up_sync(kFull, x.y, d));
        if (lane >= d)
            x = after(y, x);
    }
    __syncthreads();
    if (lane == 31)
        sums[warp] = x;
    __syncthreads();
    int2 before = carry;
    for (int i = 0; i < warp; ++i)
        before = after(before, sums[i]);
    return after(before, x);
}

__global__ void __launch_bounds__(kShareThreads) share_kernel(CacheView c, int B, int least, int4 *plan)
{
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ int differs;
    // tokens that the request shares with the one before
    if (tid == 0)
        differs = INT_MAX;
    __syncthreads();
    const int len = c.lens[r];
    int full = 0;
    if (!holds(c, c.held[r], len, 0)) {
        if (tid == 0)
            cache_error(c.error, SPEC_DEVERR_LENGTH, r);
    } else if (r > 0 && holds(c, c.held[r - 1], c.lens[r - 1], 0)) {
        full = min(len, c.lens[r - 1]) / c.page_size;
    }
    const int32_t *row = c.table + r * c.table_stride, *last = row - (r > 0 ? c.table_stride : 0);
    constexpr int U = 4;
    for (int i0 = 0; i0 < full; i0 += U * kShareThreads) {
        int a[U], b[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + j * kShareThreads + tid;
            a[j] = i < full ? row[i] : 0;
            b[j] = i < full ? last[i] : 0;
        }
        int at = INT_MAX;
#pragma unroll
        for (int j = U - 1; j >= 0; --j)
            at = a[j] != b[j] ? i0 + j * kShareThreads + tid : at;
        if (at < INT_MAX)
            atomicMin(&differs, at);
        __syncthreads();
        if (differs < INT_MAX)
            break;
        __syncthreads();
    }
    __syncthreads();
    if (tid == 0) {
        const int tokens = min(full, differs) * c.page_size;
        plan[r].z = tokens >= least ? tokens : 0;
    }
    if (!last_block(c.ticket, gridDim.x))
        return;
    // Forward: a request's group begins at .x, and the least of its links so far is .z.
    __shared__ int2 sums[kShareThreads / 32];
    __shared__ int2 carry;
    int2 before = make_int2(0, INT_MAX);
    for (int r0 = 0; r0 < B; r0 += kShareThreads) {
        const int r = r0 + tid;
        const int link = r < B ? __ldcg(&plan[r].z) : 1;
        const int2 x = scan_min(link > 0 ? make_int2(-1, link) : make_int2(r, INT_MAX), lane, warp, sums, before);
        if (r < B)
            plan[r] = make_int4(x.x, 0, x.y, 0);
        if (tid == kShareThreads - 1)
            carry = x;
        __syncthreads();
        before = carry;
        __syncthreads();
    }
    // Backward: it ends before the next request that begins one; the last of a group knows what all share.
    int next = B;
    for (int r0 = (B - 1) / kShareThreads * kShareThreads; r0 >= 0; r0 -= kShareThreads) {
        const int r = r0 + kShareThreads - 1 - tid;  // descending
        const bool begins = r + 1 < B && plan[r + 1].x == r + 1;
        // the scan's run index counts upwards with the thread: B - (r + 1), the place of the group's end
        const int2 x = scan_min(begins || r >= B ? make_int2(B - min(r + 1, B), 0) : make_int2(-1, 0), lane, warp, sums,
                                make_int2(B - next, 0));
        const int end = B - x.x;
        int4 y{};
        if (r < B) {
            y = plan[r];
            y.y = end;
            y.z = end - y.x > 1 ? plan[end - 1].z : 0;
        }
        if (tid == kShareThreads - 1)
            carry.x = end;
        __syncthreads();
        if (r < B)
            plan[r] = y;
        next = carry.x;
        __syncthreads();
    }
}

}  // namespace
}  // namespace specrej

using namespace specrej;

extern "C" {

spec_status spec_cache_share(const spec_cache *cache, int32_t B, int32_t min_tokens, int32_t *shared, void *stream)
{
    CacheView c;
    spec_status s = view_cache(cache, &c);
    if (s != SPEC_OK)
        return s;
    if (B < 0 || B > c.num_requests || min_tokens < 0 || (B > 0 && !shared) || !ptr_aligned(shared, 16))
        return SPEC_ERR_INVALID_ARG;
    if (pending())
        return SPEC_ERR_CUDA;
    if (B == 0)
        return SPEC_OK;
    return launch(false, share_kernel, dim3((unsigned)B), kShareThreads, static_cast<cudaStream_t>(stream), c, B,
                  min_tokens > 1 ? min_tokens : 1, reinterpret_cast<int4 *>(shared));
}

}  // extern "C"
