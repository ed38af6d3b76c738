// cache.cuh -- what the paged cache's translation units share: the device's view of a
// spec_cache, the host checks, error reporting and the lookup of a row's request.
#pragma once

#include "common.cuh"
#include "spec_cache.h"

namespace specrej {

constexpr int kMaxTree = SPEC_CACHE_MAX_TREE;

struct CacheView {
    char *k, *v;  // 16-bit elements
    int32_t num_layers, num_pages, page_size, heads, dim;
    int64_t layer_stride, page_stride, token_stride, head_stride;  // elements
    int32_t *table;
    int64_t table_stride;
    int32_t num_requests, max_pages;
    int32_t *lens, *held, *ref, *free_pages, *num_free, *error;
    // scratch
    uint32_t *freed;    // [ceil(num_pages / 32)] pages whose count fell to zero; zero between calls
    int32_t *ticket;    // [4] blocks done (commit, release); zero between calls
    int32_t *ncopy;     // [1] entries of the copy list
    int4 *copies;       // [num_requests] (old page, new page, rows, -)
    int2 *writers;      // [num_requests] (request, shared page it writes)
    int64_t *base;      // [num_requests] first place in the stack of a request's new pages
    int32_t *flags;     // [num_requests] reserve: copies its last page; commit: moves nothing, or is bad
};

struct ScratchPlan {
    size_t freed, ticket, ncopy, copies, writers, base, flags, total;
};

inline ScratchPlan scratch_plan(int32_t requests, int32_t pages)
{
    ScratchPlan p{};
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align256(o + bytes);
        return at;
    };
    p.ticket = take(4 * sizeof(int32_t));
    p.freed = take(((size_t)pages + 31) / 32 * sizeof(uint32_t));
    p.ncopy = take(sizeof(int32_t));
    p.copies = take(sizeof(int4) * (size_t)requests);
    p.writers = take(sizeof(int2) * (size_t)requests);
    p.base = take(sizeof(int64_t) * (size_t)requests);
    p.flags = take(sizeof(int32_t) * (size_t)requests);
    p.total = o;
    return p;
}

inline bool ptr_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool good_stride(int64_t stride, int64_t size) { return size <= 1 || (stride > 0 && stride % 8 == 0); }

// The host's checks of a cache; fills the device's view.
inline spec_status view_cache(const spec_cache *c, CacheView *out)
{
    if (!c || !c->k || !c->v || (c->dtype != SPEC_BF16 && c->dtype != SPEC_F16) || c->num_layers < 1 ||
        c->num_pages < 1 || c->page_size < 1 || c->num_kv_heads < 1 || c->head_dim < 8 || c->head_dim % 8 ||
        c->head_dim > 1024 || c->num_requests < 1 || c->max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    if (!good_stride(c->layer_stride, c->num_layers) || !good_stride(c->page_stride, c->num_pages) ||
        !good_stride(c->token_stride, c->page_size) || !good_stride(c->head_stride, c->num_kv_heads) ||
        (c->num_requests > 1 && c->table_stride < c->max_pages))
        return SPEC_ERR_INVALID_ARG;
    if (!c->page_table || !c->lens || !c->held || !c->ref_counts || !c->free_pages || !c->num_free || !c->error ||
        !c->scratch)
        return SPEC_ERR_INVALID_ARG;
    if (!ptr_aligned(c->k, 16) || !ptr_aligned(c->v, 16) || !ptr_aligned(c->scratch, 16) ||
        !ptr_aligned(c->page_table, 4) || !ptr_aligned(c->lens, 4) || !ptr_aligned(c->held, 4) ||
        !ptr_aligned(c->ref_counts, 4) || !ptr_aligned(c->free_pages, 4) || !ptr_aligned(c->num_free, 4) ||
        !ptr_aligned(c->error, 4))
        return SPEC_ERR_INVALID_ARG;
    // positions are 32-bit, and so is the number of a 16-byte vector in a page of one layer
    if ((int64_t)c->max_pages * c->page_size > INT32_MAX / 2 ||
        (int64_t)c->num_kv_heads * (c->head_dim / 8) > INT32_MAX / 2 / c->page_size)
        return SPEC_ERR_UNSUPPORTED;
    CacheView v{};
    v.k = static_cast<char *>(c->k);
    v.v = static_cast<char *>(c->v);
    v.num_layers = c->num_layers;
    v.num_pages = c->num_pages;
    v.page_size = c->page_size;
    v.heads = c->num_kv_heads;
    v.dim = c->head_dim;
    v.layer_stride = c->num_layers > 1 ? c->layer_stride : 0;
    v.page_stride = c->num_pages > 1 ? c->page_stride : 0;
    v.token_stride = c->page_size > 1 ? c->token_stride : 0;
    v.head_stride = c->num_kv_heads > 1 ? c->head_stride : 0;
    v.table = c->page_table;
    v.table_stride = c->num_requests > 1 ? c->table_stride : 0;
    v.num_requests = c->num_requests;
    v.max_pages = c->max_pages;
    v.lens = c->lens;
    v.held = c->held;
    v.ref = c->ref_counts;
    v.free_pages = c->free_pages;
    v.num_free = c->num_free;
    v.error = c->error;
    const ScratchPlan p = scratch_plan(c->num_requests, c->num_pages);
    char *s = static_cast<char *>(c->scratch);
    v.freed = reinterpret_cast<uint32_t *>(s + p.freed);
    v.ticket = reinterpret_cast<int32_t *>(s + p.ticket);
    v.ncopy = reinterpret_cast<int32_t *>(s + p.ncopy);
    v.copies = reinterpret_cast<int4 *>(s + p.copies);
    v.writers = reinterpret_cast<int2 *>(s + p.writers);
    v.base = reinterpret_cast<int64_t *>(s + p.base);
    v.flags = reinterpret_cast<int32_t *>(s + p.flags);
    *out = v;
    return SPEC_OK;
}

namespace {

constexpr int kCopyThreads = 256;

// Records an error in the cache's word.
__device__ __forceinline__ void cache_error(int32_t *error, int32_t bits, int32_t request)
{
    atomicOr(&error[0], bits);
    if (request >= 0)
        atomicMin(&error[1], request);
}

// A word that is asked for here, not behind the branches between here and its use, where it would be a load more in a
// chain.
__device__ __forceinline__ int32_t load_now(const int32_t *p) { return *const_cast<const volatile int32_t *>(p); }

__device__ __forceinline__ int pages_of(int64_t tokens, int page_size)
{
    return (int)((tokens + page_size - 1) / page_size);
}

// Whether the pages that a request holds contain its len committed tokens and n new ones.
__device__ __forceinline__ bool holds(const CacheView &c, int held, int len, int n)
{
    return len >= 0 && held >= 0 && held <= c.max_pages && (int64_t)len + n <= (int64_t)held * c.page_size;
}

// The request of row t by a 32-way search of the warp over cu[0 .. B]: the largest r with cu[r] <=
// t, and with it cu[r + 1] > t when cu does not decrease (requests of no rows are passed over).
// -1 when t lies outside [cu[0], cu[B]).
__device__ __forceinline__ int warp_find_request(const int32_t *cu, int B, int64_t t, int lane)
{
    if (t >= cu[B] || t < cu[0])
        return -1;
    int lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t at = (int64_t)lo + (int64_t)(lane + 1) * step;
        const bool below = at < hi && cu[at] <= t;
        const int k = __popc(__ballot_sync(kFull, below));
        const int64_t next_hi = (int64_t)lo + (int64_t)(k + 1) * step;
        lo += k * step;
        hi = next_hi < hi ? (int)next_hi : hi;
    }
    return lo;
}

// Whether cu[0 .. B] starts at 0, does not decrease and ends within N rows; the whole block.
__device__ __forceinline__ bool block_layout_ok(const int32_t *cu, int B, int64_t N)
{
    bool bad = false;
    for (int r = threadIdx.x; r <= B; r += blockDim.x) {
        const int32_t c = cu[r];
        bad |= r == 0 ? c != 0 : cu[r - 1] > c;
        bad |= c > N;
    }
    return !__syncthreads_or(bad);
}

// Whether this block is the last of `blocks` to come here; what the others wrote is then visible.
__device__ __forceinline__ bool last_block(int32_t *ticket, int blocks)
{
    __shared__ bool last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        last = atomicAdd(ticket, 1) == blocks - 1;
        if (last)
            *ticket = 0;
    }
    __syncthreads();
    __threadfence();
    return last;
}

constexpr int kMaxDevices = 64;

// SMs of the current device.
inline cudaError_t current_sms(int *sms)
{
    static int cached[kMaxDevices];  // written with the same value by every thread that finds it 0
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    int n = __atomic_load_n(&cached[dev], __ATOMIC_RELAXED);
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e)
            return e;
        __atomic_store_n(&cached[dev], n, __ATOMIC_RELAXED);
    }
    *sms = n;
    return cudaSuccess;
}

// `follows`: as a programmatic dependent of the call's kernel before it, which it waits for itself.  The
// first kernel of a call is launched plainly: what other calls launched before it, some as dependents of
// one another, has all ended then.
template <class... Params, class... Args>
spec_status launch(bool follows, void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

inline bool pending() { return cudaPeekAtLastError() != cudaSuccess; }

}  // namespace
}  // namespace specrej
