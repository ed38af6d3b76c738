// attention.cu -- attention of a step's new tokens over the paged cache (sm_103a).
//
// A warp per (new token, query head) walks the visible positions with a running maximum and sum.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"

namespace specrej {
namespace {

struct AttentionParams {
    const char *q;
    char *out;
    float *lse;
    int64_t q_token, q_head, out_token, out_head;  // elements
    int32_t heads, group, B;
    int64_t N;
    const int32_t *cu, *parent;
    float scale;
    int64_t layer_offset;
};

template <int DT> __device__ __forceinline__ float2 to_float2(uint32_t x)
{
    if (DT == SPEC_BF16)
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

template <int DT> __device__ __forceinline__ uint32_t from_float2(float a, float b)
{
    if (DT == SPEC_BF16) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
    const __half2 y = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&y);
}

template <int DT> __global__ void __launch_bounds__(256) attention_kernel(CacheView c, AttentionParams p)
{
    const int lane = threadIdx.x & 31;
    bool bad = false;
    for (int r = threadIdx.x; r <= p.B; r += blockDim.x) {
        const int32_t x = p.cu[r];
        bad |= (r == 0 ? x != 0 : p.cu[r - 1] > x) || x > p.N;
    }
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            cache_error(c.error, SPEC_DEVERR_LAYOUT, -1);
        return;
    }
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    const int64_t t = w / p.heads;
    const int h = (int)(w % p.heads);
    if (t >= p.cu[p.B])
        return;
    const int r = warp_find_request(p.cu, p.B, t, lane);
    const int first = p.cu[r], n = p.cu[r + 1] - first, i = (int)(t - first);
    const int len = c.lens[r];
    if (len < 0 || (int64_t)len + n > (int64_t)c.max_pages * c.page_size || (p.parent && n > kMaxTree)) {
        if (lane == 0)
            cache_error(c.error, p.parent && n > kMaxTree ? SPEC_DEVERR_TREE : SPEC_DEVERR_LENGTH, r);
        return;
    }
    uint32_t seen[kMaxTree / 32] = {};
    if (p.parent)
        for (int at = i; at >= 0;) {
#pragma unroll
            for (int j = 0; j < kMaxTree / 32; ++j)
                seen[j] |= at / 32 == j ? 1u << at % 32 : 0;
            const int up = p.parent[first + at];
            if (at == 0 ? up != -1 : up < 0 || up >= at) {
                if (lane == 0)
                    cache_error(c.error, SPEC_DEVERR_TREE, r);
                break;
            }
            at = up;
        }
    const int e = lane * 4;
    const bool on = e < c.dim;
    float q[4] = {}, acc[4] = {}, m = -INFINITY, l = 0;
    if (on) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p.q + 2 * (t * p.q_token + h * p.q_head + e));
        const float2 a = to_float2<DT>(x.x), b = to_float2<DT>(x.y);
        q[0] = a.x, q[1] = a.y, q[2] = b.x, q[3] = b.y;
    }
    const int64_t base = p.layer_offset + h / p.group * c.head_stride + e;
    for (int pos = 0; pos <= len + i; ++pos) {
        if (p.parent && pos >= len) {
            const int j = pos - len;
            uint32_t word = 0;
#pragma unroll
            for (int x = 0; x < kMaxTree / 32; ++x)
                word = j / 32 == x ? seen[x] : word;
            if (!(word >> (j % 32) & 1))
                continue;
        }
        const int page = c.table[r * c.table_stride + pos / c.page_size];
        const bool there = page >= 0 && page < c.num_pages;
        if (!there && lane == 0)
            cache_error(c.error, SPEC_DEVERR_PAGE, r);
        const int64_t at = 2 * (base + page * c.page_stride + pos % c.page_size * c.token_stride);
        float kx[4] = {}, vx[4] = {};
        if (on && there) {
            const uint2 x = *reinterpret_cast<const uint2 *>(c.k + at), y = *reinterpret_cast<const uint2 *>(c.v + at);
            const float2 a = to_float2<DT>(x.x), b = to_float2<DT>(x.y), d = to_float2<DT>(y.x), f = to_float2<DT>(y.y);
            kx[0] = a.x, kx[1] = a.y, kx[2] = b.x, kx[3] = b.y;
            vx[0] = d.x, vx[1] = d.y, vx[2] = f.x, vx[3] = f.y;
        }
        const float s = warp_sum(q[0] * kx[0] + q[1] * kx[1] + q[2] * kx[2] + q[3] * kx[3]) * p.scale;
        const float mx = fmaxf(m, s), f = expf(m - mx), g = expf(s - mx);
        l = l * f + g;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = acc[j] * f + g * vx[j];
        m = mx;
    }
    if (on) {
        const uint2 x = make_uint2(from_float2<DT>(acc[0] / l, acc[1] / l), from_float2<DT>(acc[2] / l, acc[3] / l));
        *reinterpret_cast<uint2 *>(p.out + 2 * (t * p.out_token + h * p.out_head + e)) = x;
    }
    if (lane == 0 && p.lse)
        p.lse[t * p.heads + h] = m + logf(l);
}

spec_status check_attention(const spec_cache *cache, CacheView *c, int32_t num_q_heads, int32_t B, int64_t N)
{
    spec_status s = view_cache(cache, c);
    if (s != SPEC_OK)
        return s;
    if (B < 0 || B > c->num_requests || N < 0 || num_q_heads < 1 || num_q_heads % c->heads)
        return SPEC_ERR_INVALID_ARG;
    if (c->dim > SPEC_ATTENTION_MAX_HEAD_DIM || c->page_size % 8 || num_q_heads / c->heads > 128 ||
        N * num_q_heads > INT32_MAX)
        return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

}  // namespace
}  // namespace specrej

using namespace specrej;

extern "C" {

size_t spec_attention_workspace_size(const spec_cache *cache, int32_t num_q_heads, int32_t B, int64_t N)
{
    CacheView c;
    if (check_attention(cache, &c, num_q_heads, B, N) != SPEC_OK)
        return 0;
    return 256;
}

spec_status spec_attention(const spec_cache *cache, int32_t layer, const void *q, int64_t q_token_stride,
                           int64_t q_head_stride, int32_t num_q_heads, const int32_t *cu_new, int32_t B, int64_t N,
                           const int32_t *parent, float scale, void *out, int64_t out_token_stride,
                           int64_t out_head_stride, float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    CacheView c;
    spec_status s = check_attention(cache, &c, num_q_heads, B, N);
    if (s != SPEC_OK)
        return s;
    if (layer < 0 || layer >= c.num_layers || !cu_new || !ptr_aligned(cu_new, 4) || !ptr_aligned(parent, 4) ||
        (N > 0 && (!q || !out)) || !ptr_aligned(q, 16) || !ptr_aligned(out, 16) || !ptr_aligned(lse, 4) ||
        !workspace || !(scale > 0) || !(scale < INFINITY))
        return SPEC_ERR_INVALID_ARG;
    if (!good_stride(q_token_stride, N) || !good_stride(out_token_stride, N) ||
        !good_stride(q_head_stride, num_q_heads) || !good_stride(out_head_stride, num_q_heads))
        return SPEC_ERR_INVALID_ARG;
    if (workspace_bytes < spec_attention_workspace_size(cache, num_q_heads, B, N))
        return SPEC_ERR_WORKSPACE;
    if (cudaPeekAtLastError() != cudaSuccess)
        return SPEC_ERR_CUDA;
    if (B == 0 || N == 0)
        return SPEC_OK;
    AttentionParams p{};
    p.q = static_cast<const char *>(q);
    p.out = static_cast<char *>(out);
    p.lse = lse;
    p.q_token = N > 1 ? q_token_stride : 0;
    p.out_token = N > 1 ? out_token_stride : 0;
    p.q_head = num_q_heads > 1 ? q_head_stride : 0;
    p.out_head = num_q_heads > 1 ? out_head_stride : 0;
    p.heads = num_q_heads;
    p.group = num_q_heads / c.heads;
    p.B = B;
    p.N = N;
    p.cu = cu_new;
    p.parent = parent;
    p.scale = scale;
    p.layer_offset = layer * c.layer_stride;
    const unsigned blocks = (unsigned)((N * num_q_heads + 7) / 8);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->dtype == SPEC_BF16)
        attention_kernel<SPEC_BF16><<<blocks, 256, 0, st>>>(c, p);
    else
        attention_kernel<SPEC_F16><<<blocks, 256, 0, st>>>(c, p);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
