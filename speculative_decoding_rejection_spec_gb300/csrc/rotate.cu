// rotate.cu -- the new tokens' keys and values into the pages, keys and queries turned by their positions
// (sm_103a).
//
// Elements a, b of a head that form a pair become a c - b s and b c + a s, with c and s of the row's position
// from the caller's table: fp32 throughout, rounded to 16 bits once.
//
// What bounds it (GB300): prompt chunks, memory (548 MB: 89.7 us in the kernel, 6.1 TB/s; 107 us before the first
// rows were asked for ahead of the lookup, and with batches of loads four heads long).  A decoding step's rows, the
// chain of loads (rows in all, layout, request, length, page, table: 4.3 us for 160 tokens, of which the launch takes
// 2).  Without the first of these, the number of rows that are not padding, 4.1 us, and prompt chunks from Python 90.7
// us against 92.6; but rows of padding were read then.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"

namespace specrej {
namespace {

struct Rotated {
    const char *k, *v, *q;
    char *q_out;
    int64_t k_token, k_head, v_token, v_head, q_token, q_head, out_token, out_head;  // elements
    int32_t q_heads;
    const int32_t *parent;
    const float *table;
    int64_t table_stride;
    int32_t positions, half;  // half of the elements that turn
    int32_t units;            // of a head: vectors of 8 elements, or two of them that form 8 pairs
    int32_t parts;            // warps per token
};

template <int DT> __device__ __forceinline__ void unpack16(uint4 x, float *y)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = DT == SPEC_BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]))
                                         : __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
    }
}

template <int DT> __device__ __forceinline__ uint4 pack16(const float *y)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == SPEC_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The depth of node i of a tree of n <= kMaxTree nodes; a whole warp, every lane knows it.  -1: a malformed tree.
__device__ __forceinline__ int warp_depth(const int32_t *parent, int n, int i, int lane)
{
    int up[kMaxTree / 32];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kMaxTree / 32; ++j) {
        const int node = j * 32 + lane;
        up[j] = node < n ? parent[node] : -1;
        bad |= node < n && (node == 0 ? up[j] != -1 : up[j] < 0 || up[j] >= node);
    }
    if (__any_sync(kFull, bad))
        return -1;
    int depth = 0;
    for (; i > 0; ++depth) {
        int next = 0;
#pragma unroll
        for (int j = 0; j < kMaxTree / 32; ++j) {
            const int x = __shfl_sync(kFull, up[j], i & 31);
            next = i >> 5 == j ? x : next;
        }
        i = next;
    }
    return depth;
}

// 16 bytes that are read once; they may be written by this kernel (queries turned in place, by the thread that read
// them).
__device__ __forceinline__ uint4 ld_once(const void *p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// A warp per new token, or several: a lane keeps its unit of every head, and so its sines and cosines.  The first keys,
// values and queries are asked for before the token's place is looked up.
template <int DT, bool NEIGHBOURS>
__global__ void __launch_bounds__(kCopyThreads, 3) rotate_kernel(CacheView c, Rotated in, int64_t layer_offset,
                                                                 const int32_t *cu, int B, int64_t N)
{
    const int lane = threadIdx.x & 31;
    const int64_t job = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = job / in.parts;
    const int part = (int)(job - t * in.parts);
    // units of a head: first those that turn (8 pairs, of two vectors half apart; neighbours: 4 pairs of one), then
    // the rest, vector by vector
    const int per = 32 / in.units, u = lane % in.units, mine = lane / in.units;
    const int turning = NEIGHBOURS ? in.half / 4 : in.half / 8;
    const bool turns = u < turning;
    const int e0 = (turns || NEIGHBOURS ? u : u + turning) * 8, e1 = e0 + in.half;  // e1: the other vector of a pair
    constexpr int U = 2;  // heads at a time (four: prompts 104 us against 87, for want of registers)
    const int step = per * in.parts, h0 = part * per + mine;
    auto load = [&](const char *src, int64_t src_head, int heads, int from, uint4 *x, uint4 *y) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int h = from + j * step;
            if (mine < per && h < heads) {
                x[j] = ld_once(src + 2 * (h * src_head + e0));
                if (!NEIGHBOURS && turns)
                    y[j] = ld_once(src + 2 * (h * src_head + e1));
            }
        }
    };
    const int vecs = c.dim / 8, v0 = part * 32 + lane, v_step = 32 * in.parts;
    auto load_v = [&](int from, uint4 *x) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = from + j * v_step, head = i / vecs;
            if (i < c.heads * vecs)
                x[j] = ld_stream(in.v + 2 * (t * in.v_token + head * in.v_head + (i - head * vecs) * 8));
        }
    };
    const char *k_row = in.k + 2 * t * in.k_token, *q_row = in.q + 2 * t * in.q_token;
    uint4 vx[U], kx[U], ky[U];
    const int rows = cu[B];
    if (t < rows && t < N) {  // (rows of padding are not read: another stream may be writing them)
        load(k_row, in.k_head, c.heads, h0, kx, ky);
        load_v(v0, vx);
    }
    if (!block_layout_ok(cu, B, N)) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            cache_error(c.error, SPEC_DEVERR_LAYOUT, -1);
        return;
    }
    if (t >= rows)
        return;
    const int r = warp_find_request(cu, B, t, lane);
    const int first = cu[r], n = cu[r + 1] - first, i = (int)(t - first);
    const int held = load_now(&c.held[r]);
    const int64_t len = c.lens[r], pos = len + i;
    // the step's positions lie in the table, a tree's among them
    if (len < 0 || len + n > in.positions || pos >= (int64_t)c.max_pages * c.page_size) {
        if (lane == 0)
            cache_error(c.error, SPEC_DEVERR_LENGTH, r);
        return;
    }
    const int col = (int)(pos / c.page_size);
    const int page = col < held ? c.table[r * c.table_stride + col] : -1;
    int depth = i;
    if (in.parent) {
        depth = n <= kMaxTree ? warp_depth(in.parent + first, n, i, lane) : -1;
        if (depth < 0) {
            if (lane == 0)
                cache_error(c.error, SPEC_DEVERR_TREE, r);
            return;
        }
    }
    constexpr int P = NEIGHBOURS ? 4 : 8;
    float cs[P], sn[P];
    if (turns) {
        const float *row = in.table + (len + depth) * in.table_stride + u * P;
#pragma unroll
        for (int j = 0; j < P; j += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(row + j);
            const float4 y = *reinterpret_cast<const float4 *>(row + in.half + j);
            cs[j] = x.x, cs[j + 1] = x.y, cs[j + 2] = x.z, cs[j + 3] = x.w;
            sn[j] = y.x, sn[j + 1] = y.y, sn[j + 2] = y.z, sn[j + 3] = y.w;
        }
    }
    if (page < 0 || page >= c.num_pages || c.ref[page] != 1) {
        if (lane == 0)
            cache_error(c.error, SPEC_DEVERR_PAGE, r);
        return;
    }
    const int64_t at = layer_offset + page * c.page_stride + pos % c.page_size * c.token_stride;
    for (int from = v0; from < c.heads * vecs; from += U * v_step) {
        if (from != v0)
            load_v(from, vx);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = from + j * v_step, head = i / vecs;
            if (i < c.heads * vecs)
                *reinterpret_cast<uint4 *>(c.v + 2 * (at + head * c.head_stride + (i - head * vecs) * 8)) = vx[j];
        }
    }
    if (mine >= per)
        return;
    auto turn = [&](char *dst, int64_t dst_head, int heads, int from, const uint4 *x, const uint4 *y) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int h = from + j * step;
            if (h >= heads)
                break;
            uint4 z = x[j];
            if (turns) {
                float a[8], b[8], d[8];
                unpack16<DT>(x[j], a);
                if (NEIGHBOURS) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d[2 * i] = fmaf(a[2 * i], cs[i % P], -a[2 * i + 1] * sn[i % P]);
                        d[2 * i + 1] = fmaf(a[2 * i + 1], cs[i % P], a[2 * i] * sn[i % P]);
                    }
                } else {
                    unpack16<DT>(y[j], b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        d[i] = fmaf(a[i], cs[i % P], -b[i] * sn[i % P]);
                        b[i] = fmaf(b[i], cs[i % P], a[i] * sn[i % P]);
                    }
                    *reinterpret_cast<uint4 *>(dst + 2 * (h * dst_head + e1)) = pack16<DT>(b);
                }
                z = pack16<DT>(d);
            }
            *reinterpret_cast<uint4 *>(dst + 2 * (h * dst_head + e0)) = z;
        }
    };
    for (int from = h0; from < c.heads; from += U * step) {
        if (from != h0)
            load(k_row, in.k_head, c.heads, from, kx, ky);
        turn(c.k + 2 * at, c.head_stride, c.heads, from, kx, ky);
    }
    char *out_row = in.q_out + 2 * t * in.out_token;
    for (int from = h0; from < in.q_heads; from += U * step) {
        load(q_row, in.q_head, in.q_heads, from, kx, ky);
        turn(out_row, in.out_head, in.q_heads, from, kx, ky);
    }
}

}  // namespace
}  // namespace specrej

using namespace specrej;

extern "C" {

spec_status spec_cache_append_rotated(const spec_cache *cache, int32_t layer, const void *k_new,
                                      int64_t k_token_stride, int64_t k_head_stride, const void *v_new,
                                      int64_t v_token_stride, int64_t v_head_stride, const void *q,
                                      int64_t q_token_stride, int64_t q_head_stride, int32_t num_q_heads, void *q_out,
                                      int64_t out_token_stride, int64_t out_head_stride, const int32_t *cu_new,
                                      int32_t B, int64_t N, const int32_t *parent, const spec_rotation *rotation,
                                      void *stream)
{
    CacheView c;
    spec_status s = view_cache(cache, &c);
    if (s != SPEC_OK)
        return s;
    if (layer < 0 || layer >= c.num_layers || !cu_new || !ptr_aligned(cu_new, 4) || B < 0 || B > c.num_requests ||
        N < 0 || num_q_heads < 0 || (N > 0 && (!k_new || !v_new || (num_q_heads > 0 && (!q || !q_out)))) ||
        !ptr_aligned(k_new, 16) || !ptr_aligned(v_new, 16) || !ptr_aligned(q, 16) || !ptr_aligned(q_out, 16) ||
        !ptr_aligned(parent, 4))
        return SPEC_ERR_INVALID_ARG;
    if (!good_stride(k_token_stride, N) || !good_stride(v_token_stride, N) || !good_stride(k_head_stride, c.heads) ||
        !good_stride(v_head_stride, c.heads) ||
        (num_q_heads > 0 && (!good_stride(q_token_stride, N) || !good_stride(out_token_stride, N) ||
                             !good_stride(q_head_stride, num_q_heads) || !good_stride(out_head_stride, num_q_heads))))
        return SPEC_ERR_INVALID_ARG;
    if (!rotation || !rotation->table || !ptr_aligned(rotation->table, 16) || rotation->positions < 1 ||
        rotation->dim < 2 || rotation->dim % 2 || rotation->dim > c.dim ||
        (rotation->positions > 1 && (rotation->row_stride < rotation->dim || rotation->row_stride % 4)))
        return SPEC_ERR_INVALID_ARG;
    if (N > INT32_MAX || c.dim > SPEC_ROTATION_MAX_HEAD_DIM || rotation->dim % (rotation->neighbours ? 8 : 16))
        return SPEC_ERR_UNSUPPORTED;
    int sms;
    if (pending() || current_sms(&sms) != cudaSuccess)
        return SPEC_ERR_CUDA;
    if (B == 0 || N == 0)
        return SPEC_OK;
    Rotated in{};
    in.k = static_cast<const char *>(k_new);
    in.v = static_cast<const char *>(v_new);
    in.q = static_cast<const char *>(q);
    in.q_out = static_cast<char *>(q_out);
    in.k_token = N > 1 ? k_token_stride : 0;
    in.v_token = N > 1 ? v_token_stride : 0;
    in.q_token = N > 1 ? q_token_stride : 0;
    in.out_token = N > 1 ? out_token_stride : 0;
    in.k_head = c.heads > 1 ? k_head_stride : 0;
    in.v_head = c.heads > 1 ? v_head_stride : 0;
    in.q_head = num_q_heads > 1 ? q_head_stride : 0;
    in.out_head = num_q_heads > 1 ? out_head_stride : 0;
    in.q_heads = num_q_heads;
    in.parent = parent;
    in.table = rotation->table;
    in.table_stride = rotation->positions > 1 ? rotation->row_stride : 0;
    in.positions = rotation->positions;
    in.half = rotation->dim / 2;
    in.units = c.dim / 8 - (rotation->neighbours ? 0 : in.half / 8);
    // a warp per token when they fill the device, else up to 8 that share out its heads (32/8 heads of 128, us with 1 / 2
    // / 4 / 8: 160 tokens 6.9 / 5.2 / 4.6 / 4.4; 900 tokens 7.5 / 6.3 / 5.9 / 8.5; 1800 tokens 9.1 / 7.7 / 10.0 / 15.1;
    // 2752 tokens 11.9 / 13.0 / 15.7 / 23.4.  Towards the upper end of each range the rule is late: 600 tokens 7.8 with
    // its 8 and 5.3 with 4, 1200 tokens 8.7 with its 4 and 6.5 with 2.)
    in.parts = 1;
    while (in.parts < 8 && N * in.parts < sms * 16)
        in.parts *= 2;
    const int64_t blocks = (N * in.parts + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    auto kernel = cache->dtype == SPEC_BF16
                      ? (rotation->neighbours ? rotate_kernel<SPEC_BF16, true> : rotate_kernel<SPEC_BF16, false>)
                      : (rotation->neighbours ? rotate_kernel<SPEC_F16, true> : rotate_kernel<SPEC_F16, false>);
    return launch(false, kernel, dim3((unsigned)blocks), kCopyThreads, static_cast<cudaStream_t>(stream), c, in,
                  layer * c.layer_stride, cu_new, B, N);
}

}  // extern "C"
