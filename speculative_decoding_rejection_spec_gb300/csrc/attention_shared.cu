// attention_shared.cu -- spec_attention_shared(): the kernels of attention.cuh with the pages that several requests
// share read once.
#include "attention.cuh"

using namespace specrej;

extern "C" {

size_t spec_attention_shared_workspace_size(const spec_cache *cache, int32_t num_q_heads, int32_t B, int64_t N)
{
    CacheView c;
    if (check_attention(cache, &c, num_q_heads, B, N) != SPEC_OK)
        return 0;
    return attention_plan(c, num_q_heads, N, true).total;
}

spec_status spec_attention_shared(const spec_cache *cache, int32_t layer, const void *q, int64_t q_token_stride,
                                  int64_t q_head_stride, int32_t num_q_heads, const int32_t *cu_new, int32_t B,
                                  int64_t N, const int32_t *parent, float scale, const int32_t *shared, void *out,
                                  int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    const AttentionCall a{layer, q, q_token_stride, q_head_stride, num_q_heads, cu_new, B, N, parent, scale, out,
                          out_token_stride, out_head_stride, lse, workspace, workspace_bytes, stream, 0, 0, shared};
    return attend<kShared>(cache, a);
}

}  // extern "C"
