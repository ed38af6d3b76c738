// attention_window.cu -- spec_attention_window(): the kernels of attention.cuh over the last positions and the first.
#include "attention.cuh"

using namespace specrej;

extern "C" {

spec_status spec_attention_window(const spec_cache *cache, int32_t layer, const void *q, int64_t q_token_stride,
                                  int64_t q_head_stride, int32_t num_q_heads, const int32_t *cu_new, int32_t B,
                                  int64_t N, const int32_t *parent, float scale, int32_t window, int32_t sinks,
                                  void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse,
                                  void *workspace, size_t workspace_bytes, void *stream)
{
    const AttentionCall a{layer, q, q_token_stride, q_head_stride, num_q_heads, cu_new, B, N, parent, scale, out,
                          out_token_stride, out_head_stride, lse, workspace, workspace_bytes, stream, window, sinks,
                          nullptr};
    return attend<kWindow>(cache, a);
}

}  // extern "C"
