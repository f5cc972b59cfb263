// rope_q8_attn_bf16.hip -- attention over a paged cache in 8 bits for bfloat16 queries, and the
// entry points for both types.
#include <string>

#include "rope_q8_rows.h"

namespace ropeamd {

int run_attention_q8_f16(AttnQ8Plan &p, void *stream);  // rope_q8_attn_f16.hip

}  // namespace ropeamd

using namespace ropeamd;

ROPE_API int64_t rope_attention_paged_q8_workspace(int64_t num_tokens, int64_t num_heads,
                                                   int64_t num_key_heads, int64_t head_size,
                                                   int64_t num_sequences) {
  return attention_q8_workspace(num_tokens, num_heads, num_key_heads, head_size, num_sequences);
}

ROPE_API int rope_attention_paged_q8(const rope_tensor *query, const rope_tensor *key_cache,
                                     const rope_tensor *value_cache, const rope_tensor *key_scales,
                                     const rope_tensor *value_scales,
                                     const rope_tensor *page_table, const rope_tensor *seq_lens,
                                     const rope_tensor *query_offsets, double scale,
                                     const rope_tensor *out, const rope_tensor *lse,
                                     void *workspace, int64_t workspace_bytes, void *stream) {
  AttnQ8Plan plan;
  std::string err;
  const int st = plan_attention_q8(query, key_cache, value_cache, key_scales, value_scales,
                                   page_table, seq_lens, query_offsets, scale, out, lse, workspace,
                                   workspace_bytes, &plan, &err);
  if (st != ROPE_OK) {
    g_last_error = err;
    return st;
  }
  g_last_error.clear();
  if (plan.noop) return ROPE_OK;
  return plan.dt == ROPE_F16 ? run_attention_q8_f16(plan, stream)
                             : run_attention_q8<__bf16>(plan, stream);
}
