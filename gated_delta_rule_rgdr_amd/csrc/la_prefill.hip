// la_prefill.hip -- linear attention with a decay for each head, over whole prompts.
#include "la_common.h"

namespace rgdr {
constexpr int kLaMaxPrompt = 65536;
}  // namespace rgdr

extern "C" rgdr_status la_prefill_workspace_size(int32_t B, int32_t H_v, int32_t T, int32_t D_k,
                                                 int32_t D_v, size_t *bytes) {
    using namespace rgdr;
    if (!bytes) return RGDR_ERR_NULL;
    if (const rgdr_status st = la_check_sizes(kLaMaxPrompt, B, H_v, T, D_k, D_v)) return st;
    *bytes = 0;
    return RGDR_OK;
}

extern "C" rgdr_status la_prefill(const void *query, const la_strides *query_strides,
                                  const void *key, const la_strides *key_strides,
                                  const void *value, const la_strides *value_strides,
                                  const float *g, const la_strides *g_strides,
                                  const void *state_pool, const uint8_t *state_scales,
                                  rgdr_dtype state_dtype, const int32_t *actual_seq_lengths,
                                  const int32_t *ssm_state_indices,
                                  const int32_t *num_accepted_tokens, float scale, int32_t B,
                                  int32_t H_q, int32_t H_v, int32_t T, int32_t D_k, int32_t D_v,
                                  int32_t N_slots, void *out, const la_strides *out_strides,
                                  void *state_out, uint8_t *state_scales_out, void *workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
    using namespace rgdr;
    LaArgs a;
    if (const rgdr_status st = la_check(
            a, kLaMaxPrompt, query, query_strides, key, key_strides, value, value_strides, g,
            g_strides, state_pool, state_scales, state_dtype, actual_seq_lengths,
            ssm_state_indices, num_accepted_tokens, scale, B, H_q, H_v, T, D_k, D_v, N_slots, out,
            out_strides, state_out, state_scales_out))
        return st;
    if (B == 0) return RGDR_OK;
    if (workspace && !aligned(workspace, 256)) return RGDR_ERR_ALIGN;
    (void)workspace_bytes;
    return la_launch_recurrent(a, state_dtype, D_k, stream);
}
