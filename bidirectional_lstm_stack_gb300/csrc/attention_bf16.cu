// Linear attention over prompts in bf16.
#include "attention_prompts.cuh"

namespace lstm {

int launch_attention_bf16(const AttentionArgs &p, const Spans &spans, cudaStream_t stream)
{
    return prompts::launch_keys<__nv_bfloat16>(p, spans, stream);
}

}  // namespace lstm
