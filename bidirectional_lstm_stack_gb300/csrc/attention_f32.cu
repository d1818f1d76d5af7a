// Linear attention over prompts in fp32.
#include "attention_prompts.cuh"

namespace lstm {

int launch_attention_f32(const AttentionArgs &p, const Spans &spans, cudaStream_t stream)
{
    return prompts::launch_keys<float>(p, spans, stream);
}

}  // namespace lstm
