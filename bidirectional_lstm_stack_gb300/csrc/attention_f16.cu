// Linear attention over prompts in fp16.
#include "attention_prompts.cuh"

namespace lstm {

int launch_attention_f16(const AttentionArgs &p, const Spans &spans, cudaStream_t stream)
{
    return prompts::launch_keys<__half>(p, spans, stream);
}

}  // namespace lstm
