// The selective scan's prompts, fp16 activations.
#include "scan_prompts.cuh"

int lstm::launch_scan_f16(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream)
{
    return launch_scan<__half>(p, plan, workspace, stream);
}
