// The selective scan's prompts, fp32 activations.
#include "scan_prompts.cuh"

int lstm::launch_scan_f32(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream)
{
    return launch_scan<float>(p, plan, workspace, stream);
}
