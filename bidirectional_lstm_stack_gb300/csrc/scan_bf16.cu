// The selective scan's prompts, bf16 activations.
#include "scan_prompts.cuh"

int lstm::launch_scan_bf16(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream)
{
    return launch_scan<__nv_bfloat16>(p, plan, workspace, stream);
}
