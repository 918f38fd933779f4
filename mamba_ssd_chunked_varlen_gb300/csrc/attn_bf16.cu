// The attention kernels over a bf16 cache.
#include "attn_few.cuh"
#include "attn_kernel.cuh"

namespace ssd {

cudaError_t launch_attn_bf16(const AttnParams &p, const AttnMaps &m, cudaStream_t s)
{
    return launch_type<SSD_KV_BF16>(p, m, s);
}

cudaError_t launch_attn_few_bf16(const AttnParams &p, cudaStream_t s)
{
    return launch_few<SSD_KV_BF16>(p, s);
}

}  // namespace ssd
