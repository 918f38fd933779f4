// The attention kernels over a int8 cache.
#include "attn_few.cuh"
#include "attn_kernel.cuh"

namespace ssd {

cudaError_t launch_attn_int8(const AttnParams &p, const AttnMaps &m, cudaStream_t s)
{
    return launch_type<SSD_KV_INT8>(p, m, s);
}

cudaError_t launch_attn_few_int8(const AttnParams &p, cudaStream_t s)
{
    return launch_few<SSD_KV_INT8>(p, s);
}

}  // namespace ssd
