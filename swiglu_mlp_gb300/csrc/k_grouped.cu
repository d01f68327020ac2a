// k_grouped.cu — the grouped products with 16-bit operands.
#include "grouped_launch.cuh"

namespace swg {

cudaError_t launch_grouped_16(GrpEpi epi, const GrpMaps &m, const GrpParams &p, long long units,
                              int sms, cudaStream_t s)
{
    constexpr int smem = GrpCfg<MATH_16>::SMEM_BYTES;
    switch (epi) {
    case GRP_STORE: return launch_pairs<grouped_kernel<MATH_16, GRP_STORE>, NUM_THREADS>(smem, units, sms, s, m, p);
    case GRP_SWIGLU: return launch_pairs<grouped_kernel<MATH_16, GRP_SWIGLU>, NUM_THREADS>(smem, units, sms, s, m, p);
    default: return launch_pairs<grouped_kernel<MATH_16, GRP_DSWIGLU>, NUM_THREADS>(smem, units, sms, s, m, p);
    }
}

}  // namespace swg
