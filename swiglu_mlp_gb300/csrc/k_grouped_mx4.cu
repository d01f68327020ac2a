// k_grouped_mx4.cu — the products with microscaled 4-bit operands.
#include "grouped_launch.cuh"

namespace swg {

cudaError_t launch_grouped_f4(bool nv, GrpEpi epi, const GrpMaps &m, const GrpParams &p,
                              long long units, int sms, cudaStream_t s)
{
    if (nv) {
        constexpr int smem = GrpCfg<MATH_NV>::SMEM_BYTES;
        return epi == GRP_STORE
                   ? launch_pairs<grouped_kernel<MATH_NV, GRP_STORE>, NUM_THREADS>(smem, units, sms, s, m, p)
                   : launch_pairs<grouped_kernel<MATH_NV, GRP_SWIGLU>, NUM_THREADS>(smem, units, sms, s, m, p);
    }
    constexpr int smem = GrpCfg<MATH_MX>::SMEM_BYTES;
    return epi == GRP_STORE
               ? launch_pairs<grouped_kernel<MATH_MX, GRP_STORE>, NUM_THREADS>(smem, units, sms, s, m, p)
               : launch_pairs<grouped_kernel<MATH_MX, GRP_SWIGLU>, NUM_THREADS>(smem, units, sms, s, m, p);
}

}  // namespace swg
