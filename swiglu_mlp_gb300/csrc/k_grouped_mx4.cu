// k_grouped_mx4.cu — the products with microscaled 4-bit operands.
#include "grouped_launch.cuh"

namespace swg {

template <int MATH, bool FEW>
static cudaError_t launch_f4(GrpEpi epi, const GrpMaps &m, const GrpParams &p, long long units,
                             int sms, cudaStream_t s)
{
    return epi == GRP_STORE ? launch_grouped_kernel<MATH, GRP_STORE, FEW>(m, p, units, sms, s)
                            : launch_grouped_kernel<MATH, GRP_SWIGLU, FEW>(m, p, units, sms, s);
}

cudaError_t launch_grouped_f4(bool nv, GrpEpi epi, bool few, const GrpMaps &m, const GrpParams &p,
                              long long units, int sms, cudaStream_t s)
{
    if (nv)
        return few ? launch_f4<MATH_NV, true>(epi, m, p, units, sms, s)
                   : launch_f4<MATH_NV, false>(epi, m, p, units, sms, s);
    return few ? launch_f4<MATH_MX, true>(epi, m, p, units, sms, s)
               : launch_f4<MATH_MX, false>(epi, m, p, units, sms, s);
}

}  // namespace swg
