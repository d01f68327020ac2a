// k_grouped.cu — the grouped products with 16-bit operands.
#include "grouped_launch.cuh"

namespace swg {

template <bool FEW>
static cudaError_t launch_16(GrpEpi epi, const GrpMaps &m, const GrpParams &p, long long units,
                             int sms, cudaStream_t s)
{
    switch (epi) {
    case GRP_STORE: return launch_grouped_kernel<MATH_16, GRP_STORE, FEW>(m, p, units, sms, s);
    case GRP_SWIGLU: return launch_grouped_kernel<MATH_16, GRP_SWIGLU, FEW>(m, p, units, sms, s);
    default: return launch_grouped_kernel<MATH_16, GRP_DSWIGLU, FEW>(m, p, units, sms, s);
    }
}

cudaError_t launch_grouped_16(GrpEpi epi, bool few, const GrpMaps &m, const GrpParams &p,
                              long long units, int sms, cudaStream_t s)
{
    return few ? launch_16<true>(epi, m, p, units, sms, s) : launch_16<false>(epi, m, p, units, sms, s);
}

}  // namespace swg
