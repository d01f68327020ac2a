// chunks.h — how the kernels of a plan share out its slots.  There are up to
// 2^31 - 1024 of them: what a whole grid, or a rounding up, adds to such a number
// passes 32 bits, so that sums are formed in 64.  (Plain C++, for the host as well.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SWG_BOTH __host__ __device__ __forceinline__
#else
#define SWG_BOTH inline
#endif

namespace swg {

// The slots that warp `warp` of those that rank a chunk's slots lo .. hi - 1 has: from ..
// to - 1, whole times 32 from lo on, none for the warps behind the last.
SWG_BOTH void slots_of_warp(int lo, int hi, int ranking, int warp, int &from, int &to)
{
    const int64_t per = (((int64_t)hi - lo + ranking - 1) / ranking + 31) / 32 * 32;
    const int64_t a = lo + warp * per, b = a + per;
    from = (int)(a < hi ? a : hi);
    to = warp >= ranking ? from : (int)(b < hi ? b : hi);
}

// The places behind a plan's `rows` rows that a thread fills: first, first + step, ...
SWG_BOTH void behind_rows(int rows, int cta, int ctas, int threads, int tid, int64_t &first, int64_t &step)
{
    step = (int64_t)ctas * threads;
    first = rows + (int64_t)cta * threads + tid;
}

}  // namespace swg
