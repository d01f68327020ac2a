// chunks.h — how the router's kernels share out tokens, and a plan's its slots.  There are
// up to 2^31 - 1024 of them: what a whole grid (up to 2^28 CTAs), or a rounding up, adds to
// such a number passes an int, but not 32 bits without a sign, in which all of this is
// computed (64-bit divisions take longer).  Plain C++, for the host as well.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SWG_BOTH __host__ __device__ __forceinline__
#else
#define SWG_BOTH inline
#endif

namespace swg {

// The tokens of chunk c of n: from .. to - 1.
SWG_BOTH void chunk_of(int T, uint32_t n, uint32_t c, int &from, int &to)
{
    const uint32_t t = T, per = (t + n - 1) / n, a = c * per, b = a + per;      // (b < t + n)
    from = (int)(a < t ? a : t);
    to = (int)(b < t ? b : t);
}

// The slots that warp `warp` of those that rank a chunk's slots lo .. hi - 1 has: from ..
// to - 1, whole times 32 from lo on, none for the warps behind the last.
SWG_BOTH void slots_of_warp(int lo, int hi, uint32_t ranking, uint32_t warp, int &from, int &to)
{
    const uint32_t end = hi, per = ((end - lo + ranking - 1) / ranking + 31) & ~31u;
    const uint32_t a = lo + (warp < ranking ? warp : ranking) * per, b = a + per;       // (a < end + 32 ranking)
    from = (int)(a < end ? a : end);
    to = warp >= ranking ? from : (int)(b < end ? b : end);
}

// The places behind a plan's `rows` rows that a thread fills: first, first + step, ...
SWG_BOTH void behind_rows(int rows, uint32_t cta, uint32_t ctas, uint32_t threads, uint32_t tid, uint32_t &first, uint32_t &step)
{
    step = ctas * threads;
    first = rows + cta * threads + tid;
}

}  // namespace swg
