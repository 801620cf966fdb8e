// launch_rules.h -- sizes and choices that are plain arithmetic: no CUDA in here, so that a host compiler can
// check them as well.
#pragma once

#ifdef __CUDACC__
#define LA_HD __host__ __device__
#else
#define LA_HD
#endif

namespace la {

// Beam selection reads an aligned row of V elements in 16-byte granules of `ge` elements.  Granules 0 .. whole_granules - 1
// lie in the row and are read by one load; what is left of it (the last row may end the caller's buffer) by elements.
LA_HD inline int whole_granules(int V, int ge) { return V / ge; }

// Columns per lane (1, 2 or 4) of the token recurrence with `rows` state rows per CTA and `ctas` CTAs, in one piece; brief:
// packed sequences, or at most 64 tokens.  See decay_rec_kernel for what they cost.
inline int rec_columns(int rows, long long ctas, bool brief, int sms)
{
    if (rows <= 64) return ctas <= sms ? 1 : 2;
    return ctas > sms && brief ? 4 : 2;
}

}  // namespace la
