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

}  // namespace la
