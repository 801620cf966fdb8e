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

// Segments (one CTA of a cluster each) of the token recurrence over T tokens whose sweeps have `units` CTAs of up to `rows`
// state rows.  one[n], two[n]: clusters of n CTAs that the device places at once with one, two CTAs per SM (0: none), for
// n = 2 .. kMaxRecSegments.
// Every segment but the first and the last is passed twice at the same cost per token, and the last one adds up the sums of
// n - 1 others, so the choice is the least of
//     T t                     whole                     t = 0.080, 0.077, 0.122, 0.225 us for 32, 64, 128, 256 rows
//     2 T / n t c + 0.006 n rows + 2     segments       c = 1 with an SM per CTA; half an SM each, up to 128 rows,
//                                                       1.65 (1.3 up to 32 rows)
// which is within 3 % of the best of n = 1 .. 16 on average over 400 sizes (FP32, T = 128 .. 4096, 1 to 152 CTAs).  us, whole and
// in the chosen n:
//   T = 1001  r = 64   4 CTAs 80 and 19 (16); 24 CTAs 80 and 36 (10); 64 CTAs 80 and 72 (4); 100 CTAs stay whole
//             r = 128  32 CTAs 126 and 63 (8);  r = 256  16 CTAs 230 and 85 (6), 32 CTAs 230 and 119 (4)
//   T = 128   r = 64   24 CTAs 12.8 and 10.1 (5)
// Up to 64 tokens nothing is gained (T = 64, r = 64, 24 CTAs: 7.8 whole, 8.3 in five).
constexpr int kMaxRecSegments = 16, kMinRecSplit = 128;
inline int rec_segments(long long units, int rows, int T, const int *one, const int *two)
{
    if (T < kMinRecSplit) return 1;
    const double t = rows <= 32 ? 0.080 : rows <= 64 ? 0.077 : rows <= 128 ? 0.122 : 0.225;
    const int w = rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
    double best = t * T;
    int segments = 1;
    for (int n = 2; n <= kMaxRecSegments; ++n) {
        const bool whole = units <= one[n];
        if (!whole && (rows > 128 || units > two[n])) continue;
        const double us = 2 * ((T + n - 1) / n) * t * (whole ? 1.0 : rows <= 32 ? 1.3 : 1.65) + 0.006 * n * w + 2;
        if (us < best) best = us, segments = n;
    }
    return segments;
}

// Columns per lane (1, 2 or 4) of the token recurrence with `rows` state rows per CTA and `ctas` CTAs, in one piece; brief:
// packed sequences, or at most 64 tokens.  See decay_rec_kernel for what they cost.
inline int rec_columns(int rows, long long ctas, bool brief, int sms)
{
    if (rows <= 64) return ctas <= sms ? 1 : 2;
    return ctas > sms && brief ? 4 : 2;
}

}  // namespace la
