// decay.h -- linear attention with a constant decay per head (internal): the
// sweep that prefill and the gradients share, and its launchers.
#pragma once

#include "kernels.h"

namespace la {

// One sweep over the tokens of every (b, h), forwards or backwards in time.  With
// g = decay[h] and the tokens in the sweep's own order t = 0 .. T-1,
//     S_t   = f_t S_{t-1} + w b_t c_t^T,      f_t = g (f_0 = 1 when late)
//     out_t = s_tok a_t^T S_t                 (s_state for what S_init contributes and
//                                              what earlier writes left in the state)
//     S_fin = S_{T-1}                         (g S_{T-1} when late)
// Prefill is the forward sweep (a, b, c) = (q, k, v).  The gradients are three more:
//     dq   forwards,   (dy, v, k),  S_init = S0^T,    s = scale
//     dk   backwards,  (v, dy, q),  S_init = dS_T^T,  w = scale, late
//     dv   backwards,  (k, q, dy),  S_init = dS_T,    w = scale, late;  S_fin = dS0
// (late: the last token reads dS_T undecayed, and dS0 = g G_1.)
struct DecaySweep {
    const void *a = nullptr, *b = nullptr;   // [.., ra]
    const void *c = nullptr;                 // [.., n]
    void *out = nullptr;                     // [.., n]
    const float *S_init = nullptr;           // [B,H,ra,n], or [B,H,n,ra] when init_t; nullptr: zero
    float *S_fin = nullptr;                  // [B,H,ra,n] or nullptr (not kept); may equal S_init
    int ra = 0, n = 0;
    bool init_t = false, rev = false, late = false;
    float out_scale = 1.f, write_scale = 1.f;
};

struct DecayArgs {
    const float *decay = nullptr;            // [H]
    const int *cu_seqlens = nullptr;         // packed sequences (token-major), or nullptr: [B,H,T,d]
    int H = 0, T = 0;                        // T: tokens per sequence, or in all when packed
    int len_min = 0, len_max = 0x7fffffff;   // packed: the lengths this launch takes
    int *status = nullptr;
    int sms = 0;                             // of the device
};

// The token recurrence in FP32 on CUDA cores, for any 1 <= ra, n <= 256 and either
// element type; `sweeps` (1..3) run as one grid.
cudaError_t launch_decay_rec(const DecaySweep *sweeps, int count, const DecayArgs &a, bool bf16, int B,
                             cudaStream_t stream);

// The same sweeps in chunks of 128 tokens on the tensor cores (decay_tc.cu): BF16, every
// sweep with the same ra (64 or 128), n a multiple of 64, late == rev, arrays 16-byte
// aligned.  Maps: boxes of 64 columns x 128 tokens with the 128-byte swizzle over
// [B*H, T, d], or [tokens, H, d] when packed.
struct TcSweepMaps {
    CUtensorMap a, b, c, out;   // (out: boxes of 64 columns x 32 tokens)
};
struct DecayTcParams {
    TcSweepMaps maps[3];
    DecaySweep sw[3];
    int tiles[3] = {};     // 64-column tiles of each sweep
    DecayArgs d;
    int B = 0;
    // The split of [B,H,T,d] sweeps (decay_split): nseg segments of seg_chunks chunks; the first nseg - 1
    // are parts of part_chunks chunks (nparts of them), whose sums the state pass leaves in
    // parts [B*H][tiles][nparts + 1][ra][64] (the last one: the state that enters the sweep).
    int nseg = 1, seg_chunks = 0, part_chunks = 0, nparts = 0;
    float *parts = nullptr;
};
cudaError_t launch_decay_tc(const DecayTcParams &p, int ra, cudaStream_t stream);

// One token, S in place: S <- g S + k v^T, y = scale q^T S.  dv a multiple of 4, S and
// v 4-element aligned, r <= 256.
cudaError_t launch_decay_decode(const void *q, const void *k, const void *v, bool bf16, const float *decay, float *S,
                                int B, int H, int r, int dv, float scale, void *y, cudaStream_t stream);

// Beam selection and state reordering (beam.cu).
struct BeamSelectArgs {
    const void *logits = nullptr;       // [B][K][V], rows row_stride elements apart
    long long row_stride = 0;
    const float *scores = nullptr;      // [B][K]
    const unsigned char *done = nullptr;   // [B][K] or nullptr
    float *next_scores = nullptr;       // [B][K]; may equal scores
    int *parents = nullptr, *tokens = nullptr;   // [B][K]
    unsigned char *done_out = nullptr;  // [B][K] or nullptr; may equal done
    int K = 0, V = 0, eos = -1;
};
constexpr int kMaxBeams = 32;
cudaError_t launch_beam_select(const BeamSelectArgs &a, int B, bool bf16, int sms, cudaStream_t stream);

// slot j of request b <- slot parents[b][j]; S slots of s_len floats, z slots of z_len
// (z may be nullptr).  S_out, z_out equal S, z (in place) or do not overlap them.
cudaError_t launch_state_reorder(const float *S, const float *z, const int *parents, int B, int K, long long s_len,
                                 long long z_len, float *S_out, float *z_out, int *status, cudaStream_t stream);

}  // namespace la
