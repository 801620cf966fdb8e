// gdelta_tc.h -- the gated delta rule in chunks of 64 tokens on the tensor cores (internal).
#pragma once

#include "gdelta.h"

namespace la {

// BF16, r 64 or 128, dv a multiple of 64, q, k, v 16-byte aligned.
// Maps: boxes of 64 columns x 64 tokens with the 128-byte swizzle over [B*heads, T, d], or [tokens, heads, d] when packed.
struct GdeltaTcMaps {
    CUtensorMap q, k, v;
};

struct GdeltaTcArgs {
    GdeltaShape s;
    const float *S0 = nullptr;      // [B,H,r,dv] or nullptr
    float *S_out = nullptr;         // may equal S0
    uint16_t *y = nullptr;
    float scale = 1.f;
    uint8_t *ws = nullptr;          // A, X and the gates of every chunk and head (256-byte aligned)
    int first = 0, chunks = 0;      // dense: this launch's chunks of every sequence (0: all of them)
    int *slot_base = nullptr;       // packed: the plan's tables, B + 1 and B entries, or nullptr (up to 32 sequences: no plan)
    int *order = nullptr;
};

// Chunks of the call (packed: at most this many), the plan's bytes and the whole workspace's.
long long gdelta_tc_slots(int B, int T, bool packed);
size_t gdelta_tc_plan_bytes(int B);
size_t gdelta_tc_workspace_bytes(int B, int H, int T, bool packed);

cudaError_t launch_gdelta_tc(const GdeltaTcMaps &m, const GdeltaTcArgs &a, int sms, cudaStream_t stream);

// The gradients (gdelta_bwd.cu): [B,H,T,d], r 64 or 128, dv 64 or 128, token arrays 16-byte aligned, the workspace 256-byte.
struct GdeltaTcBackMaps {
    CUtensorMap q, k, v, dy;
};
struct GdeltaTcBackArgs {
    GdeltaShape s;
    const float *S0 = nullptr, *dS_T = nullptr;
    float *dS0 = nullptr, *dalpha = nullptr, *dbeta = nullptr;
    uint16_t *dv_out = nullptr;
    void *dq = nullptr, *dk = nullptr;      // BF16 [B,H,T,r], or FP32 where key heads are shared
    float scale = 1.f;
    // per chunk and head: prep's images and gates; E and N (two parts); the state before it and the gradient behind it (two parts)
    uint8_t *ws = nullptr, *E = nullptr, *N = nullptr, *S = nullptr, *dS = nullptr;
};
size_t gdelta_tc_backward_bytes(const GdeltaShape &s);
cudaError_t launch_gdelta_tc_backward(const GdeltaTcBackMaps &m, const GdeltaShape &s, const GdeltaBackward &g, int sms,
                                      cudaStream_t stream);
cudaError_t launch_gdelta_prep_backward(const CUtensorMap &q, const CUtensorMap &k, const GdeltaTcArgs &a, cudaStream_t stream);

}  // namespace la
