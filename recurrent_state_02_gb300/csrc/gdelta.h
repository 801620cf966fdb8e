// gdelta.h -- the gated delta rule (internal): its sweeps and their launchers.
#pragma once

#include "kernels.h"

namespace la {

// Gates below this count as this in the sums of the gates' gradient, which then divide it out again (2^-64).
constexpr float kLeastGate = 5.421010862427522e-20f;

// The sizes and gates that every launcher shares.  Value heads H, query and key heads Hk (H a
// multiple): value head h reads key head h / (H / Hk).
struct GdeltaShape {
    int B = 0, H = 0, Hk = 0, T = 0, r = 0, dv = 0;   // T: tokens per sequence, or in all when packed
    const float *alpha = nullptr, *beta = nullptr;    // [B,H,T] ([T,H] when packed) or nullptr (1)
    const int *cu_seqlens = nullptr;                  // packed sequences, or nullptr: [B,H,T,d]
    int *status = nullptr;                            // device status word
};

struct GdeltaForward {
    const void *q = nullptr, *k = nullptr, *v = nullptr;
    const float *S0 = nullptr;                        // [B,H,r,dv] or nullptr (zero)
    void *y = nullptr;
    float *S_out = nullptr;                           // [B,H,r,dv]; may equal S0
    float scale = 1.f;
};

// The token recurrence in FP32 on CUDA cores, for any 1 <= r, dv <= 256 and either element type.
cudaError_t launch_gdelta_rec(const GdeltaShape &s, const GdeltaForward &f, bool bf16, cudaStream_t stream);

// The same for a dense call in segments where few heads leave SMs idle: workspace floats (0: none needed), and the launch.
size_t gdelta_rec_floats(int B, int H, int T, int r, int dv, int sms);
cudaError_t launch_gdelta_rec_segments(const GdeltaShape &s, const GdeltaForward &f, bool bf16, int sms, float *ws, cudaStream_t stream);

// One token, S in place; dv a multiple of 4, S 16-byte aligned, r <= 256.
cudaError_t launch_gdelta_decode(const GdeltaShape &s, const void *q, const void *k, const void *v, bool bf16, float *S,
                                 float scale, void *y, cudaStream_t stream);

struct GdeltaBackward {
    const void *q = nullptr, *k = nullptr, *v = nullptr, *dy = nullptr;
    const float *S0 = nullptr, *dS_T = nullptr;       // [B,H,r,dv] or nullptr (zero)
    void *dq = nullptr, *dk = nullptr, *dv_out = nullptr;
    float *dalpha = nullptr, *dbeta = nullptr;        // [B,H,T] or nullptr
    float *dS0 = nullptr;
    float scale = 1.f;
    float *ws = nullptr;                              // gdelta_rec_backward_floats floats
};

// The gradients as four such recurrences and two passes over their FP32 results.
size_t gdelta_rec_backward_floats(int B, int H, int T, int r, int dv);
cudaError_t launch_gdelta_rec_backward(const GdeltaShape &s, const GdeltaBackward &g, bool bf16, cudaStream_t stream);

// dq and dk [B,Hk,T,r] as the sums of FP32 [B,H,T,r] over the value heads that share a key head.
cudaError_t launch_gdelta_group_sum(const GdeltaShape &s, const float *dq, const float *dk, bool bf16, void *dq_out, void *dk_out,
                                    cudaStream_t stream);

// Token log-probabilities (logprob.cu): rows of logits, row_stride elements apart.
struct LogprobArgs {
    const void *logits = nullptr;
    long long row_stride = 0;
    const int *tokens = nullptr;                      // [N]; negative: the row is skipped
    int N = 0, V = 0, top = 0;
    float *logprobs = nullptr, *entropy = nullptr, *lse = nullptr;   // [N]; entropy, lse or nullptr
    float *top_logprobs = nullptr;                    // [N,top]
    int *top_tokens = nullptr;                        // [N,top]
    int *status = nullptr;
};
constexpr int kMaxTop = 32;
cudaError_t launch_token_logprobs(const LogprobArgs &a, bool bf16, int sms, cudaStream_t stream);

struct LogprobGradArgs {
    const void *logits = nullptr;
    long long row_stride = 0, grad_stride = 0;
    const int *tokens = nullptr;
    const float *lse = nullptr, *entropy = nullptr, *dlogprobs = nullptr, *dentropy = nullptr;   // [N]
    int N = 0, V = 0;
    void *dlogits = nullptr;
    int *status = nullptr;
};
cudaError_t launch_token_logprobs_backward(const LogprobGradArgs &a, bool bf16, int sms, cudaStream_t stream);

}  // namespace la
