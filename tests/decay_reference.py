"""64-bit references of the decayed linear attention and the beam search operators,
written from their formulas (torch on the CPU, one token at a time), and the error bounds
that the tests hold the kernels to.

Every reference can also be run on absolute values: the sums it then returns bound how far
rounded products and sums can move each element, which is what the tolerances multiply.

Unit round-offs used (half a step): BF16 2^-8, FP32 2^-24.  A kernel that truncates its
FP32 accumulation counts 2^-23 per addition."""
import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().cpu().double()


def prefill(q, k, v, decay, S0, scale):
    """[B,H,T,*] -> (y, S_T)."""
    q, k, v, g = f64(q), f64(k), f64(v), f64(decay)[None, :, None, None]
    B, H, T, r = q.shape
    S = torch.zeros((B, H, r, v.shape[3]), dtype=torch.float64) if S0 is None else f64(S0).clone()
    y = torch.zeros(v.shape, dtype=torch.float64)
    for t in range(T):
        S = g * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        y[:, :, t] = scale * (q[:, :, t, :, None] * S).sum(2)
    return y, S


def backward(q, k, v, dy, decay, S0, dS_T, scale):
    """dL/dq, dL/dk, dL/dv, dL/dS0 by the chain rule through the recurrence."""
    q, k, v, dy, g = f64(q), f64(k), f64(v), f64(dy), f64(decay)[None, :, None, None]
    B, H, T, r = q.shape
    n = v.shape[3]
    zero = torch.zeros((B, H, r, n), dtype=torch.float64)
    S = zero.clone() if S0 is None else f64(S0).clone()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(T):
        S = g * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        dq[:, :, t] = scale * (S * dy[:, :, t, None, :]).sum(3)
    dS = zero.clone() if dS_T is None else f64(dS_T).clone()
    for t in reversed(range(T)):
        dS = dS + scale * q[:, :, t, :, None] * dy[:, :, t, None, :]
        dk[:, :, t] = (dS * v[:, :, t, None, :]).sum(3)
        dv[:, :, t] = (dS * k[:, :, t, :, None]).sum(2)
        dS = g * dS
    return dq, dk, dv, dS


def absolute(*ts):
    return [None if t is None else t.detach().abs() for t in ts]


def bounds(T, r, n, bf16, abs_out, out, chunked):
    """(bound of an output row's elements): abs_out is the reference on absolute values."""
    # the sums: T writes carried along, r (or n) products, a few factors
    acc = (T + max(r, n) + 16) * (2 * U32)
    tol = acc * abs_out
    if bf16:
        tol = tol + U16 * out.abs()            # the output's own rounding
        if chunked:
            tol = tol + 1.02 * U16 * abs_out   # the scores, or the carried state, as BF16 operands
    return tol + 1e-30


def state_bound(T, abs_S, chunked):
    """The state: FP32 throughout; the chunked form splits w v into two BF16 parts, which
    keep it to U16^2, and accumulates at most 16 products of 16 per chunk of 128."""
    tol = (T + 16) * (2 * U32) * abs_S
    if chunked:
        tol = tol + U16 * U16 * abs_S
    return tol + 1e-30


def check(got, ref, tol, what):
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got - ref).abs()
    worst = float((err / tol).max()) if err.numel() else 0.0
    print(f"[decay] {what}: largest error / bound {worst:.3f}")
    assert worst <= 1.0, f"{what}: error {worst:.3f} of its bound"


def select(logits, scores, done, eos):
    """The K best candidates of every request, in Python numbers and 64 bits."""
    B, K, V = logits.shape
    x, s = f64(logits), f64(scores)
    outs = ([], [], [], [])
    for b in range(B):
        cand = []
        for k in range(K):
            if done is not None and bool(done[b, k]):
                if math.isfinite(float(s[b, k])):
                    cand.append((-float(s[b, k]), k, eos))
                continue
            row = x[b, k]
            lse = float(torch.logsumexp(row, 0))
            if not math.isfinite(lse) or not math.isfinite(float(s[b, k])):
                continue
            c = float(s[b, k]) + row - lse
            cand += [(-float(c[i]), k, i) for i in range(V) if row[i] != -math.inf]
        cand.sort()
        best = cand[:K]
        row = [], [], [], []
        for j in range(K):
            own = done is not None and bool(done[b, j])
            score, par, tok, end = (-best[j][0], best[j][1], best[j][2], None) if j < len(best) else (-math.inf, j, 0, own)
            if end is None:
                end = (done is not None and bool(done[b, par])) or tok == eos
            for lst, val in zip(row, (score, par, tok, int(end))):
                lst.append(val)
        for o, r_ in zip(outs, row):
            o.append(r_)
    return [torch.tensor(o, dtype=d) for o, d in zip(outs, (torch.float64, torch.int32, torch.int32, torch.uint8))]
