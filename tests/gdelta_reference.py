"""64-bit references of the gated delta rule and the token log-probabilities, written from their formulas, one token
(one row) at a time, and the error bounds that the tests hold the kernels to.

With keys of length one, 0 <= alpha, beta <= 1, every step alpha (I - beta k k^T) shrinks a difference between two states, so
rounding errors enter once and do not grow: an output's error is a sum of independent roundings, each relative to a term as large
as the output's own terms.  Unit round-offs (half a step): BF16 2^-8, FP32 2^-24.
  FP32 inputs: a sum of up to 256 products per token, and the state rounded twice by each of T tokens (scaled, written to), none of
      which it need forget: sqrt(256 + 2 T) half steps of 2^-24 of the norm.
  BF16 inputs, BF16 outputs: the output's own rounding and at most three on the way (the state, the scores and the written rows
      as tensor-core operands): 4 x 2^-8 of the norm.
  BF16 inputs, FP32 outputs: derived operands are split into two BF16 parts, which keeps each to 2^-16 x 1/2 of its size, and a result
      passes at most four of them; random in sign they add up to sqrt(4) 2^-17 = 2^-16 of the norm.
What a sum cancels does not shrink its terms' errors, so each norm is that of the terms where that is larger: of the r products in
lam = G^T k (for dv), of lam . e (for dbeta), and of the tokens' terms q . dq and v . dv from t on (for dalpha, where they
are what S and G at t hold).  Single elements may be off by eight such norms' share (8 standard deviations of a sum of roundings)."""
import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().cpu().double()


def _wide(x, H, dim=1):
    return f64(x).repeat_interleave(H // x.shape[dim], dim=dim)


def _gate(a, shape):
    return torch.ones(shape, dtype=torch.float64) if a is None else f64(a)


def prefill(q, k, v, alpha, beta, S0, scale):
    """[B,H,T,*] -> (y, S_T, errors e, states after each token's decay S')."""
    v = f64(v)
    B, H, T, n = v.shape
    q, k = _wide(q, H), _wide(k, H)
    a, b = _gate(alpha, (B, H, T)), _gate(beta, (B, H, T))
    S = torch.zeros((B, H, q.shape[3], n), dtype=torch.float64) if S0 is None else f64(S0).clone()
    y, e, decayed = torch.zeros_like(v), torch.zeros_like(v), []
    for t in range(T):
        S = a[:, :, t, None, None] * S
        decayed.append(S)
        e[:, :, t] = v[:, :, t] - (k[:, :, t, :, None] * S).sum(2)
        S = S + k[:, :, t, :, None] * (b[:, :, t, None] * e[:, :, t])[:, :, None, :]
        y[:, :, t] = scale * (q[:, :, t, :, None] * S).sum(2)
    return y, S, e, decayed


def backward(q, k, v, dy, alpha, beta, S0, dS_T, scale):
    """(dq, dk, dv, dalpha, dbeta, dS0) by the chain rule, dalpha from the states themselves, so that no gate is divided by; and
    the roots of the summed squares of the terms of dv, dalpha and dbeta."""
    y, S, e, decayed = prefill(q, k, v, alpha, beta, S0, scale)
    B, H, T, n = y.shape
    Hk, r = q.shape[1], q.shape[3]
    rep = H // Hk
    q, k, dy = _wide(q, H), _wide(k, H), scale * f64(dy)
    a, b = _gate(alpha, (B, H, T)), _gate(beta, (B, H, T))
    before = [torch.zeros_like(S) if S0 is None else f64(S0)]
    for t in range(T):
        before.append(decayed[t] + k[:, :, t, :, None] * (b[:, :, t, None] * e[:, :, t])[:, :, None, :])
    G = torch.zeros_like(S) if dS_T is None else f64(dS_T).clone()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(y)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    dv_terms, db_terms, da_terms = torch.zeros_like(y), torch.zeros_like(b), torch.zeros_like(a)
    tail = torch.zeros((B, H), dtype=torch.float64) if dS_T is None else (S * f64(dS_T)).square().sum((2, 3))
    for t in reversed(range(T)):
        dq[:, :, t] = (before[t + 1] * dy[:, :, t, None, :]).sum(3)
        G = G + q[:, :, t, :, None] * dy[:, :, t, None, :]
        G0 = G
        lam = (G * k[:, :, t, :, None]).sum(2)
        dv[:, :, t] = b[:, :, t, None] * lam
        db[:, :, t] = (lam * e[:, :, t]).sum(2)
        dk[:, :, t] = b[:, :, t, None] * (G * e[:, :, t, None, :]).sum(3) - (decayed[t] * dv[:, :, t, None, :]).sum(3)
        G = G - k[:, :, t, :, None] * dv[:, :, t, None, :]
        da[:, :, t] = (G * before[t]).sum((2, 3))
        G = a[:, :, t, None, None] * G
        terms = (G0 * k[:, :, t, :, None]).square().sum(2).sqrt()
        dv_terms[:, :, t] = b[:, :, t, None] * terms
        db_terms[:, :, t] = (terms * e[:, :, t]).square().sum(2).sqrt()
        tail = tail + (q[:, :, t] * dq[:, :, t]).square().sum(2) + (f64(v)[:, :, t] * dv[:, :, t]).square().sum(2)
        da_terms[:, :, t] = tail.sqrt() / a[:, :, t].clamp(min=1e-300)
    dq, dk = (x.reshape(B, Hk, rep, T, r).sum(2) for x in (dq, dk))
    return (dq, dk, dv, da, db, G), (None, None, dv_terms, da_terms, db_terms, None)


def tolerance(inputs, out, T):
    """The bound of an output's 2-norm error, relative to its norm, from the inputs' type, its own and the tokens."""
    if inputs == torch.float32:
        return math.sqrt(256 + 2 * T) * U32
    return 4 * U16 if out == torch.bfloat16 else 2.0 ** -16


def check(got, ref, inputs, what, T=64, terms=None):
    tol = tolerance(inputs, got.dtype, T)
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if not ref.numel():
        return
    err, norm = (got - ref), float(ref.norm())
    if terms is not None:
        norm = max(norm, float(terms.norm()))
    rel = float(err.norm()) / max(norm, 1e-30)
    rms = norm / math.sqrt(ref.numel())
    big = float((err.abs() / (rms + ref.abs()).clamp(min=1e-30)).max())
    print(f"[gdelta] {what}: relative {rel:.2e} (bound {tol:.1e}), largest element {big:.2e} (bound {8 * tol:.1e})")
    assert rel <= tol and big <= 8 * tol, f"{what}: {rel:.3e} and {big:.3e} against {tol:.3e}"


NAMES = ("dq", "dk", "dv", "dalpha", "dbeta", "dS0")


def check_all(got, ref, inputs, T):
    """The six gradients (None where a gate was not given) against backward()'s."""
    for x, z, m, name in zip(got, *ref, NAMES):
        if x is not None:
            check(x, z, inputs, name, T, m)


def score(logits, tokens, top):
    """(logprob, entropy, lse, top logprobs, top tokens) per row, in Python numbers."""
    x = f64(logits)
    outs = [], [], [], [], []
    for row, t in zip(x, tokens.tolist()):
        none = ([-math.inf] * top, [-1] * top)
        if t < 0:
            vals = (0.0, 0.0, 0.0, *none)
        else:
            lse = float(torch.logsumexp(row, 0))
            if lse == -math.inf:
                vals = (-math.inf, 0.0, lse, *none)
            elif not math.isfinite(lse):
                vals = (math.nan, math.nan, math.nan, *none)
            else:
                m = float(row.max())          # (a row of one huge value keeps its log-probabilities)
                d = row - m
                lg = float(d.exp().sum().log())
                p = (d - lg).exp()
                H = lg - float((p * torch.where(p > 0, d, 0.0)).sum())
                val, at = torch.sort(d, descending=True, stable=True)
                order = [(float(a), int(b)) for a, b in zip(val[:top], at[:top]) if a != -math.inf]
                best = [a - lg for a, _ in order] + [-math.inf] * (top - len(order))
                vals = (float(d[t]) - lg, H, m + lg, best, [b for _, b in order] + [-1] * (top - len(order)))
        for o, v in zip(outs, vals):
            o.append(v)
    res = [torch.tensor(o, dtype=torch.float64) for o in outs[:4]]
    return (*res[:3], res[3].reshape(len(outs[3]), top), torch.tensor(outs[4], dtype=torch.int32).reshape(len(outs[4]), top))


def score_backward(logits, tokens, dlogprobs, dentropy):
    """dL/dlogits."""
    x = f64(logits)
    out = torch.zeros_like(x)
    for n, t in enumerate(tokens.tolist()):
        if t < 0 or float(torch.logsumexp(x[n], 0)) == -math.inf:
            continue
        lp = torch.log_softmax(x[n], 0)
        p = lp.exp()
        plogp = torch.where(p > 0, p * lp, 0.0)
        w, h = float(dlogprobs[n]), 0.0 if dentropy is None else float(dentropy[n])
        out[n] = -w * p - h * (plogp - p * float(plogp.sum()))
        out[n, t] += w
    return out
