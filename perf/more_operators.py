"""What the gated delta rule and the token log-probabilities are measured on.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes a case's inputs on the
GPU from a seed, ``run()`` is one pass through an operator (the framework's where ``own`` is true, else the same
mathematics in elementary torch operations), ``work()`` is what a pass cannot do without, and ``exact()`` is the
operator's definition in 64 bits.

    prefill   S' = alpha_t S_{t-1},  S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,  y_t = scale S_t^T q_t
              (q and k may have fewer heads than v: each is shared by neighbouring ones)
    packed    the same over sequences of different lengths packed one after another
    decode    one token of it, the state updated in place
    backward  gradients of prefill: dq, dk, dv, dalpha, dbeta, dS0 from dy, dS_T
    score     log-probabilities of given tokens, the entropy of their rows and the best alternatives
    score_bw  the gradient of the log-probabilities and the entropies with respect to the logits
"""
import math
import random

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CHUNK = 64  # tokens per chunk of the plain form


def listed():
    return [
        # a training or scoring batch: the framework's headline prefill shape
        dict(name="prefill_b4_h16_t4096", op="prefill", dtype="bf16", B=4, H=16, Hk=16, T=4096, r=128, dv=128, state=False),
        # a small exact run with odd sizes and shared keys (FP32 through and through)
        dict(name="prefill_fp32_t1001", op="prefill", dtype="fp32", B=2, H=4, Hk=2, T=1001, r=64, dv=96, state=True),
        # a serving batch of ragged prompts, each from its own carried state, two value heads to a key head
        dict(name="packed_48_prompts_h16", op="packed", dtype="bf16", B=48, H=16, Hk=8, lo=128, hi=8192, mix=8, r=128, dv=128),
        # ragged continuations of a few tokens each
        dict(name="packed_16_short_h8", op="packed", dtype="bf16", B=16, H=8, Hk=8, lo=1, hi=200, mix=3, r=128, dv=128),
        # a serving batch's decode step: bound by the state's traffic
        dict(name="decode_b256_h16", op="decode", dtype="bf16", B=256, H=16, Hk=16, r=128, dv=128),
        # one request's decode step: bound by latency
        dict(name="decode_b1_h16", op="decode", dtype="bf16", B=1, H=16, Hk=8, r=128, dv=128),
        # the gradients of the training batch
        dict(name="backward_b4_h16_t4096", op="backward", dtype="bf16", B=4, H=16, Hk=16, T=4096, r=128, dv=128, state=False),
        # gradients of a short ragged sequence through a carried state, shared keys
        dict(name="backward_b1_h8_t777", op="backward", dtype="bf16", B=1, H=8, Hk=4, T=777, r=128, dv=128, state=True),
        # scoring a batch of sampled tokens over a large vocabulary, with the alternatives an answer shows
        dict(name="score_n2048_v131072", op="score", dtype="bf16", N=2048, V=131072, top=8),
        # the log-probabilities of one decode step's token
        dict(name="score_n1_v32003", op="score", dtype="fp32", N=1, V=32003, top=5),
        # the loss of a training batch: every token's log-probability, with an entropy bonus
        dict(name="score_bw_n8192_v32000", op="score_bw", dtype="bf16", N=8192, V=32000),
        # a few rows of an odd vocabulary
        dict(name="score_bw_n60_v32003", op="score_bw", dtype="fp32", N=60, V=32003),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "packed", "decode", "backward", "score", "score_bw"])
    if op in ("score", "score_bw"):
        c = dict(op=op, dtype=rng.choice(["bf16", "fp32"]), N=_log(rng, 1, 8192), V=_log(rng, 100, 150000))
        while c["N"] * c["V"] > 260_000_000 // (2 if c["dtype"] == "fp32" else 1):
            c["N"] = max(1, c["N"] // 2)
        if op == "score":
            c["top"] = rng.choice([0, 1, 5, 8, 20])
        return c
    share = rng.choice([1, 1, 2, 4])
    if op == "decode":
        Hk = _log(rng, 1, 16)
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), B=_log(rng, 1, 256), H=Hk * share, Hk=Hk,
                 r=rng.choice([64, 96, 128, 128]), dv=rng.choice([64, 80, 128, 128]))
        while c["B"] * c["H"] > 4096:
            c["B"] = max(1, c["B"] // 2)
        return c
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"]) if op != "packed" else "bf16"
    sizes = [64, 128, 128, 128] if dtype == "bf16" else [32, 64, 96, 128]
    Hk = _log(rng, 1, 16)
    c = dict(op=op, dtype=dtype, B=_log(rng, 1, 16), H=Hk * share, Hk=Hk, r=rng.choice(sizes), dv=rng.choice(sizes))
    most = 262144 if dtype == "bf16" else 32768  # tokens x heads
    if op == "packed":
        c.update(lo=1, hi=_log(rng, 16, 4096), mix=rng.randrange(1000), B=_log(rng, 1, 64))
        while c["B"] * c["H"] * c["hi"] > 2 * 262144:
            c["hi"] = max(16, c["hi"] // 2)
            c["B"] = max(1, c["B"] // 2)
        return c
    c.update(T=_log(rng, 1, 8192), state=rng.random() < 0.5)
    while c["B"] * c["H"] * c["T"] > most:
        if c["B"] > 1:
            c["B"] //= 2
        else:
            c["T"] = max(1, c["T"] // 2)
    return c


def _lens(case):
    """The lengths of a packed case: log-uniform in lo..hi, fixed by the case."""
    rng = random.Random(case["mix"])
    return [_log(rng, case["lo"], case["hi"]) for _ in range(case["B"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sd=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * sd).to(dtype)

    def unit(*shape, dtype):  # queries and keys come normalised to length one
        x = torch.randn(shape, generator=g, device="cuda")
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    op, st = case["op"], dict(case)
    dt = _DTYPE[case["dtype"]]
    if op in ("score", "score_bw"):
        N, V = case["N"], case["V"]
        # logits of a trained model's spread; one row in sixteen is padding (no token)
        st["logits"] = normal(N, V, sd=3.0, dtype=dt)
        tokens = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        if N > 1:
            tokens[torch.rand(N, generator=g, device="cuda") < 1 / 16] = -1
        st["tokens"] = tokens
        if op == "score_bw":
            # what the forward pass left: the rows' log-sum-exp and entropy
            x = st["logits"]
            lse, ent = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
            for i in range(0, N, 1024):
                p = torch.log_softmax(x[i:i + 1024].double(), dim=1)
                lse[i:i + 1024] = (x[i:i + 1024].double()[:, 0] - p[:, 0]).float()
                ent[i:i + 1024] = -(p.exp() * p).sum(1).float()
            st["lse"], st["entropy"] = torch.where(tokens < 0, 0.0, lse), torch.where(tokens < 0, 0.0, ent)
            st["dlogprobs"], st["dentropy"] = normal(N), normal(N, sd=0.01)
        return st
    H, Hk, r, dv, B = (case[n] for n in ("H", "Hk", "r", "dv", "B"))
    st["scale"] = r ** -0.5
    # a head's memory reaches from two tokens to a thousand, and varies from token to token
    a_log = math.log(0.7 * 1024) * torch.rand(H, generator=g, device="cuda")

    def gates(*shape):  # head last
        a = torch.exp(-torch.exp(a_log) / 1024 * torch.nn.functional.softplus(1.0 + normal(*shape)) / 1.3)
        return a, torch.sigmoid(normal(*shape))

    if op == "packed":
        lens = _lens(case)
        total = sum(lens)
        st["lens"] = lens
        st["cu"] = torch.tensor([0] + [sum(lens[: i + 1]) for i in range(B)], dtype=torch.int32, device="cuda")
        st["q"], st["k"], st["v"] = unit(total, Hk, r, dtype=dt), unit(total, Hk, r, dtype=dt), normal(total, H, dv, dtype=dt)
        st["alpha"], st["beta"] = gates(total, H)
        st["S0"] = normal(B, H, r, dv, sd=0.3)
        return st
    T = 1 if op == "decode" else case["T"]
    st["q"], st["k"], st["v"] = unit(B, Hk, T, r, dtype=dt), unit(B, Hk, T, r, dtype=dt), normal(B, H, T, dv, dtype=dt)
    st["alpha"], st["beta"] = (x.transpose(1, 2).contiguous() for x in gates(B, T, H))
    if op == "decode":
        st["alpha"], st["beta"] = st["alpha"][:, :, 0].contiguous(), st["beta"][:, :, 0].contiguous()
        st["S"] = normal(B, H, r, dv, sd=0.3)
        return st
    st["S0"] = normal(B, H, r, dv, sd=0.3) if case["state"] else None
    if op == "backward":
        st["dy"] = normal(B, H, T, dv, dtype=dt)
        st["dS_T"] = normal(B, H, r, dv, sd=0.3) if case["state"] else None
    return st


class _Chunks:
    """The chunked form over [B,H,T,*] in 32 bits (T padded with tokens that write nothing).  With G the running sum of
    log alpha inside a chunk and S the state before it:
        E = (I + L)^-1 (V - e^G K S),  L = strictly-lower(e^{Gi-Gj} K K^T) diag(beta),  V' = beta E,
        Y = scale (e^G Q S + A V'),  A = lower(e^{Gi-Gj} Q K^T),   S' = e^{G_last} S + (e^{G_last - G} K)^T V'."""

    def __init__(self, q, k, v, alpha, beta):
        B, H, T, _ = v.shape
        rep = H // q.shape[1]
        q, k = (x.float().repeat_interleave(rep, dim=1) for x in (q, k))
        C = min(_CHUNK, T)
        N = -(-T // C)
        cut = lambda x, fill=0.0: torch.nn.functional.pad(x, (0, 0) * (x.dim() - 3) + (0, N * C - T), value=fill).reshape(  # noqa: E731
            B, H, N, C, *x.shape[3:])
        self.B, self.H, self.T, self.C, self.N = B, H, T, C, N
        self.cut = cut
        self.q, self.k, self.v, self.beta = cut(q), cut(k), cut(v.float()), cut(beta)
        G = torch.cumsum(torch.log(cut(alpha, 1.0).double()), dim=3)  # (64 bits: differences of long sums)
        self.eG, self.eR = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
        i = torch.arange(C, device=v.device)
        d = G[..., :, None] - G[..., None, :]
        self.lower = torch.exp(torch.where(i[:, None] >= i[None], d, -math.inf)).float()
        self.strict = torch.where(i[:, None] > i[None], self.lower, 0.0)
        kt = self.k.transpose(3, 4)
        self.A = (self.q @ kt) * self.lower
        self.L = (self.k @ kt) * self.strict
        Lb = self.L * self.beta[..., None, :]
        X = torch.eye(C, device=v.device).expand(B, H, N, C, C).clone()
        for j in range(1, C):  # forward substitution, a row at a time
            X[..., j, :j] -= (Lb[..., j, None, :j] @ X[..., :j, :j])[..., 0, :]
        self.X = X

    def forward(self, S):
        """(states before each chunk [B,H,N,r,dv], E [B,H,N,C,dv], the state after the last)."""
        XV, XK = self.X @ self.v, self.X @ (self.eG * self.k)
        kd = (self.eR * self.k).transpose(3, 4)
        states, es = [], []
        for n in range(self.N):
            states.append(S)
            E = XV[:, :, n] - XK[:, :, n] @ S
            es.append(E)
            S = self.eG[:, :, n, -1:] * S + kd[:, :, n] @ (self.beta[:, :, n, :, None] * E)
        return torch.stack(states, 2), torch.stack(es, 2), S

    def outputs(self, S, E):
        return self.eG * (self.q @ S) + self.A @ (self.beta[..., None] * E)

    def whole(self, x):
        return x.reshape(self.B, self.H, self.N * self.C, *x.shape[4:])[:, :, : self.T]


def _plain_prefill(q, k, v, alpha, beta, S0, scale):
    B, H, _, dv = v.shape
    c = _Chunks(q, k, v, alpha, beta)
    S0 = torch.zeros((B, H, q.shape[3], dv), device=v.device) if S0 is None else S0
    S, E, S_T = c.forward(S0)
    return scale * c.whole(c.outputs(S, E)), S_T


def _plain_backward(q, k, v, alpha, beta, S0, scale, dy, dS_T):
    B, H, T, dv = v.shape
    Hk, r = q.shape[1], q.shape[3]
    c = _Chunks(q, k, v, alpha, beta)
    zero = torch.zeros((B, H, r, dv), device=v.device)
    S, E, _ = c.forward(zero if S0 is None else S0)
    dY = c.cut(scale * dy.float())
    b = c.beta[..., None]
    # backwards over the chunks: D = dL/dV', N = dL/dR with R = V - e^G K S, and the state's gradient
    Xt, kt = c.X.transpose(3, 4), c.k.transpose(3, 4)
    AtY = c.A.transpose(3, 4) @ dY
    dS, qY = zero if dS_T is None else dS_T, (c.eG * c.q).transpose(3, 4) @ dY
    ds, Ds, Ns = [], [], []
    for n in reversed(range(c.N)):
        ds.append(dS)
        D = AtY[:, :, n] + c.eR[:, :, n] * (c.k[:, :, n] @ dS)
        N = Xt[:, :, n] @ (b[:, :, n] * D)
        Ds.append(D)
        Ns.append(N)
        dS = c.eG[:, :, n, -1:] * dS + qY[:, :, n] - kt[:, :, n] @ (c.eG[:, :, n] * N)
    dSn, D, N = (torch.stack(x[::-1], 2) for x in (ds, Ds, Ns))
    V = b * E
    dA = (dY @ V.transpose(3, 4)) * c.lower
    Z = N @ E.transpose(3, 4)
    dL = -Z * c.strict * c.beta[..., None, :]  # (gradient of K K^T below the diagonal)
    ST = S.transpose(3, 4)
    dq = dA @ c.k + c.eG * (dY @ ST)
    dk = dA.transpose(3, 4) @ c.q + dL @ c.k + dL.transpose(3, 4) @ c.k
    dk = dk - c.eG * (N @ ST) + c.eR * (V @ dSn.transpose(3, 4))
    dbeta = (D * E).sum(4) - (c.L * Z).sum(3)
    # log alpha_t scales what the states from t on hold of the ones before: <S, dS> at the chunk's end, and what the
    # chunk's tokens from t on read and write
    dG = (c.q * dq).sum(4) - (c.v * N).sum(4)
    end = (dSn * torch.cat([S[:, :, 1:], S[:, :, :1] * 0], 2)).sum((3, 4))
    last = c.eG[:, :, -1, -1:] * S[:, :, -1] + (c.eR[:, :, -1] * c.k[:, :, -1]).transpose(2, 3) @ V[:, :, -1]
    end[:, :, -1] = (dSn[:, :, -1] * last).sum((2, 3))
    dlog = end[..., None] + dG.flip(3).cumsum(3).flip(3)
    dlog = c.whole(dlog[..., None])[..., 0]
    dq, dk = (c.whole(x).reshape(B, Hk, H // Hk, T, r).sum(2).to(q.dtype) for x in (dq, dk))
    return dq, dk, c.whole(N).to(v.dtype), dlog / alpha, c.whole(dbeta[..., None])[..., 0], dS


def _plain_score(x, tokens, top):
    """Rows of logits in 32 bits: (log-probability, entropy, log-sum-exp, best log-probabilities, their tokens)."""
    none = tokens < 0
    xf = x.float()
    m = xf.max(dim=1, keepdim=True).values
    e = (xf - m).exp()
    s = e.sum(1)
    lse = m[:, 0] + s.log()
    ent = s.log() - (e * (xf - m)).sum(1) / s
    at = tokens.clamp(min=0).long()[:, None]
    lp = torch.gather(xf, 1, at)[:, 0] - lse
    skip = lambda v: torch.where(none, 0.0, v)  # noqa: E731
    if not top:
        return skip(lp), skip(ent), skip(lse)
    best, where = torch.sort(xf, dim=1, descending=True, stable=True)
    best, where = best[:, :top] - lse[:, None], where[:, :top].int()
    pad = top - best.shape[1]
    best, where = torch.nn.functional.pad(best, (0, pad), value=-math.inf), torch.nn.functional.pad(where, (0, pad), value=-1)
    return skip(lp), skip(ent), skip(lse), torch.where(none[:, None], -math.inf, best), torch.where(none[:, None], -1, where)


def _plain_score_bw(x, tokens, lse, ent, dlp, dent):
    logp = x.float() - lse[:, None]
    p = logp.exp()
    g = -p * (dlp[:, None] + dent[:, None] * (logp + ent[:, None]))
    n = torch.arange(x.shape[0], device=x.device)
    g[n, tokens.clamp(min=0).long()] += dlp
    return torch.where(tokens[:, None] < 0, 0.0, g).to(x.dtype)


def _plain(st):
    op = st["op"]
    if op == "score":
        return _plain_score(st["logits"], st["tokens"], st["top"])
    if op == "score_bw":
        return _plain_score_bw(st["logits"], st["tokens"], st["lse"], st["entropy"], st["dlogprobs"], st["dentropy"])
    q, k, v, alpha, beta, scale = (st[n] for n in ("q", "k", "v", "alpha", "beta", "scale"))
    if op == "decode":
        S, rep = st["S"], st["H"] // st["Hk"]
        qf, kf = (x.float().repeat_interleave(rep, dim=1) for x in (q, k))
        S.mul_(alpha[..., None, None])
        S.add_(kf.transpose(2, 3) @ (beta[..., None, None] * (v.float() - kf @ S)))
        return (scale * (qf @ S)).to(q.dtype), S
    if op == "packed":
        lens = torch.tensor(st["lens"], device="cuda")
        t = torch.arange(max(st["lens"]), device="cuda")
        real = t[None] < lens[:, None]
        at = torch.where(real, st["cu"][:-1, None] + t[None], 0)
        fill = lambda x, f: torch.where(real.reshape(*real.shape, *[1] * (x.dim() - 1)), x[at].float(), f).transpose(1, 2)  # noqa: E731
        y, S_T = _plain_prefill(fill(q, 0.0), fill(k, 0.0), fill(v, 0.0), fill(alpha, 1.0), fill(beta, 0.0), st["S0"], scale)
        return y.transpose(1, 2)[real].to(q.dtype), S_T
    if op == "prefill":
        y, S_T = _plain_prefill(q, k, v, alpha, beta, st["S0"], scale)
        return y.to(q.dtype), S_T
    return _plain_backward(q, k, v, alpha, beta, st["S0"], scale, st["dy"], st["dS_T"])


def run(st):
    if not own:
        return _plain(st)
    import recurrent_state_02_gb300 as la
    op = st["op"]
    if op == "score":
        lp, ent, lse, best, where = la.token_logprobs(st["logits"], st["tokens"], top=st["top"])
        return (lp, ent, lse, best, where) if st["top"] else (lp, ent, lse)
    if op == "score_bw":
        return la.token_logprobs_backward(st["logits"], st["tokens"], st["lse"], st["entropy"], st["dlogprobs"], dentropy=st["dentropy"])
    q, k, v = st["q"], st["k"], st["v"]
    gates = dict(alpha=st["alpha"], beta=st["beta"], scale=st["scale"])
    if op == "decode":
        return la.gated_delta_decode_step(q, k, v, st["S"], **gates), st["S"]
    if op == "packed":
        return la.gated_delta_prefill_varlen(q, k, v, st["cu"], S0=st["S0"], **gates)
    if op == "prefill":
        return la.gated_delta_prefill(q, k, v, S0=st["S0"], **gates)
    return la.gated_delta_backward(q, k, v, st["dy"], S0=st["S0"], dS_T=st["dS_T"], **gates)


def work(case):
    op = case["op"]
    el = 2 if case["dtype"] == "bf16" else 4
    if op == "score":
        n = case["N"] * case["V"]
        return {"bytes": el * n + case["N"] * (16 + 8 * case["top"]), "flops": 6 * n}
    if op == "score_bw":
        n = case["N"] * case["V"]
        return {"bytes": 2 * el * n + 20 * case["N"], "flops": 6 * n}
    B, H, Hk, r, dv = (case[n] for n in ("B", "H", "Hk", "r", "dv"))
    state = 4 * B * H * r * dv
    if op == "decode":
        return {"bytes": 2 * state + B * (el * (2 * Hk * r + 2 * H * dv) + 8 * H), "flops": 8 * B * H * r * dv}
    tokens = sum(_lens(case)) if op == "packed" else B * case["T"]
    if op == "backward":
        return {"bytes": tokens * (el * (4 * Hk * r + 3 * H * dv) + 16 * H) + state * (3 if case["state"] else 1),
                "flops": 22 * tokens * H * r * dv}
    return {"bytes": tokens * (el * (2 * Hk * r + 2 * H * dv) + 8 * H) + state * (2 if op == "packed" or case["state"] else 1),
            "flops": 8 * tokens * H * r * dv}


def _outer(a, b):
    return a[..., :, None] * b[..., None, :]


def _read(S, x):
    return (x[..., None, :] @ S)[..., 0, :]


def _walk(q, k, v, a, b, S):
    """The rule itself in 64 bits, token by token over [B,H,T,*]: (y / scale, errors, S)."""
    y, e = torch.empty_like(v), torch.empty_like(v)
    for t in range(v.shape[2]):
        S = a[:, :, t, None, None] * S
        e[:, :, t] = v[:, :, t] - _read(S, k[:, :, t])
        S = S + _outer(k[:, :, t], b[:, :, t, None] * e[:, :, t])
        y[:, :, t] = _read(S, q[:, :, t])
    return y, e, S


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "score":
        x, tok, top = st["logits"], st["tokens"].long(), case["top"]
        none = tok < 0
        outs = [torch.zeros(case["N"], dtype=torch.float64, device="cuda") for _ in range(3)]
        best = torch.full((case["N"], top), -math.inf, dtype=torch.float64, device="cuda")
        for i in range(0, case["N"], 256):
            s = slice(i, i + 256)
            xd = x[s].double()
            lse = torch.logsumexp(xd, dim=1)
            lp = xd - lse[:, None]
            outs[0][s] = torch.gather(lp, 1, tok[s].clamp(min=0)[:, None])[:, 0]
            outs[1][s] = -(lp.exp() * lp).sum(1)
            outs[2][s] = lse
            n = min(top, case["V"])
            best[s, :n] = torch.topk(lp, n, dim=1).values
        outs = [torch.where(none, 0.0, o) for o in outs]
        return (*outs, torch.where(none[:, None], -math.inf, best), None) if top else tuple(outs)
    if op == "score_bw":
        x, tok = st["logits"], st["tokens"].long()
        out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for i in range(0, case["N"], 256):
            s = slice(i, i + 256)
            xd = x[s].double()
            lp = torch.log_softmax(xd, dim=1)
            p = lp.exp()
            H = -(p * lp).sum(1, keepdim=True)
            w, h = st["dlogprobs"][s, None].double(), st["dentropy"][s, None].double()
            hit = torch.arange(case["V"], device="cuda")[None] == tok[s, None]
            out[s] = torch.where(tok[s, None] < 0, 0.0, w * (hit.double() - p) - h * p * (lp + H))
        return out
    B, H, Hk, r, dv = (case[n] for n in ("B", "H", "Hk", "r", "dv"))
    scale, rep = st["scale"], H // Hk
    if op == "decode":
        wide = lambda x: x.double().repeat_interleave(rep, dim=1)  # noqa: E731
        y, _, S = _walk(wide(st["q"]), wide(st["k"]), st["v"].double(), st["alpha"].double()[..., None],
                        st["beta"].double()[..., None], st["S"].double())
        return scale * y, S
    if op == "packed":
        lens, cu = st["lens"], st["cu"].tolist()
        wide = lambda x: x.double().repeat_interleave(rep, dim=1)  # noqa: E731
        y = torch.zeros((cu[-1], H, dv), dtype=torch.float64, device="cuda")
        order = sorted(range(B), key=lambda b: -lens[b])
        S = st["S0"].double()[order]
        start = torch.tensor([cu[b] for b in order], device="cuda")
        for t in range(max(lens)):
            n = sum(x > t for x in lens)  # the sequences that have a token t come first
            at = start[:n] + t
            k, b = wide(st["k"][at]), st["beta"][at].double()
            P = st["alpha"][at].double()[..., None, None] * S[:n]
            S[:n] = P + _outer(k, b[..., None] * (st["v"][at].double() - _read(P, k)))
            y[at] = _read(S[:n], wide(st["q"][at]))
        out = torch.empty_like(S)
        out[order] = S
        return scale * y, out
    q, k = (st[n].double().repeat_interleave(rep, dim=1) for n in ("q", "k"))
    v, a, b = (st[n].double() for n in ("v", "alpha", "beta"))
    zero = torch.zeros((B, H, r, dv), dtype=torch.float64, device="cuda")
    S0 = zero if st["S0"] is None else st["S0"].double()
    y, e, S_T = _walk(q, k, v, a, b, S0)
    if op == "prefill":
        return scale * y, S_T
    dy = scale * st["dy"].double()
    dS_T = zero if st["dS_T"] is None else st["dS_T"].double()
    T = case["T"]
    # the chain rule, token by token: G is the gradient of S_t
    G, lam, dk = dS_T, torch.empty_like(v), torch.empty_like(k)
    for t in reversed(range(T)):
        G = G + _outer(q[:, :, t], dy[:, :, t])
        lam[:, :, t] = _read(G, k[:, :, t])
        dk[:, :, t] = b[:, :, t, None] * _read(G.transpose(2, 3), e[:, :, t])
        G = a[:, :, t, None, None] * (G - _outer(k[:, :, t], b[:, :, t, None] * lam[:, :, t]))
    dvv = b[..., None] * lam
    S, dq = S0, torch.empty_like(q)
    for t in range(T):
        S = a[:, :, t, None, None] * S
        dk[:, :, t] -= _read(S.transpose(2, 3), dvv[:, :, t])
        S = S + _outer(k[:, :, t], b[:, :, t, None] * e[:, :, t])
        dq[:, :, t] = _read(S.transpose(2, 3), dy[:, :, t])
    dlog = (y * dy).sum(3) - (v * dvv).sum(3)
    dlog = (S_T * dS_T).sum((2, 3))[..., None] + dlog.flip(2).cumsum(2).flip(2)
    dq, dk = (x.reshape(B, Hk, rep, T, r).sum(2) for x in (dq, dk))
    return dq, dk, dvv, dlog / a, (lam * e).sum(3), G
