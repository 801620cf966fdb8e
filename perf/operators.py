"""What the decayed linear attention, the beam selection and the state reordering are measured on.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes a case's inputs on the
GPU from a seed, ``run()`` is one pass through an operator (the framework's where ``own`` is true, else the same
mathematics in elementary torch operations), ``work()`` is what a pass cannot do without, and ``exact()`` is the
operator's definition in 64 bits.

    prefill   S_t = g S_{t-1} + k_t v_t^T,  y_t = scale q_t^T S_t        (g: the head's decay)
    packed    the same over sequences of different lengths packed one after another
    decode    one token of it, the state updated in place
    backward  gradients of prefill: dq, dk, dv, dS0 from dy, dS_T
    select    the best K of K beams x V tokens by score + log-probability
    reorder   state j of a request becomes the state of its parent beam, in place
"""
import math
import random

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CHUNK = 128  # tokens per chunk of the plain form


def listed():
    return [
        # a training or scoring batch: the framework's headline prefill shape
        dict(name="prefill_b4_h16_t4096", op="prefill", dtype="bf16", B=4, H=16, T=4096, r=128, dv=128, state=False),
        # one very long prompt: the framework's long prefill
        dict(name="prefill_b1_h32_t65536", op="prefill", dtype="bf16", B=1, H=32, T=65536, r=128, dv=128, state=False),
        # a serving batch of ragged prompts, each from its own carried state
        dict(name="packed_48_prompts_h16", op="packed", dtype="bf16", B=48, H=16, lo=128, hi=8192, mix=8, r=128, dv=128),
        # a small exact run with odd sizes (FP32 through and through)
        dict(name="prefill_fp32_t1001", op="prefill", dtype="fp32", B=2, H=4, T=1001, r=64, dv=96, state=True),
        # a serving batch's decode step: bound by the state's traffic
        dict(name="decode_b256_h16", op="decode", dtype="bf16", B=256, H=16, r=128, dv=128),
        # one request's decode step: bound by latency
        dict(name="decode_b1_h16", op="decode", dtype="bf16", B=1, H=16, r=128, dv=128),
        # the gradients of the training batch
        dict(name="backward_b4_h16_t4096", op="backward", dtype="bf16", B=4, H=16, T=4096, r=128, dv=128, state=False),
        # gradients of a short ragged sequence through a carried state, narrow keys
        dict(name="backward_b1_h8_t777", op="backward", dtype="bf16", B=1, H=8, T=777, r=64, dv=128, state=True),
        # a serving batch's beam step over a large vocabulary
        dict(name="select_b64_k4_v131072", op="select", dtype="bf16", B=64, K=4, V=131072),
        # one request's beam step over an odd vocabulary
        dict(name="select_b1_k5_v32003", op="select", dtype="fp32", B=1, K=5, V=32003),
        # the states of that serving batch's beams, with their normalisers
        dict(name="reorder_b64_k4_h16", op="reorder", B=64, K=4, H=16, r=128, dv=128, norm=True),
        # one request's few states
        dict(name="reorder_b1_k4_h8", op="reorder", B=1, K=4, H=8, r=64, dv=64, norm=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "packed", "decode", "backward", "select", "reorder"])
    if op == "select":
        c = dict(op=op, dtype=rng.choice(["bf16", "fp32"]), B=_log(rng, 1, 64), K=rng.randint(1, 12), V=_log(rng, 100, 150000))
        while c["B"] * c["K"] * c["V"] > 33_000_000:
            c["B"] = max(1, c["B"] // 2)
        return c
    if op == "reorder":
        c = dict(op=op, B=_log(rng, 1, 64), K=rng.randint(2, 10), H=_log(rng, 1, 32), r=rng.choice([33, 64, 96, 128]),
                 dv=rng.choice([64, 80, 128]), norm=rng.random() < 0.5)
        while c["B"] * c["K"] * c["H"] > 4096:
            c["B"] = max(1, c["B"] // 2)
        return c
    if op == "decode":
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), B=_log(rng, 1, 256), H=_log(rng, 1, 32),
                 r=rng.choice([64, 96, 128, 128]), dv=rng.choice([64, 80, 128, 128]))
        while c["B"] * c["H"] > 4096:
            c["B"] = max(1, c["B"] // 2)
        return c
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    sizes = [64, 128, 128] if dtype == "bf16" else [32, 64, 96, 128]
    c = dict(op=op, dtype=dtype, B=_log(rng, 1, 16), H=_log(rng, 1, 32), r=rng.choice(sizes), dv=rng.choice(sizes))
    most = 262144 if dtype == "bf16" else 32768  # tokens x heads
    if op == "packed":
        c.update(dtype="bf16", r=rng.choice([64, 128, 128]), dv=rng.choice([64, 128, 128]), lo=1, hi=_log(rng, 16, 4096),
                 mix=rng.randrange(1000), B=_log(rng, 1, 64))
        while c["B"] * c["H"] * c["hi"] > 2 * 262144:
            c["hi"] = max(16, c["hi"] // 2)
            c["H"] = max(1, c["H"] // 2)
        return c
    c.update(T=_log(rng, 1, 16384), state=rng.random() < 0.5)
    while c["B"] * c["H"] * c["T"] > most:
        k = "B" if c["B"] > 1 else "H" if c["H"] > 1 else "T"
        c[k] = max(1, c[k] // 2)
    return c


def _lens(case):
    """The lengths of a packed case: log-uniform in lo..hi, fixed by the case."""
    rng = random.Random(case["mix"])
    return [_log(rng, case["lo"], case["hi"]) for _ in range(case["B"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sd=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * sd).to(dtype)

    op, st = case["op"], dict(case)
    if op == "select":
        B, K, V = case["B"], case["K"], case["V"]
        # logits of a trained model's spread; cumulative scores of a few tokens; one finished beam in sixteen
        st["logits"] = normal(B, K, V, sd=3.0, dtype=_DTYPE[case["dtype"]])
        st["scores"] = -4.0 - 2.0 * torch.rand((B, K), generator=g, device="cuda")
        st["done"] = (torch.rand((B, K), generator=g, device="cuda") < 1 / 16).to(torch.uint8)
        st["eos"] = 2
        return st
    if op == "reorder":
        B, K, H, r, dv = (case[n] for n in ("B", "K", "H", "r", "dv"))
        st["S"] = normal(B * K, H, r, dv)
        st["z"] = torch.rand((B * K, H, r), generator=g, device="cuda") * 99 + 1 if case["norm"] else None
        st["parents"] = torch.randint(0, K, (B, K), generator=g, device="cuda", dtype=torch.int32)
        return st
    dt, H, r, dv = _DTYPE[case["dtype"]], case["H"], case["r"], case["dv"]
    B = case["B"]
    # a head's memory reaches from two tokens to a thousand: -log(decay) log-uniform in 2^-10 .. 0.7
    u = torch.rand(H, generator=g, device="cuda", dtype=torch.float64)
    st["decay"] = torch.exp(-torch.exp(u * math.log(0.7 * 1024)) / 1024).float()
    st["scale"] = r ** -0.5
    if op == "decode":
        st["q"], st["k"], st["v"] = normal(B, H, 1, r, dtype=dt), normal(B, H, 1, r, dtype=dt), normal(B, H, 1, dv, dtype=dt)
        st["S"] = normal(B, H, r, dv)
        return st
    if op == "packed":
        lens = _lens(case)
        total = sum(lens)
        st["lens"] = lens
        st["cu"] = torch.tensor([0] + [sum(lens[: i + 1]) for i in range(B)], dtype=torch.int32, device="cuda")
        st["q"], st["k"], st["v"] = normal(total, H, r, dtype=dt), normal(total, H, r, dtype=dt), normal(total, H, dv, dtype=dt)
        st["S0"] = normal(B, H, r, dv)
        return st
    T = case["T"]
    st["q"], st["k"], st["v"] = normal(B, H, T, r, dtype=dt), normal(B, H, T, r, dtype=dt), normal(B, H, T, dv, dtype=dt)
    st["S0"] = normal(B, H, r, dv) if case["state"] else None
    if op == "backward":
        st["dy"] = normal(B, H, T, dv, dtype=dt)
        st["dS_T"] = normal(B, H, r, dv) if case["state"] else None
    return st


def _powers(decay, n):
    """decay[h] ** n for whole n >= 0 (0 ** 0 = 1), formed in 64 bits: [H, *n.shape] in 32."""
    return (decay.double().reshape(-1, *([1] * n.dim())) ** n.double()).float()


def _sweep(q, k, v, decay, S0, off, lens=None):
    """Causal products in chunks over [B,H,T,*]: y_t = q_t^T (decay^{t+off} S0 + sum_{j<=t} decay^{t-j} k_j v_j^T), and
    the state that the last token hands on, decay^T S0 + sum_j decay^{T-off-j} k_j v_j^T.  lens: [B] lengths (the
    rows past them are zero)."""
    q, k, v = q.float(), k.float(), v.float()
    B, H, T, r = q.shape
    dv = v.shape[3]
    dev = q.device
    t = torch.arange(T, device=dev)
    n_tok = torch.full((B,), T, device=dev) if lens is None else lens
    left = n_tok[:, None] - off - t[None]  # steps from token t's write to the final state
    w = torch.where(left >= 0, _powers(decay, left.clamp(min=0)), torch.zeros((), device=dev)).permute(1, 0, 2)  # [B,H,T]
    S_T = (k * w[..., None]).transpose(2, 3) @ v
    if S0 is not None:
        S_T = S_T + _powers(decay, n_tok).t()[:, :, None, None] * S0
    C = min(_CHUNK, max(1, T))
    N = -(-T // C)
    pad = N * C - T
    qc, kc, vc = (torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(B, H, N, C, x.shape[3]) for x in (q, k, v))
    i = torch.arange(C, device=dev)
    d = i[:, None] - i[None]
    D = torch.where(d >= 0, _powers(decay, d.clamp(min=0)), torch.zeros((), device=dev))  # [H,C,C]
    y = ((qc @ kc.transpose(3, 4)) * D[None, :, None]) @ vc
    if N > 1 or S0 is not None:
        # the state before chunk n, to be read with decay^{i+off}: its distance to a write at j of chunk m is (n-m)C - j - off
        dS = (kc * _powers(decay, C - off - i)[None, :, None, :, None]).transpose(3, 4) @ vc  # [B,H,N,r,dv]
        m = torch.arange(N, device=dev)
        e = (m[:, None] - 1 - m[None]) * C
        M = torch.where(e >= 0, _powers(decay, e.clamp(min=0)), torch.zeros((), device=dev))  # [H,N,N]
        S = (M[None] @ dS.reshape(B, H, N, r * dv)).reshape(B, H, N, r, dv)
        if S0 is not None:
            S = S + _powers(decay, m * C)[None, :, :, None, None] * S0[:, :, None]
        y = y + (qc * _powers(decay, i + off)[None, :, None, :, None]) @ S
    return y.reshape(B, H, N * C, dv)[:, :, :T], S_T


def _plain_select(logits, scores, done, eos):
    """In 64 bits: candidates of nearly the same score decide which tokens are chosen."""
    x = logits.double()
    B, K, V = x.shape
    m = x.max(dim=2, keepdim=True).values
    lse = m + (x - m).exp().sum(dim=2, keepdim=True).log()
    low = torch.tensor(-math.inf, device=x.device, dtype=torch.float64)
    cand = torch.where(lse.isfinite(), scores.double()[..., None] + x - lse, low)
    token = torch.arange(V, device=x.device)
    only = torch.where(token == eos, scores.double()[..., None], low)  # a finished beam stays as it is
    cand = torch.where(done[..., None] != 0, only, cand).reshape(B, K * V)
    best, at = torch.sort(cand, dim=1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    empty = best == low  # fewer than K candidates: the slot keeps its own beam
    slot = torch.arange(K, device=x.device).expand(B, K)
    parents = torch.where(empty, slot, at // V)
    tokens = torch.where(empty, torch.zeros_like(at), at % V)
    ended = (torch.gather(done, 1, parents) != 0) | (~empty & (tokens == eos))
    return best.float(), parents.int(), tokens.int(), ended.to(torch.uint8)


def _plain(st):
    op = st["op"]
    if op == "select":
        return _plain_select(st["logits"], st["scores"], st["done"], st["eos"])
    if op == "reorder":
        B, K = st["parents"].shape
        at = (torch.arange(B, device="cuda")[:, None] * K + st["parents"]).reshape(-1)
        st["S"].copy_(st["S"][at])
        if st["z"] is not None:
            st["z"].copy_(st["z"][at])
        return st["S"], st["z"]
    q, k, v, decay, scale = st["q"], st["k"], st["v"], st["decay"], st["scale"]
    if op == "decode":
        S = st["S"]
        S.copy_(decay[None, :, None, None] * S + k.float().transpose(2, 3) @ v.float())
        return (scale * (q.float() @ S)).to(q.dtype), S
    if op == "packed":
        lens = torch.tensor(st["lens"], device="cuda")
        t = torch.arange(max(st["lens"]), device="cuda")
        real = t[None] < lens[:, None]
        at = torch.where(real, st["cu"][:-1, None] + t[None], 0)
        wide = [torch.where(real[..., None, None], x[at].float(), 0.0).transpose(1, 2) for x in (q, k, v)]
        y, S_T = _sweep(*wide, decay, st["S0"], 1, lens)
        return (scale * y.transpose(1, 2)[real]).to(q.dtype), S_T
    if op == "prefill":
        y, S_T = _sweep(q, k, v, decay, st["S0"], 1)
        return (scale * y).to(q.dtype), S_T
    dy = st["dy"]
    turned = lambda x: None if x is None else x.transpose(2, 3)  # noqa: E731
    back = lambda *xs: [x.flip(2) for x in xs]  # noqa: E731
    dq, _ = _sweep(dy, v, k, decay, turned(st["S0"]), 1)
    # backwards in time the state that enters is dS_T, read without a decay by the last token
    rq, rk, rv, rdy = back(scale * q.float(), k, v, dy)
    dk, _ = _sweep(rv, rdy, rq, decay, turned(st["dS_T"]), 0)
    dvv, dS0 = _sweep(rk, rq, rdy, decay, st["dS_T"], 0)
    return (scale * dq).to(q.dtype), dk.flip(2).to(q.dtype), dvv.flip(2).to(q.dtype), dS0


def run(st):
    if not own:
        return _plain(st)
    import recurrent_state_02_gb300 as la
    op = st["op"]
    if op == "select":
        return la.beam_select(st["logits"], st["scores"], done=st["done"], eos=st["eos"])
    if op == "reorder":
        return la.state_reorder(st["S"], st["parents"], z=st["z"])
    if op == "decode":
        return la.decay_decode_step(st["q"], st["k"], st["v"], st["decay"], st["S"], scale=st["scale"]), st["S"]
    if op == "packed":
        return la.decay_prefill_varlen(st["q"], st["k"], st["v"], st["decay"], st["cu"], S0=st["S0"], scale=st["scale"])
    if op == "prefill":
        return la.decay_prefill(st["q"], st["k"], st["v"], st["decay"], S0=st["S0"], scale=st["scale"])
    return la.decay_backward(st["q"], st["k"], st["v"], st["dy"], st["decay"], S0=st["S0"], dS_T=st["dS_T"], scale=st["scale"])


def work(case):
    op = case["op"]
    el = 2 if case.get("dtype") == "bf16" else 4
    if op == "select":
        n = case["B"] * case["K"] * case["V"]
        return {"bytes": el * n + 18 * case["B"] * case["K"], "flops": 4 * n}
    if op == "reorder":
        K = case["K"]
        slot = 4 * case["H"] * case["r"] * (case["dv"] + (1 if case["norm"] else 0))
        # parents drawn uniformly: a slot moves with probability 1 - 1/K, and a state is read by another
        # slot with probability 1 - (1 - 1/K)^(K-1)
        return {"bytes": case["B"] * K * slot * ((1 - 1 / K) + (1 - (1 - 1 / K) ** (K - 1))) + 4 * case["B"] * K, "flops": 0}
    heads, r, dv = case["B"] * case["H"], case["r"], case["dv"]
    state = 4 * heads * r * dv
    if op == "decode":
        return {"bytes": 2 * state + el * heads * 2 * (r + dv), "flops": 5 * heads * r * dv}
    tokens = case["H"] * sum(_lens(case)) if op == "packed" else heads * case["T"]
    if op == "backward":
        return {"bytes": el * tokens * (4 * r + 3 * dv) + state * (3 if case["state"] else 1), "flops": 10 * tokens * r * dv}
    return {"bytes": el * tokens * 2 * (r + dv) + state * (2 if op == "packed" or case["state"] else 1), "flops": 4 * tokens * r * dv}


def _recur(a, b, c, decay, S, first):
    """The recurrence itself in 64 bits, token by token: S <- decay S + b_t c_t^T (the first token's S is taken as it is
    unless `first`), out_t = a_t^T S.  a, b [B,H,T,r], c [B,H,T,dv]."""
    g = decay.double()[None, :, None, None]
    outs = torch.empty(c.shape, dtype=torch.float64, device=c.device)
    for t in range(a.shape[2]):
        if t > 0 or first:
            S = g * S
        S = torch.addcmul(S, b[:, :, t, :, None].double(), c[:, :, t, None, :].double())
        outs[:, :, t] = torch.matmul(a[:, :, t, None, :].double(), S)[:, :, 0]
    return outs, S


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "select":
        nxt = []
        for b in range(case["B"]):
            found = []
            for k in range(case["K"]):
                s, x = float(st["scores"][b, k]), st["logits"][b, k].double()
                if st["done"][b, k]:
                    found.append(s)
                else:
                    top = torch.topk(x, min(case["K"], x.numel())).values
                    found += (s + top - torch.logsumexp(x, 0)).tolist()
            nxt.append(sorted(found, reverse=True)[: case["K"]])
        if any(len(row) < case["K"] for row in nxt):
            nxt = [row + [-math.inf] * (case["K"] - len(row)) for row in nxt]
        return torch.tensor(nxt, dtype=torch.float64), None, None, None
    if op == "reorder":
        S, z = st["S"].double(), None if st["z"] is None else st["z"].double()
        T, w = S.clone(), None if z is None else z.clone()
        for b, row in enumerate(st["parents"].tolist()):
            for j, p in enumerate(row):
                T[b * case["K"] + j] = S[b * case["K"] + p]
                if z is not None:
                    w[b * case["K"] + j] = z[b * case["K"] + p]
        return T, w
    decay, scale = st["decay"], st["scale"]
    B, H, r, dv = case["B"], case["H"], case["r"], case["dv"]
    zero = torch.zeros((B, H, r, dv), dtype=torch.float64, device="cuda")
    if op == "decode":
        y, S = _recur(st["q"], st["k"], st["v"], decay, st["S"].double(), True)
        return scale * y, S
    if op == "packed":
        lens, cu = st["lens"], st["cu"].tolist()
        S, y = st["S0"].double(), torch.zeros((cu[-1], H, dv), dtype=torch.float64, device="cuda")
        g = decay.double()[None, :, None, None]
        order = sorted(range(B), key=lambda b: -lens[b])
        S = S[order]
        start = torch.tensor([cu[b] for b in order], device="cuda")
        for t in range(max(lens)):
            n = sum(x > t for x in lens)  # the sequences that have a token t come first
            at = start[:n] + t
            S[:n] = torch.addcmul(g * S[:n], st["k"][at][..., None].double(), st["v"][at][..., None, :].double())
            y[at] = torch.matmul(st["q"][at][..., None, :].double(), S[:n])[:, :, 0]
        out = torch.empty_like(S)
        out[order] = S
        return scale * y, out
    S0 = zero if st["S0"] is None else st["S0"].double()
    if op == "prefill":
        y, S = _recur(st["q"], st["k"], st["v"], decay, S0, True)
        return scale * y, S
    dS_T = zero if st["dS_T"] is None else st["dS_T"].double()
    q, k, v, dy = (st[n].double() for n in ("q", "k", "v", "dy"))
    dq, _ = _recur(dy, v, k, decay, S0.transpose(2, 3), True)
    dk, _ = _recur(v.flip(2), dy.flip(2), scale * q.flip(2), decay, dS_T.transpose(2, 3), False)
    dvv, G = _recur(k.flip(2), scale * q.flip(2), dy.flip(2), decay, dS_T, False)
    return scale * dq, dk.flip(2), dvv.flip(2), decay.double()[None, :, None, None] * G
