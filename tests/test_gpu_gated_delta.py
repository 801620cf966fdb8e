"""The gated delta rule on the GPU (la_gated_delta_*) against its 64-bit recurrence, one token at a time; the bounds are
derived in gdelta_reference."""
import pytest
import torch

import gdelta_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    from recurrent_state_02_gb300 import build
    build.build()
    import recurrent_state_02_gb300 as la_mod
    assert torch.cuda.is_available()
    return la_mod


GATES = [1.0, 0.5, 0.99609375, 0.3, 0.9, 1.0 - 2.0 ** -20, 0.97, 0.999]


def make(B, H, Hk, T, r, dv, dtype, state, seed, layout="bh"):
    g = torch.Generator().manual_seed(seed)
    shape = (lambda h, d: (B, h, T, d)) if layout == "bh" else (lambda h, d: (T, h, d))
    q, k = (torch.randn(shape(Hk, r), generator=g) for _ in range(2))
    q, k = ((x / x.norm(dim=-1, keepdim=True)).to(dtype).cuda() for x in (q, k))
    v, dy = (torch.randn(shape(H, dv), generator=g).to(dtype).cuda() for _ in range(2))
    S0, dS_T = (torch.randn((B, H, r, dv), generator=g).mul(0.3).cuda() if state else None for _ in range(2))
    base = torch.tensor([GATES[(h + seed) % len(GATES)] for h in range(H)])
    base = base[None, :, None].expand(B, H, T) if layout == "bh" else base[None].expand(T, H)
    alpha = base ** (0.5 + torch.rand(base.shape, generator=g))
    beta = torch.sigmoid(torch.randn(base.shape, generator=g))
    return q, k, v, dy, alpha.contiguous().cuda(), beta.cuda(), S0, dS_T


SIZES = [
    # B, H, Hk, T, r, dv
    (1, 1, 1, 1, 128, 128), (2, 4, 2, 2, 64, 64), (1, 4, 4, 16, 128, 128), (1, 4, 2, 17, 128, 128), (1, 4, 1, 33, 128, 128),
    (1, 2, 2, 63, 128, 128), (2, 2, 1, 64, 128, 128), (1, 3, 3, 65, 128, 128), (1, 2, 2, 128, 128, 64), (1, 2, 2, 200, 128, 192),
    (1, 2, 2, 300, 128, 256), (1, 2, 2, 130, 64, 128), (1, 2, 1, 129, 64, 64), (1, 2, 2, 500, 128, 128), (2, 6, 2, 37, 33, 7),
    (1, 1, 1, 50, 256, 160), (1, 2, 1, 19, 1, 1), (1, 1, 1, 70, 96, 80), (1, 2, 2, 40, 128, 100), (1, 1, 1, 40, 20, 256),
]
ids = lambda s: "x".join(map(str, s))  # noqa: E731
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


@DTYPES
@pytest.mark.parametrize("state", [False, True], ids=["zero", "S0"])
@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_prefill_parity(la, size, state, dtype):
    q, k, v, _, alpha, beta, S0, _ = make(*size, dtype, state, seed=sum(size))
    scale = size[4] ** -0.5
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0, scale=scale)
    assert la.last_device_status() == 0
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, scale)
    R.check(S, ref_S, dtype, "S", q.shape[2])
    R.check(y, ref_y, dtype, "y", q.shape[2])


@DTYPES
@pytest.mark.parametrize("T", [1, 70])
def test_gates_left_out(la, T, dtype):
    """alpha None and beta None are ones, together the ungated rule."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(1, 2, 2, T, 128, 128, dtype, True, 3)
    for a, b in ((None, beta), (alpha, None), (None, None)):
        y, S = la.gated_delta_prefill(q, k, v, a, b, S0=S0, scale=0.1)
        ref_y, ref_S, _, _ = R.prefill(q, k, v, a, b, S0, 0.1)
        R.check(S, ref_S, dtype, "S", q.shape[2])
        R.check(y, ref_y, dtype, "y", q.shape[2])
        got = la.gated_delta_backward(q, k, v, dy, a, b, S0=S0, dS_T=dS_T, scale=0.1)
        ref = R.backward(q, k, v, dy, a, b, S0, dS_T, 0.1)
        assert (got[3] is None) == (a is None) and (got[4] is None) == (b is None)
        R.check_all(got, ref, dtype, T)
    if dtype == torch.float32:
        y, S = la.gated_delta_prefill(q, k, v, S0=S0)
        y2, S2 = la.delta_rule(q, k, v, None, S0=S0)
        assert torch.allclose(y, y2, rtol=1e-4, atol=1e-5) and torch.allclose(S, S2, rtol=1e-4, atol=1e-5)


@DTYPES
def test_zero_gates(la, dtype):
    """alpha = 0 forgets everything before; beta = 0 writes nothing.  Their gradients too (dalpha is 0 where alpha is)."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(2, 2, 2, 150, 128, 128, dtype, True, 5)
    alpha[:, :, 40], alpha[:, 1, 99:101], alpha[1, 0, 0], alpha[0, 0, 64] = 0.0, 0.0, 0.0, 0.0
    beta[:, :, 10:14], beta[0, 1, 100:], beta[1, 1, 64] = 0.0, 0.0, 1.0
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0)
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, 1.0)
    R.check(S, ref_S, dtype, "S", q.shape[2])
    R.check(y, ref_y, dtype, "y", q.shape[2])
    got = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T)
    assert la.last_device_status() == 0
    ref, terms = R.backward(q, k, v, dy, alpha, beta, S0, dS_T, 1.0)
    assert not got[3][alpha == 0].any()
    zero = alpha.cpu() == 0
    ref[3][zero], terms[3][zero] = 0.0, 0.0
    R.check_all(got, (ref, terms), dtype, 150)


@DTYPES
def test_tiny_gates(la, dtype):
    """Gates down to the smallest numbers forget like zeros, and spoil nothing around them."""
    q, k, v, _, alpha, beta, S0, _ = make(1, 2, 2, 150, 128, 128, dtype, True, 6)
    alpha[:, 0, ::7], alpha[:, 1, 20:90], alpha[0, 0, 3] = 1e-30, 1e-3, 1e-42
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0)
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, 1.0)
    R.check(S, ref_S, dtype, "S", q.shape[2])
    R.check(y, ref_y, dtype, "y", q.shape[2])


@DTYPES
@pytest.mark.parametrize("same", ["key", "pair"])
def test_repeated_keys(la, same, dtype):
    """One key for all tokens (the memory overwrites a single row) or two in turn: the in-chunk system at its worst."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(1, 2, 2, 200, 128, 128, dtype, True, 7)
    k = k[:, :, :1].expand_as(k).contiguous() if same == "key" else k[:, :, :2].repeat(1, 1, 100, 1).contiguous()
    beta[:, 1] = 1.0
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0)
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, 1.0)
    R.check(S, ref_S, dtype, "S", q.shape[2])
    R.check(y, ref_y, dtype, "y", q.shape[2])
    got = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T)
    R.check_all(got, R.backward(q, k, v, dy, alpha, beta, S0, dS_T, 1.0), dtype, 200)


@DTYPES
def test_no_tokens(la, dtype):
    q, k, v, dy, alpha, beta, S0, dS_T = make(2, 4, 2, 0, 128, 64, dtype, True, 1)
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0)
    assert y.numel() == 0 and torch.equal(S, S0)
    assert not la.gated_delta_prefill(q, k, v)[1].any()
    assert torch.equal(la.gated_delta_backward(q, k, v, dy, alpha, beta, dS_T=dS_T)[5], dS_T)
    assert not la.gated_delta_backward(q, k, v, dy, alpha, beta)[5].any()


def off(t):
    """The same values one element off a 16-byte boundary."""
    buf = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)
    buf[1:].copy_(t.reshape(-1))
    return buf[1:].view(t.shape)


@DTYPES
@pytest.mark.parametrize("T", [5, 150])
def test_in_place_and_misaligned(la, T, dtype):
    q, k, v, dy, alpha, beta, S0, dS_T = make(1, 2, 1, T, 128, 128, dtype, True, 2)
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0, scale=0.1)
    S2 = S0.clone()
    y2, _ = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S2, scale=0.1, S_out=S2)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    S3, y3 = off(S0), off(y)
    la.gated_delta_prefill(off(q), off(k), off(v), off(alpha), off(beta), S0=S3, scale=0.1, y=y3, S_out=S3)
    assert la.last_device_status() == 0
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, 0.1)
    R.check(S3, ref_S, dtype, "S", T)
    R.check(y3, ref_y, dtype, "y", T)
    got = la.gated_delta_backward(off(q), off(k), off(v), off(dy), off(alpha), off(beta), S0=off(S0), dS_T=off(dS_T), scale=0.1)
    R.check_all(got, R.backward(q, k, v, dy, alpha, beta, S0, dS_T, 0.1), dtype, T)


@DTYPES
@pytest.mark.parametrize("split", [1, 64, 100, 130])
def test_continues(la, split, dtype):
    """Two calls chained through the state agree with one."""
    q, k, v, _, alpha, beta, S0, _ = make(1, 2, 2, 200, 128, 128, dtype, True, 3)
    cut = lambda x, a, b: x[:, :, a:b].contiguous()  # noqa: E731
    _, S1 = la.gated_delta_prefill(*(cut(x, 0, split) for x in (q, k, v, alpha, beta)), S0=S0)
    y2, S2 = la.gated_delta_prefill(*(cut(x, split, 200) for x in (q, k, v, alpha, beta)), S0=S1)
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, 1.0)
    R.check(S2, ref_S, dtype, "S", 200)
    R.check(y2, ref_y[:, :, split:], dtype, "y", 200)


PACKS = [[5, 0, 64, 1, 63, 130, 2], [200], [1, 1, 1], [0, 0], [65, 64, 128, 17, 16, 15], [3, 300, 0, 77]]


@DTYPES
@pytest.mark.parametrize("r,dv", [(128, 128), (64, 192), (40, 24)], ids=["128x128", "64x192", "40x24"])
@pytest.mark.parametrize("lens", PACKS, ids=lambda s: "_".join(map(str, s)))
def test_packed(la, lens, r, dv, dtype):
    """Every sequence is its own prefill; rows outside them stay, and what they hold reaches nothing (NaN)."""
    lead, B, H, Hk = 3, len(lens), 4, 2
    total = lead + sum(lens) + 5
    q, k, v, _, alpha, beta, _, _ = make(B, H, Hk, total, r, dv, dtype, False, 11, layout="tok")
    S0 = torch.randn((B, H, r, dv), generator=torch.Generator().manual_seed(1)).mul(0.3).cuda()
    cu = torch.tensor([lead + sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    outside = torch.ones(total, dtype=torch.bool)
    outside[lead:lead + sum(lens)] = False
    for x in (q, k, v, alpha, beta):
        x[outside.cuda()] = float("nan")
    y = torch.full((total, H, dv), 7.0, device="cuda", dtype=dtype)
    S_in = S0.clone()
    y, S = la.gated_delta_prefill_varlen(q, k, v, cu, alpha, beta, S0=S_in, scale=0.3, y=y, S_out=S_in)
    assert la.last_device_status() == 0
    assert (y[outside.cuda()] == 7.0).all()
    bh = lambda x, s: x[s].transpose(0, 1)[None]  # noqa: E731
    for b, n in enumerate(lens):
        s = slice(int(cu[b]), int(cu[b]) + n)
        ref_y, ref_S, _, _ = R.prefill(*(bh(x, s) for x in (q, k, v, alpha, beta)), S0[b:b + 1], 0.3)
        R.check(S[b:b + 1], ref_S, dtype, f"S {b}", n)
        R.check(bh(y, s), ref_y, dtype, f"y {b}", n)


def test_packed_neighbours_are_not_read(la):
    """A NaN in one sequence stays there, although its neighbours' last chunks reach over it."""
    lens = [70, 30, 100, 10]
    q, k, v, _, alpha, beta, _, _ = make(4, 2, 2, sum(lens), 128, 128, torch.bfloat16, False, 12, layout="tok")
    cu = torch.tensor([0, 70, 100, 200, 210], dtype=torch.int32, device="cuda")
    want_y, want_S = la.gated_delta_prefill_varlen(q, k, v, cu, alpha, beta)
    for x in (q, k, v, alpha, beta):
        x[70:100] = float("nan")
    y, S = la.gated_delta_prefill_varlen(q, k, v, cu, alpha, beta)
    keep = [0, 2, 3]
    assert torch.equal(S[keep], want_S[keep])
    assert torch.equal(y[:70], want_y[:70]) and torch.equal(y[100:], want_y[100:])


def test_packed_many_sequences(la):
    """More sequences than the plan takes at a time, and more of them times all tokens than 2^30."""
    g = torch.Generator().manual_seed(21)
    B, H, Hk, r, dv = 3000, 8, 4, 64, 64
    lens = torch.randint(0, 31, (B,), generator=g)
    lens[[5, 1500, 2999]] = torch.tensor([700, 130, 65])
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), lens.cumsum(0)))
    total = int(cu[-1])
    assert B * H * total > 1 << 30
    q, k, v, _, alpha, beta, _, _ = make(1, H, Hk, total, r, dv, torch.bfloat16, False, 22, layout="tok")
    S0 = torch.randn((B, H, r, dv), generator=g).mul(0.3).cuda()
    y, S = la.gated_delta_prefill_varlen(q, k, v, cu.int().cuda(), alpha, beta, S0=S0, scale=0.2)
    assert la.last_device_status() == 0
    bh = lambda x, s: x[s].transpose(0, 1)[None]  # noqa: E731
    for b in [0, 1, 5, 1023, 1024, 1500, 2047, 2048, 2998, 2999]:
        s = slice(int(cu[b]), int(cu[b + 1]))
        ref_y, ref_S, _, _ = R.prefill(*(bh(x, s) for x in (q, k, v, alpha, beta)), S0[b:b + 1], 0.2)
        R.check(S[b:b + 1], ref_S, torch.bfloat16, f"S {b}", int(lens[b]))
        R.check(bh(y, s), ref_y, torch.bfloat16, f"y {b}", int(lens[b]))


def test_packed_bad_bounds(la):
    """A sequence outside the batch, or of negative length, is skipped and recorded; the others run."""
    q, k, v, _, alpha, beta, _, _ = make(3, 2, 2, 100, 128, 128, torch.bfloat16, False, 13, layout="tok")
    cu = torch.tensor([0, 40, 30, 101], dtype=torch.int32, device="cuda")   # 0..40, 40..30, 30..101
    S = torch.full((3, 2, 128, 128), 3.0, device="cuda")
    y = torch.full((100, 2, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    la.gated_delta_prefill_varlen(q, k, v, cu, alpha, beta, y=y, S_out=S)
    assert la.last_device_status() == 2 and la.last_device_status() == 0
    assert (S[1:] == 3.0).all() and (y[40:] == 7.0).all()
    bh = lambda x: x[:40].transpose(0, 1)[None]  # noqa: E731
    ref_y, ref_S, _, _ = R.prefill(*(bh(x) for x in (q, k, v, alpha, beta)), None, 1.0)
    R.check(S[:1], ref_S, torch.bfloat16, "S")
    R.check(bh(y), ref_y, torch.bfloat16, "y")


@DTYPES
@pytest.mark.parametrize("size", [(1, 1, 1, 128, 128), (3, 4, 2, 64, 64), (2, 6, 1, 33, 7), (2, 2, 2, 256, 160), (70, 4, 4, 128, 100),
                                  (1, 2, 1, 1, 1), (99, 8, 4, 128, 128), (100, 8, 2, 64, 64), (41, 16, 8, 60, 256),
                                  (305, 4, 4, 1, 64)], ids=ids)
def test_decode_steps(la, size, dtype):
    """Steps of one token each, the state in place, against one prefill of them."""
    B, H, Hk, r, dv = size
    T = 4
    q, k, v, _, alpha, beta, _, _ = make(B, H, Hk, T, r, dv, dtype, False, 21)
    S0 = torch.randn((B, H, r, dv), generator=torch.Generator().manual_seed(2)).mul(0.3).cuda()
    S = S0.clone()
    ys = [la.gated_delta_decode_step(*(x[:, :, t:t + 1].contiguous() for x in (q, k, v)), S, alpha[:, :, t].contiguous(),
                                     beta[:, :, t].contiguous(), scale=0.2) for t in range(T)]
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, 0.2)
    assert la.last_device_status() == 0
    R.check(S, ref_S, torch.float32, "S")
    R.check(torch.cat(ys, 2), ref_y, dtype, "y")
    S3 = off(S0)
    y = la.gated_delta_decode_step(*(off(x[:, :, :1].contiguous()) for x in (q, k, v)), S3, off(alpha[:, :, 0].contiguous()),
                                   off(beta[:, :, 0].contiguous()), scale=0.2)
    ref_y, ref_S, _, _ = R.prefill(*(x[:, :, :1] for x in (q, k, v, alpha, beta)), S0, 0.2)
    R.check(S3, ref_S, torch.float32, "S, misaligned")
    R.check(y, ref_y, dtype, "y, misaligned")


@DTYPES
@pytest.mark.parametrize("state", [False, True], ids=["zero", "S0"])
@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_backward_parity(la, size, state, dtype):
    q, k, v, dy, alpha, beta, S0, dS_T = make(*size, dtype, state, seed=sum(size) + 1)
    scale = size[4] ** -0.5
    got = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, scale=scale)
    assert la.last_device_status() == 0
    R.check_all(got, R.backward(q, k, v, dy, alpha, beta, S0, dS_T, scale), dtype, size[3])


def test_backward_differences(la):
    """The gradients against central differences of the forward call, summed against fixed weights in 64 bits."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(1, 2, 1, 70, 32, 24, torch.float32, True, 31)

    def loss(**kw):
        a = dict(q=q, k=k, v=v, alpha=alpha, beta=beta, S0=S0)
        a.update(kw)
        y, S = la.gated_delta_prefill(a["q"], a["k"], a["v"], a["alpha"], a["beta"], S0=a["S0"], scale=0.5)
        return float((y.double() * dy.double()).sum() + (S.double() * dS_T.double()).sum())

    got = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, scale=0.5)
    g = torch.Generator().manual_seed(4)
    for name, x, dx in zip(("q", "k", "v", "alpha", "beta", "S0"), (q, k, v, alpha, beta, S0), got):
        d = torch.randn(x.shape, generator=g).cuda() * (0.1 if name in ("alpha", "beta") else 1.0) * x.abs().mean()
        h = 2.0 ** -6
        up, down = loss(**{name: x + h * d}), loss(**{name: x - h * d})
        slope, want = (up - down) / (2 * h), float((dx.double() * d.double()).sum())
        # the difference's own error: h^2 of the third derivative (the direction has about the values' size, so of the loss's terms
        # themselves), and FP32 outputs summed over 10^4 values
        size = float((dy.double().abs().mean() * dx.double().norm() * d.double().norm()))
        assert abs(slope - want) <= 2.0 ** -9 * size + 2.0 ** -12 * abs(want), (name, slope, want)


@DTYPES
def test_workspace_and_poison(la, dtype):
    """A caller's workspace full of NaN gives the same bits; one byte less is refused."""
    size = (1, 4, 2, 150 if dtype == torch.bfloat16 else 300, 128, 128)
    q, k, v, dy, alpha, beta, S0, dS_T = make(*size, dtype, True, 8)
    first = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0)
    need = la.gated_delta_prefill_workspace_bytes(*size, dtype=dtype)
    if need:
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        for x, z in zip(first, la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0, workspace=ws)):
            assert torch.equal(x, z)
        with pytest.raises(la.LinAttnError):
            la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0, workspace=ws[:-1])
    first = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T)
    need = la.gated_delta_backward_workspace_bytes(*size, dtype=dtype)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for x, z in zip(first, la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, workspace=ws)):
        assert torch.equal(x, z)
    with pytest.raises(la.LinAttnError):
        la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, workspace=ws[:-1])


def test_long_sequences_of_few_heads(la):
    """They go in two parts; in place, from a carried state, with a last chunk that is not full, and as a graph."""
    size = (2, 4, 2, 9800, 64, 64)
    q, k, v, _, alpha, beta, S0, _ = make(*size, torch.bfloat16, True, 33)
    S = S0.clone()
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S, S_out=S)
    apart, S2 = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0)
    assert la.last_device_status() == 0 and torch.equal(S, S2) and torch.equal(y, apart)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0)
    for _ in range(3):
        for x in held:
            x.zero_()
        graph.replay()
        assert torch.equal(held[0], y) and torch.equal(held[1], S)
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, 1.0)
    R.check(S, ref_S, torch.bfloat16, "S", size[3])
    R.check(y, ref_y, torch.bfloat16, "y", size[3])


@pytest.mark.parametrize("size", [(1, 1, 1, 2048, 256, 256), (2, 4, 2, 1001, 64, 96), (1, 3, 1, 777, 33, 7), (1, 1, 1, 2000, 1, 130),
                                  (1, 2, 1, 3000, 100, 64)], ids=ids)
def test_segments(la, size):
    """FP32 sequences of few heads, in segments: in place, with a gate of 0 and none in the same call, a workspace of NaN, as a graph."""
    q, k, v, _, alpha, beta, S0, _ = make(*size, torch.float32, True, 55)
    alpha[:, :, size[3] // 2] = 0.0
    alpha[:, :, -20:] = 1.0
    S = S0.clone()
    need = la.gated_delta_prefill_workspace_bytes(*size, dtype=torch.float32)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S, scale=0.5, S_out=S, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0, scale=0.5)
    graph.replay()
    assert torch.equal(held[0], y) and torch.equal(held[1], S)
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, 0.5)
    assert la.last_device_status() == 0
    R.check(S, ref_S, torch.float32, "S", size[3])
    R.check(y, ref_y, torch.float32, "y", size[3])


@DTYPES
def test_offsets_past_32_bits(la, dtype):
    """A sequence of more than 2^31 elements: its end is that of its last tokens run from the state before them, and the
    same packed."""
    T, r, dv = (1 << 24) + 4096 + 37, 64 if dtype == torch.bfloat16 else 1, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k = (torch.randn((1, 1, T, r), generator=g, device="cuda", dtype=dtype).mul_(r ** -0.5) for _ in range(2))
    v = torch.randn((1, 1, T, dv), generator=g, device="cuda", dtype=dtype)
    alpha, beta = (torch.rand((1, 1, T), generator=g, device="cuda").mul_(0.4).add_(c) for c in (0.6, 0.1))
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta)
    cut = (T - 1000) // 64 * 64
    part = lambda s: [x[:, :, s].contiguous() for x in (q, k, v, alpha, beta)]  # noqa: E731
    _, before = la.gated_delta_prefill(*part(slice(0, cut)))
    y2, S2 = la.gated_delta_prefill(*part(slice(cut, T)), S0=before)
    def same(a, b, what):          # (FP32 sequences of few heads go in segments, whose sums round in another order)
        if dtype == torch.bfloat16:
            assert torch.equal(a, b), what
        else:
            R.check(a, R.f64(b), dtype, what, 2000)
    same(S, S2, "S")
    same(y[:, :, cut:], y2, "y")
    assert torch.isfinite(S).all()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y3, S3 = la.gated_delta_prefill_varlen(*(x.reshape(T, 1, -1) for x in (q, k, v)), cu, alpha.reshape(T, 1), beta.reshape(T, 1))
    same(S, S3, "S packed")
    for s in (slice(0, 1000), slice(T - 1000, T)):
        same(y[0, 0, s], y3[s, 0], "y packed")
    assert la.last_device_status() == 0


def test_decode_offsets_past_32_bits(la):
    B, H, r, dv = 8200, 16, 128, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    S = torch.randn((B, H, r, dv), generator=g, device="cuda")
    q, k, v = (torch.randn((B, H, 1, 128), generator=g, device="cuda", dtype=torch.bfloat16).mul_(0.1) for _ in range(3))
    alpha, beta = (torch.rand((B, H), generator=g, device="cuda") for _ in range(2))
    ends = [0, 1, B // 2, B - 2, B - 1]
    few = [x[ends].contiguous() for x in (q, k, v, S, alpha, beta)]
    y = la.gated_delta_decode_step(q, k, v, S, alpha, beta)
    y_few = la.gated_delta_decode_step(*few)
    assert torch.equal(S[ends], few[3]) and torch.equal(y[ends], y_few)


def test_streams_and_graphs(la):
    """Calls on a side stream, captured into a graph and replayed on new inputs, give the eager calls' bits."""
    size = (1, 4, 2, 150, 128, 128)
    q, k, v, dy, alpha, beta, S0, dS_T = make(*size, torch.bfloat16, True, 9)
    new = make(*size, torch.bfloat16, True, 10)
    cu = torch.tensor([0, 50, 150], dtype=torch.int32, device="cuda")

    def calls():
        S = S0.clone()
        out = [*la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0)]
        out += la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T)
        tok = [x[0].transpose(0, 1).contiguous() for x in (q, k, v, alpha, beta)]
        out += la.gated_delta_prefill_varlen(*tok[:3], cu, *tok[3:])
        one = [x[:, :, :1].contiguous() for x in (q, k, v)]
        out += [la.gated_delta_decode_step(*one, S, alpha[:, :, 0].contiguous(), beta[:, :, 0].contiguous()), S]
        return out

    calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = calls()
    torch.cuda.current_stream().wait_stream(side)
    for x, z in zip(on_side, calls()):
        assert torch.equal(x, z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for old, fresh in zip((q, k, v, dy, alpha, beta, S0, dS_T), new):
        old.copy_(fresh)
    graph.replay()
    for x, z in zip(held, calls()):
        assert torch.equal(x, z)
    assert la.last_device_status() == 0


def test_generation(la):
    """A prompt, packed prompts, then single tokens whose logits are scored: one run, against the 64-bit recurrence, and the
    gradients of those scores back through the memory."""
    B, H, Hk, T, r, dv, V, steps = 2, 4, 2, 90, 128, 128, 333, 5
    q, k, v, _, alpha, beta, _, _ = make(B, H, Hk, T + steps, r, dv, torch.bfloat16, False, 41)
    g = torch.Generator().manual_seed(5)
    head = (torch.randn((H * dv, V), generator=g) / 8).cuda()
    picked = torch.randint(0, V, (steps, B), generator=g, dtype=torch.int32).cuda()
    cut = lambda a, b: [x[:, :, a:b].contiguous() for x in (q, k, v, alpha, beta)]  # noqa: E731
    y0, S = la.gated_delta_prefill(*cut(0, T))
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, None, 1.0)
    scores = []
    for t in range(steps):
        qt, kt, vt, at, bt = cut(T + t, T + t + 1)
        y = la.gated_delta_decode_step(qt, kt, vt, S, at[:, :, 0].contiguous(), bt[:, :, 0].contiguous())
        logits = y.float().reshape(B, H * dv) @ head
        lp, ent, lse, best, which = la.token_logprobs(logits, picked[t], top=3)
        scores.append(lp)
        ref = R.score(logits, picked[t].cpu(), 3)
        assert torch.equal(which.cpu(), ref[4])
        assert torch.allclose(lp.cpu().double(), ref[0], rtol=1e-5, atol=1e-5)
    R.check(S, ref_S, torch.bfloat16, "S")
    R.check(y0, ref_y[:, :, :T], torch.bfloat16, "y")
    # a training step on the same tokens: logits of every token, the scores' gradient, and back through the memory
    n = T + steps
    y, _ = la.gated_delta_prefill(q, k, v, alpha, beta)
    rows = y.transpose(1, 2).reshape(B * n, H * dv).float()
    target = torch.randint(-1, V, (B * n,), generator=g, dtype=torch.int32).cuda()
    logits = rows @ head
    lp, ent, lse, _, _ = la.token_logprobs(logits, target)
    dlogits = la.token_logprobs_backward(logits, target, lse, ent, torch.full_like(lp, -1.0 / (B * n)))
    dy = (dlogits @ head.t()).reshape(B, n, H, dv).transpose(1, 2).to(torch.bfloat16).contiguous()
    got = la.gated_delta_backward(q, k, v, dy, alpha, beta)
    R.check_all(got, R.backward(q, k, v, dy, alpha, beta, None, None, 1.0), torch.bfloat16, n)
    assert la.last_device_status() == 0
