"""Decayed linear attention on the GPU (la_decay_*) against its 64-bit recurrence.

Tolerances are elementwise and derived in decay_reference: the FP32 recurrence rounds each
of its sums (U32 = 2^-24), the chunked BF16 form also rounds the scores or the carried
state once (U16 = 2^-8) before a product whose absolute terms the reference sums up."""
import pytest
import torch

import decay_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    from recurrent_state_02_gb300 import build
    build.build()
    import recurrent_state_02_gb300 as la_mod
    assert torch.cuda.is_available()
    return la_mod


DECAYS = [1.0, 0.0, 0.5, 0.99609375, 0.3, 0.9, 1e-3, 1.0 - 2.0 ** -20]


def make(B, H, T, r, dv, dtype, state, seed, layout="bh"):
    g = torch.Generator().manual_seed(seed)
    shape = (lambda d: (B, H, T, d)) if layout == "bh" else (lambda d: (T, H, d))
    q, k = (torch.randn(shape(r), generator=g).to(dtype).cuda() for _ in range(2))
    v, dy = (torch.randn(shape(dv), generator=g).to(dtype).cuda() for _ in range(2))
    S0, dS_T = ((torch.randn((B, H, r, dv), generator=g)).cuda() if state else None for _ in range(2))
    decay = torch.tensor([DECAYS[(h + seed) % len(DECAYS)] for h in range(H)]).cuda()
    return q, k, v, dy, decay, S0, dS_T


def chunked(dtype):
    return dtype == torch.bfloat16   # (the tolerance covers both BF16 paths)


SIZES = [
    # B, H, T, r, dv
    (1, 1, 1, 128, 128), (2, 3, 2, 64, 64), (1, 8, 31, 128, 128), (1, 8, 33, 128, 128), (1, 2, 64, 64, 128),
    (1, 2, 127, 128, 64), (2, 8, 128, 128, 128), (1, 3, 129, 64, 64), (1, 8, 300, 128, 128), (1, 2, 513, 128, 192),
    (1, 2, 777, 64, 256), (1, 2, 40, 96, 80), (2, 2, 37, 33, 7), (1, 1, 50, 256, 160), (1, 2, 19, 1, 1),
    (1, 1, 130, 128, 100), (8, 20, 70, 64, 32), (8, 20, 70, 128, 32), (8, 20, 9, 100, 32), (8, 20, 9, 40, 32), (8, 20, 66, 200, 32),
    (160, 1, 65, 20, 20),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("state", [False, True], ids=["zero", "S0"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_prefill_parity(la, size, state, dtype):
    B, H, T, r, dv = size
    q, k, v, _, decay, S0, _ = make(*size, dtype, state, seed=sum(size))
    scale = r ** -0.5
    y, S = la.decay_prefill(q, k, v, decay, S0=S0, scale=scale)
    assert la.last_device_status() == 0
    ref_y, ref_S = R.prefill(q, k, v, decay, S0, scale)
    abs_y, abs_S = R.prefill(*R.absolute(q, k, v), decay, *R.absolute(S0), scale)
    R.check(S, ref_S, R.state_bound(T, abs_S, chunked(dtype)), "S")
    R.check(y, ref_y, R.bounds(T, r, dv, dtype == torch.bfloat16, abs_y, ref_y, chunked(dtype)), "y")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_prefill_no_tokens_copies_the_state(la, dtype):
    q, k, v, _, decay, S0, _ = make(2, 3, 0, 128, 64, dtype, True, 1)
    y, S = la.decay_prefill(q, k, v, decay, S0=S0)
    assert y.numel() == 0 and torch.equal(S, S0)
    y, S = la.decay_prefill(q, k, v, decay)
    assert not S.any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", [5, 300])
def test_prefill_in_place_and_misaligned(la, T, dtype):
    """S0 may be S_out; a state 4 bytes off a 16-byte boundary, and q, k, v, y one element off theirs, give
    the same values to rounding."""
    q, k, v, _, decay, S0, _ = make(1, 3, T, 128, 128, dtype, True, 2)
    y, S = la.decay_prefill(q, k, v, decay, S0=S0, scale=0.1)
    S2 = S0.clone()
    y2, _ = la.decay_prefill(q, k, v, decay, S0=S2, scale=0.1, S_out=S2)
    assert torch.equal(y, y2) and torch.equal(S, S2)

    def off(t):
        buf = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)
        buf[1:].copy_(t.reshape(-1))
        return buf[1:].view(t.shape)

    S3 = off(S0)
    y3 = off(y)
    la.decay_prefill(off(q), off(k), off(v), decay, S0=S3, scale=0.1, y=y3, S_out=S3)
    assert la.last_device_status() == 0
    ref_y, ref_S = R.prefill(q, k, v, decay, S0, 0.1)
    abs_y, abs_S = R.prefill(*R.absolute(q, k, v), decay, S0.abs(), 0.1)
    R.check(S3, ref_S, R.state_bound(T, abs_S, chunked(dtype)), "S")
    R.check(y3, ref_y, R.bounds(T, 128, 128, dtype == torch.bfloat16, abs_y, ref_y, chunked(dtype)), "y")


@pytest.mark.parametrize("split", [1, 100, 128, 200])
def test_prefill_continues(la, split):
    """Two calls chained through the state agree with one."""
    q, k, v, _, decay, S0, _ = make(1, 8, 300, 128, 128, torch.bfloat16, True, 3)
    cut = lambda x, a, b: x[:, :, a:b].contiguous()  # noqa: E731
    _, S1 = la.decay_prefill(cut(q, 0, split), cut(k, 0, split), cut(v, 0, split), decay, S0=S0)
    y2, S2 = la.decay_prefill(cut(q, split, 300), cut(k, split, 300), cut(v, split, 300), decay, S0=S1)
    ref_y, ref_S = R.prefill(q, k, v, decay, S0, 1.0)
    abs_y, abs_S = R.prefill(*R.absolute(q, k, v), decay, S0.abs(), 1.0)
    R.check(S2, ref_S, 2 * R.state_bound(300, abs_S, True), "S")
    R.check(y2, ref_y[:, :, split:], 2 * R.bounds(300, 128, 128, True, abs_y, ref_y, True)[:, :, split:], "y")


@pytest.mark.parametrize("size", [(1, 2, 2000, 128, 128), (1, 3, 1500, 64, 64), (2, 8, 1921, 128, 64), (1, 1, 5000, 64, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_split_sweeps(la, size):
    """Few heads and a long sequence: the sweep runs in segments (also over its own state, and with a workspace of the
    caller's), and so do the three sweeps of the gradients."""
    B, H, T, r, dv = size
    assert la.decay_prefill_workspace_bytes(*size) > 0
    q, k, v, dy, decay, S0, dS_T = make(*size, torch.bfloat16, True, seed=sum(size))
    scale = r ** -0.5
    ref_y, ref_S = R.prefill(q, k, v, decay, S0, scale)
    abs_y, abs_S = R.prefill(*R.absolute(q, k, v), decay, *R.absolute(S0), scale)
    ws = torch.full((la.decay_prefill_workspace_bytes(*size),), 255, dtype=torch.uint8, device="cuda")
    S = S0.clone()
    y, _ = la.decay_prefill(q, k, v, decay, S0=S, scale=scale, S_out=S, workspace=ws)
    assert la.last_device_status() == 0
    R.check(S, ref_S, R.state_bound(T, abs_S, True), "S")
    R.check(y, ref_y, R.bounds(T, r, dv, True, abs_y, ref_y, True), "y")
    with pytest.raises(la.LinAttnError):
        la.decay_prefill(q, k, v, decay, S0=S0, workspace=ws[:-1])
    got = la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T, scale=scale)
    assert la.last_device_status() == 0
    ref = R.backward(q, k, v, dy, decay, S0, dS_T, scale)
    mag = R.backward(*R.absolute(q, k, v, dy), decay, *R.absolute(S0, dS_T), scale)
    for x, z, m, name in zip(got[:3], ref[:3], mag[:3], ("dq", "dk", "dv")):
        R.check(x, z, R.bounds(T, r, dv, True, m, z, True), name)
    R.check(got[3], ref[3], R.state_bound(T, mag[3], True), "dS0")


# one CTA per 32 columns: 1 to 65 of them, so that 16 to 3 segments run, or one
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", [
    (1, 1, 128, 20, 20), (1, 2, 129, 96, 40), (2, 3, 255, 40, 100), (1, 3, 600, 64, 50), (1, 5, 200, 100, 150), (2, 10, 131, 30, 64),
    (1, 10, 150, 50, 100), (3, 12, 513, 100, 30), (1, 12, 520, 64, 100), (4, 16, 512, 40, 9), (5, 13, 515, 40, 9),
    (1, 2, 700, 200, 256), (1, 5, 160, 256, 200), (1, 1, 515, 20, 60), (1, 4, 513, 100, 100), (1, 1, 512, 256, 100),
    (1, 1, 1030, 200, 200), (1, 1, 2049, 128, 20)], ids=lambda s: "x".join(map(str, s)))
def test_recurrence_in_segments(la, size, dtype):
    """Few CTAs and some length: the recurrence runs its segments side by side, over its own state too, and so do the
    sweeps of the gradients.  (A term is rounded at most twice per segment and token: within the bounds.)"""
    B, H, T, r, dv = size
    q, k, v, dy, decay, S0, dS_T = make(*size, dtype, True, seed=sum(size))
    scale = r ** -0.5
    S = S0.clone()
    y, _ = la.decay_prefill(q, k, v, decay, S0=S, scale=scale, S_out=S)
    got = la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T, scale=scale)
    assert la.last_device_status() == 0
    ref_y, ref_S = R.prefill(q, k, v, decay, S0, scale)
    abs_y, abs_S = R.prefill(*R.absolute(q, k, v), decay, *R.absolute(S0), scale)
    bf16 = dtype == torch.bfloat16
    R.check(S, ref_S, R.state_bound(T, abs_S, False), "S")
    R.check(y, ref_y, R.bounds(T, r, dv, bf16, abs_y, ref_y, False), "y")
    ref = R.backward(q, k, v, dy, decay, S0, dS_T, scale)
    mag = R.backward(*R.absolute(q, k, v, dy), decay, *R.absolute(S0, dS_T), scale)
    for x, z, m, name in zip(got[:3], ref[:3], mag[:3], ("dq", "dk", "dv")):
        R.check(x, z, R.bounds(T, r, dv, bf16, m, z, False), name)
    R.check(got[3], ref[3], R.state_bound(T, mag[3], False), "dS0")


def test_recurrence_in_segments_is_captured(la):
    """A graph of the call gives the same bits as the call, twice."""
    q, k, v, _, decay, S0, _ = make(1, 3, 300, 40, 70, torch.float32, True, seed=9)
    y, S = la.decay_prefill(q, k, v, decay, S0=S0)
    y2, S2 = torch.zeros_like(y), torch.zeros_like(S)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.decay_prefill(q, k, v, decay, S0=S0, y=y2, S_out=S2)
    for _ in range(2):
        y2.zero_(), S2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(S, S2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("r,dv", [(128, 128), (64, 128), (40, 24)])
def test_packed(la, r, dv, dtype):
    """Ragged lengths (none, one, chunk borders); rows outside every sequence hold NaN and reach no result, and
    their outputs stay as they were."""
    lens, H = [0, 1, 2, 31, 32, 33, 127, 128, 129, 0, 256, 300, 5], 3
    lead, gap = 3, 2
    total = lead + sum(lens) + gap
    q, k, v, _, decay, _, _ = make(len(lens), H, total, r, dv, dtype, False, 4, layout="tok")
    S0 = torch.randn((len(lens), H, r, dv), generator=torch.Generator().manual_seed(5)).cuda()
    for t in (q, k, v):
        t[:lead] = float("nan")
        t[total - gap:] = float("nan")
    cu = torch.tensor([lead + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    y = torch.full((total, H, dv), 7.0, device="cuda", dtype=dtype)
    S = S0.clone()
    la.decay_prefill_varlen(q, k, v, decay, cu, S0=S, scale=0.25, y=y, S_out=S)
    assert la.last_device_status() == 0
    assert (y[:lead] == 7).all() and (y[total - gap:] == 7).all()
    for b, n in enumerate(lens):
        a = int(cu[b])
        one = [x[a:a + n].transpose(0, 1)[None] for x in (q, k, v)]
        ref_y, ref_S = R.prefill(*one, decay, S0[b:b + 1], 0.25)
        abs_y, abs_S = R.prefill(*R.absolute(*one), decay, S0[b:b + 1].abs(), 0.25)
        R.check(S[b:b + 1], ref_S, R.state_bound(n, abs_S, chunked(dtype)), f"S {n}")
        R.check(y[a:a + n].transpose(0, 1)[None], ref_y,
                R.bounds(n, r, dv, dtype == torch.bfloat16, abs_y, ref_y, chunked(dtype)), f"y {n}")


@pytest.mark.parametrize("B", [256, 300])
def test_packed_many_sequences(la, B):
    """Batches on both sides of the size up to which the longest sequences run first: every sequence finds its own rows
    and state (short ones, which take the recurrence, beside chunked ones)."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 60, (B,), generator=g).tolist()
    lens[B - 1], lens[7] = 400, 0
    H, total = 1, sum(lens)
    q, k, v, _, _, _, _ = make(1, H, total, 64, 64, torch.bfloat16, False, 8, layout="tok")
    decay = torch.tensor([0.97], device="cuda")
    S0 = torch.randn((B, H, 64, 64), generator=g).cuda()
    cu = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    y, S = la.decay_prefill_varlen(q, k, v, decay, cu, S0=S0, scale=0.5)
    assert la.last_device_status() == 0
    for b in [*range(0, B, 17), 7, 8, B - 2, B - 1]:
        a, n = int(cu[b]), lens[b]
        one = [x[a:a + n].transpose(0, 1)[None] for x in (q, k, v)]
        ref_y, ref_S = R.prefill(*one, decay, S0[b:b + 1], 0.5)
        abs_y, abs_S = R.prefill(*R.absolute(*one), decay, S0[b:b + 1].abs(), 0.5)
        R.check(S[b:b + 1], ref_S, R.state_bound(n, abs_S, True), f"S {b}")
        R.check(y[a:a + n].transpose(0, 1)[None], ref_y, R.bounds(n, 64, 64, True, abs_y, ref_y, True), f"y {b}")


def test_packed_neighbours_do_not_leak(la):
    """A sequence of NaN between two others leaves them finite and unchanged."""
    lens, H = [100, 70, 300, 40], 2
    total = sum(lens)
    q, k, v, _, decay, _, _ = make(4, H, total, 128, 128, torch.bfloat16, False, 6, layout="tok")
    cu = torch.tensor([0, 100, 170, 470, 510], dtype=torch.int32, device="cuda")
    y, S = la.decay_prefill_varlen(q, k, v, decay, cu)
    for t in (q, k, v):
        t[100:170] = float("nan")
    y2, S2 = la.decay_prefill_varlen(q, k, v, decay, cu)
    keep = [0, 2, 3]
    assert torch.equal(S[keep], S2[keep]) and torch.equal(y[:100], y2[:100]) and torch.equal(y[170:], y2[170:])
    assert torch.isnan(S2[1]).all()


def test_packed_bad_bounds_are_recorded(la):
    q, k, v, _, decay, _, _ = make(3, 2, 64, 128, 64, torch.bfloat16, False, 7, layout="tok")
    cu = torch.tensor([0, 40, 20, 64], dtype=torch.int32, device="cuda")   # sequence 1 has a negative length
    S = torch.full((3, 2, 128, 64), 5.0, device="cuda")
    y = torch.full((64, 2, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    la.decay_prefill_varlen(q, k, v, decay, cu, y=y, S_out=S)
    assert la.last_device_status() == 2 and la.last_device_status() == 0
    assert (S[1] == 5).all() and not (S[0] == 5).all() and not (S[2] == 5).all()
    cu = torch.tensor([0, 40, 50, 65], dtype=torch.int32, device="cuda")   # past the total
    la.decay_prefill_varlen(q, k, v, decay, cu, y=y, S_out=S)
    assert la.last_device_status() == 2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", [(1, 1, 128, 128), (3, 8, 128, 128), (2, 2, 64, 64), (2, 3, 96, 80), (1, 2, 256, 256),
                                  (2, 2, 33, 7), (1, 2, 5, 132), (40, 16, 128, 64)], ids=lambda s: "x".join(map(str, s)))
def test_decode(la, size, dtype):
    B, H, r, dv = size
    q, k, v, _, decay, S0, _ = make(B, H, 1, r, dv, dtype, True, sum(size))
    S = S0.clone()
    y = la.decay_decode_step(q, k, v, decay, S, scale=0.5)
    ref_y, ref_S = R.prefill(q, k, v, decay, S0, 0.5)
    abs_y, abs_S = R.prefill(*R.absolute(q, k, v), decay, S0.abs(), 0.5)
    R.check(S, ref_S, R.state_bound(1, abs_S, False), "S")
    R.check(y, ref_y, R.bounds(1, r, dv, dtype == torch.bfloat16, abs_y, ref_y, False), "y")
    # a state off its 16-byte boundary takes the token recurrence
    buf = torch.empty(S0.numel() + 1, device="cuda")
    S2 = buf[1:].view(S0.shape).copy_(S0)
    y2 = la.decay_decode_step(q, k, v, decay, S2, scale=0.5)
    R.check(S2, ref_S, R.state_bound(1, abs_S, False), "S")
    R.check(y2, ref_y, R.bounds(1, r, dv, dtype == torch.bfloat16, abs_y, ref_y, False), "y")


BWD = [(1, 1, 1, 128, 128), (1, 3, 2, 64, 64), (2, 8, 31, 128, 128), (1, 2, 127, 128, 64), (1, 2, 128, 64, 128),
       (1, 8, 129, 128, 128), (1, 8, 300, 64, 64), (1, 2, 40, 96, 80), (1, 2, 37, 33, 7), (1, 1, 30, 256, 160),
       (1, 2, 400, 128, 192)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("state", [False, True], ids=["zero", "states"])
@pytest.mark.parametrize("size", BWD, ids=lambda s: "x".join(map(str, s)))
def test_backward_parity(la, size, state, dtype):
    B, H, T, r, dv = size
    q, k, v, dy, decay, S0, dS_T = make(*size, dtype, state, seed=sum(size) + 1)
    scale = r ** -0.5
    got = la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T, scale=scale)
    assert la.last_device_status() == 0
    ref = R.backward(q, k, v, dy, decay, S0, dS_T, scale)
    mag = R.backward(*R.absolute(q, k, v, dy), decay, *R.absolute(S0, dS_T), scale)
    for x, y, m, name in zip(got[:3], ref[:3], mag[:3], ("dq", "dk", "dv")):
        R.check(x, y, R.bounds(T, r, dv, dtype == torch.bfloat16, m, y, chunked(dtype)), name)
    R.check(got[3], ref[3], R.state_bound(T, mag[3], chunked(dtype)), "dS0")


def test_backward_no_tokens(la):
    q, k, v, dy, decay, S0, dS_T = make(2, 2, 0, 128, 64, torch.bfloat16, True, 9)
    assert torch.equal(la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T)[3], dS_T)
    assert not la.decay_backward(q, k, v, dy, decay)[3].any()


@pytest.mark.parametrize("which", ["q", "k", "v", "S0"])
def test_backward_against_differences(la, which):
    """The loss <y, dy> + <S_T, dS_T> is linear in each of q, k, v and S0 alone, so a central difference of any
    step equals the derivative: (L(x + u) - L(x - u)) / 2 = <grad, u>, to the rounding of the two losses
    (FP32 kernel, losses summed in 64 bits: (T + r + 16) 2 U32 of the absolute terms each)."""
    T, r, dv = 70, 48, 40
    q, k, v, dy, decay, S0, dS_T = make(1, 4, T, r, dv, torch.float32, True, 10)
    x = dict(q=q, k=k, v=v, S0=S0)
    u = torch.randn(x[which].shape, generator=torch.Generator().manual_seed(11)).cuda()

    def loss(sign):
        z = dict(x)
        z[which] = x[which] + sign * u
        y, S = la.decay_prefill(z["q"], z["k"], z["v"], decay, S0=z["S0"], scale=0.3)
        return float((y.double() * dy.double()).sum() + (S.double() * dS_T.double()).sum())

    grads = dict(zip(("q", "k", "v", "S0"), la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T, scale=0.3)))
    mag = {n: t.abs() for n, t in x.items()}
    mag[which] = mag[which] + u.abs()
    ay, aS = R.prefill(mag["q"], mag["k"], mag["v"], decay, mag["S0"], 0.3)
    size = float((ay * R.f64(dy).abs()).sum() + (aS * R.f64(dS_T).abs()).sum())
    tol = 3 * (T + r + 16) * 2 * R.U32 * size
    assert abs((loss(1) - loss(-1)) / 2 - float((grads[which].double() * u.double()).sum())) <= tol


def test_streams_and_graphs(la):
    """The calls run on the current stream, and can be captured and replayed on new inputs."""
    q, k, v, dy, decay, S0, dS_T = make(2, 4, 300, 128, 128, torch.bfloat16, True, 12)

    def once():
        y, S = la.decay_prefill(q, k, v, decay, S0=S0, scale=0.1)
        yd = la.decay_decode_step(q[:, :, :1].contiguous(), k[:, :, :1].contiguous(), v[:, :, :1].contiguous(), decay, S)
        return (y, S, yd) + la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T, scale=0.1)

    want = [t.clone() for t in once()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = once()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = once()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))
    q.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], -want[0]) and la.last_device_status() == 0


def test_python_refusals(la):
    q, k, v, dy, decay, S0, _ = make(1, 2, 8, 64, 64, torch.bfloat16, True, 13)
    with pytest.raises(ValueError):
        la.decay_prefill(q, k[:, :, ::2], v, decay)
    with pytest.raises(ValueError):
        la.decay_prefill(q, k, v.float(), decay)
    with pytest.raises(ValueError):
        la.decay_prefill(q, k, v, decay.double())
    with pytest.raises(ValueError):
        la.decay_prefill(q, k, v, None)
    with pytest.raises(ValueError):
        la.decay_prefill(q, k, v, decay[:1])
    with pytest.raises(ValueError):
        la.decay_decode_step(q, k, v, decay, S0)
    with pytest.raises(la.LinAttnError):
        la.decay_prefill(q, k, v, decay, scale=float("nan"))
    with pytest.raises(ValueError):
        la.decay_prefill(q.half(), k.half(), v.half(), decay)


@pytest.mark.parametrize("r,dv", [(128, 128), (64, 64), (64, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_packed_tail_is_isolated(la, r, dv, bad):
    """Sequences of one chunk and of several, with a ragged last one, right before rows that are not finite (another
    sequence's, long and short, and what lies behind the last one): outputs and states have the bits of the run with
    finite rows there, whatever the timing of the loads (L2 warm and flushed)."""
    lens, ends, H = [129, 40, 200, 3, 255, 20, 257, 40, 300, 3, 1000, 130, 385, 7, 100], {40, 3, 20, 130, 7}, 16
    total = sum(lens) + 150
    q, k, v, _, _, _, _ = make(1, H, total, r, dv, torch.bfloat16, False, 21, layout="tok")
    decay = torch.tensor([DECAYS[h % len(DECAYS)] for h in range(H)]).cuda()
    S0 = torch.randn((len(lens), H, r, dv), generator=torch.Generator().manual_seed(22)).cuda()
    start = [sum(lens[:i]) for i in range(len(lens) + 1)]
    cu = torch.tensor(start, dtype=torch.int32, device="cuda")
    keep = [b for b, n in enumerate(lens) if n not in ends]
    rows = torch.cat([torch.arange(start[b], start[b + 1]) for b in keep]).cuda()
    y, S = la.decay_prefill_varlen(q, k, v, decay, cu, S0=S0, scale=0.25)
    assert la.last_device_status() == 0 and torch.isfinite(y[rows]).all() and torch.isfinite(S).all()
    spoilt = torch.ones(total, dtype=torch.bool, device="cuda")
    spoilt[rows] = False
    for t in (q, k, v):
        t[spoilt] = bad
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(24):
        if i % 2:
            flush.fill_(i)
        y2, S2 = la.decay_prefill_varlen(q, k, v, decay, cu, S0=S0, scale=0.25)
        assert torch.equal(y[rows], y2[rows]) and torch.equal(S[keep], S2[keep]), i
    # one sequence alone, nothing but padding behind it
    for n in (129, 130, 200, 255, 257, 300, 385, 1000):
        one = [torch.randn((n + 128, H, d), generator=torch.Generator().manual_seed(n + d)).bfloat16().cuda() for d in (r, r, dv)]
        cu1 = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        y, S = la.decay_prefill_varlen(*one, decay, cu1, scale=0.25)
        for t in one:
            t[n:] = bad
        for i in range(6):
            if i % 2:
                flush.fill_(i)
            y2, S2 = la.decay_prefill_varlen(*one, decay, cu1, scale=0.25)
            assert torch.equal(y[:n], y2[:n]) and torch.equal(S, S2) and torch.isfinite(y2[:n]).all(), (n, i)
    assert la.last_device_status() == 0


def test_backward_workspace_of_the_callers(la):
    """Gradients in segments over a workspace of the caller's: larger than asked for gives the same bits; one byte short, off
    its 256-byte boundary or elsewhere is refused and leaves the outputs to the next call."""
    size = (1, 2, 1500, 128, 128)
    q, k, v, dy, decay, S0, dS_T = make(*size, torch.bfloat16, True, seed=23)
    need = la.decay_backward_workspace_bytes(*size)
    assert need > 0
    want = la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T, scale=0.1)
    buf = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    got = la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T, scale=0.1, workspace=buf)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and (buf[need:] == 255).all()
    for ws in (buf[:need - 1], buf[16:16 + need], buf[128:]):
        with pytest.raises(la.LinAttnError):
            la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T, scale=0.1, workspace=ws)
    with pytest.raises(ValueError):
        la.decay_backward(q, k, v, dy, decay, S0=S0, dS_T=dS_T, scale=0.1, workspace=buf.cpu())
    with pytest.raises(la.LinAttnError):
        la.decay_prefill(q, k, v, decay, workspace=buf[16:])
    assert la.last_device_status() == 0
