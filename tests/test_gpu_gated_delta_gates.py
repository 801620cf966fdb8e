"""The gates' gradient of the gated delta rule (la_gated_delta_backward) where gates are small, against 64 bits.

dalpha_t = <S_{t-1}, G_t - k_t dv_t^T> does not depend on alpha_t: it is as large where the gate is 1e-30 as where it is 1.  Bounds: the
state before the token and the gradient behind its gate each carry the relative error that gdelta_reference derives for
FP32 results (`tolerance`), of their own size or of what earlier (later) and larger ones have left of theirs: s_t = max(|S_t|, alpha_t s_{t-1}) and
the same backwards.  Errors that are random to the other factor leave sqrt(2) tolerance s g / sqrt(r dv) of it in the product as a
standard deviation, and its own sums the tolerance of its value: that is the bound of the 2-norm over all tokens, and eight of it that of
a single one.  Nothing is divided by a gate."""
import math

import pytest
import torch

import gdelta_reference as R
from test_gpu_gated_delta import DTYPES, ids, la, make  # noqa: F401  (la: the fixture)

pytestmark = pytest.mark.gpu


def sizes_and_gradient(q, k, v, dy, alpha, beta, S0, dS_T, scale):
    """(dalpha, s_{t-1} g_t / sqrt(r dv)) of every token."""
    _, S, e, decayed = R.prefill(q, k, v, alpha, beta, S0, scale)
    B, H, T, n = e.shape
    q, k, dy, a, b = R._wide(q, H), R._wide(k, H), scale * R.f64(dy), R.f64(alpha), R.f64(beta)
    norm = lambda x: x.square().sum((2, 3)).sqrt()  # noqa: E731
    before = [torch.zeros_like(S) if S0 is None else R.f64(S0)]
    sizes = [norm(before[0])]
    for t in range(T):
        before.append(decayed[t] + k[:, :, t, :, None] * (b[:, :, t, None] * e[:, :, t])[:, :, None, :])
        sizes.append(torch.maximum(norm(before[-1]), a[:, :, t] * sizes[-1]))
    G = torch.zeros_like(S) if dS_T is None else R.f64(dS_T).clone()
    g = norm(G)
    da, size = torch.zeros_like(a), torch.zeros_like(a)
    for t in reversed(range(T)):
        G = G + q[:, :, t, :, None] * dy[:, :, t, None, :]
        g = torch.maximum(norm(G), g)
        lam = (G * k[:, :, t, :, None]).sum(2)
        G = G - k[:, :, t, :, None] * (b[:, :, t, None] * lam)[:, :, None, :]
        g = torch.maximum(norm(G), g)
        da[:, :, t] = (G * before[t]).sum((2, 3))
        size[:, :, t] = sizes[t] * g / math.sqrt(G.shape[2] * n)
        G, g = a[:, :, t, None, None] * G, a[:, :, t] * g
    return da, size


def check_gates(got, args, dtype, T, what):
    alpha = args[4]
    ref, size = sizes_and_gradient(*args)
    zero = alpha.cpu() == 0              # (where 0 is written)
    assert torch.isfinite(got).all() and not got[alpha == 0].any(), what
    err = torch.where(zero, 0.0, (got.cpu().double() - ref).abs())
    unit = math.sqrt(2) * size + ref.abs()
    tol = R.tolerance(dtype, torch.float32, T)
    rel, big = float(err.norm() / unit.norm().clamp(min=1e-300)), float((err / unit.clamp(min=1e-300)).max())
    print(f"[gates] {what}: {rel:.2e} (bound {tol:.1e}), largest {big:.2e} (bound {8 * tol:.1e})")
    assert rel <= tol and big <= 8 * tol, (what, rel, big, tol)


def backward(la, args, dtype, what):  # noqa: F811
    q, k, v, dy, alpha, beta, S0, dS_T, scale = args
    got = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, scale=scale)
    assert la.last_device_status() == 0
    T = q.shape[2]
    check_gates(got[3], args, dtype, T, what)
    ref, terms = R.backward(*args[:8], scale)
    R.check_all((*got[:3], None, *got[4:]), (ref, terms), dtype, T)
    return got


SIZES = [(1, 2, 2, 150, 128, 128), (2, 4, 2, 131, 64, 64), (1, 2, 1, 70, 128, 64), (1, 2, 2, 97, 64, 128), (1, 3, 3, 40, 33, 7),
         (1, 1, 1, 66, 256, 160), (1, 2, 1, 130, 1, 3), (2, 2, 2, 16, 128, 128), (1, 2, 1, 1, 64, 64)]
SMALL = [1e-2, 1e-3, 1e-5, 1e-8, 1e-12, 1e-30, 1e-42]


@DTYPES
@pytest.mark.parametrize("gate", SMALL)
def test_single_small_gates(la, gate, dtype):  # noqa: F811
    """A small gate here and there, at the ends of chunks too, two of them side by side."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(1, 2, 2, 150, 128, 128, dtype, True, 71)
    for t in (0, 17, 63, 64, 100, 101, 127, 149):
        alpha[:, 0, t] = gate
    alpha[:, 1, 70] = gate
    backward(la, (q, k, v, dy, alpha, beta, S0, dS_T, 128 ** -0.5), dtype, f"gate {gate}")


@DTYPES
@pytest.mark.parametrize("state", [False, True], ids=["zero", "S0"])
@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_small_gates_of_all_sizes(la, size, state, dtype):  # noqa: F811
    """Every seventh gate is small, from 1e-2 down to a denormal number, and one is 0."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(*size, dtype, state, sum(size) + 5)
    for i, t in enumerate(range(0, size[3], 7)):
        alpha[:, :, t] = SMALL[i % len(SMALL)]
    alpha[0, 0, size[3] // 2] = 0.0
    backward(la, (q, k, v, dy, alpha, beta, S0, dS_T, size[4] ** -0.5), dtype, str(size))


@DTYPES
@pytest.mark.parametrize("gate", [0.05, 1e-2, 1e-4, 1e-20, 1e-40])
def test_all_gates_small(la, gate, dtype):  # noqa: F811
    """A memory that forgets nearly everything with every token."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(1, 4, 2, 140, 128, 128, dtype, True, 73)
    alpha *= gate
    backward(la, (q, k, v, dy, alpha, beta, S0, dS_T, 1.0), dtype, f"all {gate}")


@DTYPES
def test_small_gradients(la, dtype):  # noqa: F811
    """Gradients as small as a mean over a large batch makes them lose nothing behind a small gate."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(1, 2, 2, 140, 128, 128, dtype, True, 74)
    alpha[:, :, ::9] = 1e-30
    backward(la, (q, k, v, (dy.float() * 2.0 ** -30).to(dtype), alpha, beta, S0, dS_T * 2.0 ** -30, 1.0), dtype, "small gradients")


@DTYPES
def test_small_gate_against_differences(la, dtype):  # noqa: F811
    """dalpha at a gate near 0 is the slope of the loss there: states are linear in one gate, so a difference over a step of 1/2 is it."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(1, 2, 1, 100, 64, 64, torch.float32, True, 75)
    alpha[:, :, 40] = 1e-30

    def loss(a):
        y, S = la.gated_delta_prefill(q, k, v, a, beta, S0=S0, scale=0.5)
        return (y.double() * dy.double()).sum((2, 3)) + (S.double() * dS_T.double()).sum((2, 3))

    other = alpha.clone()
    other[:, :, 40] = 0.5
    slope = (loss(other) - loss(alpha)) / 0.5
    cast = lambda x: x.to(dtype)  # noqa: E731
    got = la.gated_delta_backward(cast(q), cast(k), cast(v), cast(dy), alpha, beta, S0=S0, dS_T=dS_T, scale=0.5)[3][:, :, 40]
    # the loss is a sum of 100 x 64 + 64 x 64 products of outputs that are off by 2^-20 of their norm; BF16: its inputs' own roundings, of
    # which some 100 tokens' carry into the state, 2^-8 of terms of the sums' size
    scale = float((S0.norm() * dS_T.norm()) + dy.norm() * 30)
    bound = 2.0 ** -18 * scale if dtype == torch.float32 else 2.0 ** -8 * scale
    assert (got.double() - slope).abs().max() <= bound, (got, slope, bound)
    assert slope.abs().max() > 4 * 2.0 ** -18 * scale          # (there is a slope to find)


@DTYPES
def test_reset_by_the_smallest_gate(la, dtype):  # noqa: F811
    """The smallest normal number for a gate of 0: the same outputs and other gradients, and there the derivative (at 0 itself, 0 is written)."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(1, 2, 2, 150, 128, 128, dtype, True, 78)
    where = torch.zeros_like(alpha, dtype=torch.bool)
    where[:, 0, [0, 30, 64]], where[:, 1, [63, 149]] = True, True
    least = torch.where(where, torch.finfo(torch.float32).tiny, alpha)
    reset = torch.where(where, 0.0, alpha)
    for x, z in zip(la.gated_delta_prefill(q, k, v, least, beta, S0=S0), la.gated_delta_prefill(q, k, v, reset, beta, S0=S0)):
        assert torch.equal(x, z)
    got, at_0 = (la.gated_delta_backward(q, k, v, dy, a, beta, S0=S0, dS_T=dS_T) for a in (least, reset))
    for i in (0, 1, 2, 4):
        assert torch.equal(got[i], at_0[i]), R.NAMES[i]
    assert torch.equal(got[3][~where], at_0[3][~where]) and not at_0[3][where].any()
    ref, size = sizes_and_gradient(q, k, v, dy, reset, beta, S0, dS_T, 1.0)      # (the derivative at 0)
    err = (got[3].cpu().double() - ref).abs()[where.cpu()]
    assert (err <= 8 * R.tolerance(dtype, torch.float32, 150) * (math.sqrt(2) * size + ref.abs())[where.cpu()]).all(), err
    assert ref[where.cpu()].abs().min() > 1e-3


@DTYPES
def test_gradients_that_nobody_wants(la, dtype):  # noqa: F811
    """Without room for dalpha or dbeta the C entry forms the others all the same, to the bit."""
    B, H, Hk, T, r, dv = size = (1, 4, 2, 150, 128, 128)
    q, k, v, dy, alpha, beta, S0, dS_T = make(*size, dtype, True, 77)
    want = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, scale=0.2)
    need = la.gated_delta_backward_workspace_bytes(*size, dtype=dtype)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for left_out in ((3,), (4,), (3, 4)):
        out = [None if i in left_out else torch.full_like(x, float("nan")) for i, x in enumerate(want)]
        at = [0 if x is None else x.data_ptr() for x in out]
        la._call("la_gated_delta_backward", q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), 0 if dtype == torch.bfloat16 else 1,
                 alpha.data_ptr(), beta.data_ptr(), S0.data_ptr(), B, H, Hk, T, r, dv, 0.2, dy.data_ptr(), dS_T.data_ptr(), *at[:3],
                 at[3] or None, at[4] or None, at[5], ws.data_ptr(), need)
        assert la.last_device_status() == 0
        for x, z in zip(out, want):
            assert x is None or torch.equal(x, z), left_out


def test_repeated_calls_and_workspaces(la):  # noqa: F811
    """A workspace full of NaN and a captured call give the same bits."""
    for dtype in (torch.bfloat16, torch.float32):
        size = (2, 4, 2, 200, 128, 128)
        q, k, v, dy, alpha, beta, S0, dS_T = make(*size, dtype, True, 76)
        alpha[:, :, ::11] = 1e-20
        first = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T)
        ws = torch.full((la.gated_delta_backward_workspace_bytes(*size, dtype=dtype),), 255, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, workspace=ws)
        for _ in range(2):
            graph.replay()
            for x, z in zip(first, held):
                assert torch.equal(x, z)
