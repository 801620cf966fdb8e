"""Token log-probabilities on the GPU against their 64-bit definition.

Tolerances.  A log-probability is (x_token - m) - log s in FP32: m and x are the inputs, s a sum of exponentials whose own errors
(2^-22 each, and their sums' roundings) are relative, so log s is off by 2^-21 and the result by that and half a step of
each difference, 2^-24 of its terms.  The entropy is log s - sum a 2^a / s: its terms are at most a few units, 2^-20 in all.
lse adds half a step of its size.  The gradient is p (c0 + dH log p): p is off by 2^-22, by 2^-24 of |x - lse| log2 e, up to 2^-18 of
p at |x - lse| = 40, and by the half step of the lse that is passed, 2^-24 of its size (no more than 128: rows further off
are summed again); BF16 outputs by half a step of their own."""
import math

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


DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


def near(got, ref, tol, what):
    got = got.cpu().double()
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    err = torch.where(same, 0.0, (got - ref).abs())
    bound = tol * (1 + ref.abs())
    bad = ~(err <= torch.where(torch.isfinite(ref), bound, 0.0))
    assert not bad.any(), (what, got[bad][:4], ref[bad][:4])


def check_score(la, logits, tokens, top):
    got = la.token_logprobs(logits, tokens, top=top)
    assert la.last_device_status() == 0
    ref = R.score(logits, tokens.cpu(), top)
    near(got[0], ref[0], 2.0 ** -20, "logprob")
    near(got[1], ref[1], 2.0 ** -19, "entropy")
    near(got[2], ref[2], 2.0 ** -20, "lse")
    assert torch.equal(got[4].cpu(), ref[4]), "tokens"
    near(got[3], ref[3], 2.0 ** -20, "alternatives")
    return got


def make(N, V, dtype, seed, sd=3.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((N, V + pad), generator=g) * sd).to(dtype).cuda()[:, :V]
    tokens = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    if N > 2:
        tokens[1] = -1
    return x, tokens.cuda()


@DTYPES
@pytest.mark.parametrize("N,V,top", [(1, 1, 1), (1, 1, 4), (3, 2, 3), (1, 7, 0), (5, 100, 8), (2, 255, 20), (2, 257, 32), (1, 2048, 32),
                                     (1, 32003, 5), (4, 32000, 1), (700, 1000, 8), (310, 8191, 5), (1, 200003, 32)])
def test_score(la, N, V, top, dtype):
    check_score(la, *make(N, V, dtype, N + V), top)


@DTYPES
@pytest.mark.parametrize("pad", [1, 8, 13])
def test_padded_rows_and_offsets(la, pad, dtype):
    x, tokens = make(9, 1000, dtype, 5, pad=pad)
    a = check_score(la, x, tokens, 5)
    b = la.token_logprobs(x.contiguous(), tokens, top=5)
    assert torch.equal(a[4], b[4])
    x, tokens = make(1, 1001, dtype, 6)
    check_score(la, x[:, 1:], (tokens - 1).clamp(min=0), 5)      # a row that starts off a 16-byte boundary


@DTYPES
@pytest.mark.parametrize("V", [300, 5000, 70001])
def test_ties_go_to_the_lower_index(la, V, dtype):
    """Rows of one value, of two, and ascending and descending ones: more equal logits than any buffer holds."""
    rows = torch.zeros((6, V))
    rows[1, V // 2:] = 1.0
    rows[2] = torch.arange(V) / V
    rows[3] = -torch.arange(V) / V
    rows[4, ::7] = 2.0
    rows[5, -1] = 3.0
    tokens = torch.tensor([0, V - 1, 5, 5, 7, 0], dtype=torch.int32).cuda()
    for top in (1, 8, 32):
        check_score(la, rows.to(dtype).cuda(), tokens, top)


@DTYPES
def test_masks_and_odd_values(la, dtype):
    """-infinity, the type's lowest value, rows with nothing left, NaN, +infinity, huge and tiny logits."""
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(3)
    x = torch.randn((12, 500), generator=g)
    x[0, 3:] = -math.inf            # three left
    x[1] = -math.inf                # none
    x[2, 100:] = low
    x[3] = low
    x[4, 7] = math.nan
    x[5, 9] = math.inf
    x[6] *= 1e4
    x[7] *= 1e-30
    x[8] += 1e4
    x[9, 1:] = -math.inf            # one left: probability one, entropy zero
    x[10, ::2] = -math.inf
    x[11] = -0.0
    x[11, 250] = 0.0
    tokens = torch.tensor([1, 2, 3, 4, 5, 6, 7, 8, 9, 0, 4, 0], dtype=torch.int32).cuda()
    x = x.to(dtype).cuda()
    got = check_score(la, x, tokens, 8)
    assert float(got[0][9]) == 0.0 and float(got[1][9]) == 0.0
    dlp, dent = torch.randn(12, generator=g).cuda(), torch.randn(12, generator=g).cuda()
    d = la.token_logprobs_backward(x, tokens, got[2], got[1], dlp, dent)
    fine = [i for i in range(12) if i not in (4, 5)]
    check_grad(d[fine], x[fine], tokens[fine], dlp[fine], dent[fine])
    assert torch.isnan(d[4]).all() and torch.isnan(d[5]).all()


def test_tokens_out_of_range(la):
    x, tokens = make(4, 100, torch.float32, 8)
    tokens[0], tokens[2] = 100, -7
    got = la.token_logprobs(x, tokens, top=2)
    assert la.last_device_status() == 2 and la.last_device_status() == 0
    for i in (0, 1, 2):
        assert float(got[0][i]) == 0 and float(got[1][i]) == 0 and float(got[2][i]) == 0 and (got[4][i] == -1).all()
    d = la.token_logprobs_backward(x, tokens, got[2], got[1], torch.ones(4, device="cuda"))
    assert la.last_device_status() == 2
    assert not d[:3].any() and d[3].any()


def test_rows_do_not_depend_on_the_batch(la):
    """A row's results have the same bits alone and among others of the same launch shape; padding rows are not read."""
    x, tokens = make(400, 3001, torch.bfloat16, 12)
    full = la.token_logprobs(x, tokens, top=4)
    x[1] = float("nan")             # (token -1)
    perm = torch.randperm(400, generator=torch.Generator().manual_seed(1)).cuda()
    again = la.token_logprobs(x[perm].contiguous(), tokens[perm].contiguous(), top=4)
    for a, b in zip(full, again):
        assert torch.equal(a[perm], b)


def check_grad(got, logits, tokens, dlp, dent):
    ref = R.score_backward(logits, tokens.cpu(), dlp.cpu(), None if dent is None else dent.cpu())
    got_d = got.cpu().double()
    own = R.U16 if got.dtype == torch.bfloat16 else R.U32
    # p (|dlp| + |dent| (|log p| + H)), the terms that the roundings are relative to
    x = logits.cpu().double()
    lse = torch.logsumexp(x, 1, keepdim=True).abs().clamp(max=128).nan_to_num()
    lp = torch.log_softmax(x, 1)
    p = lp.exp().nan_to_num()
    H = -torch.where(p > 0, p * lp, 0.0).sum(1, keepdim=True)
    lp = lp.clamp(min=-200).nan_to_num()
    size = p * (dlp.cpu().double().abs()[:, None] + (0.0 if dent is None else dent.cpu().double().abs()[:, None] * (lp.abs() + H)))
    bound = own * ref.abs() + (2.0 ** -19 + 2.0 ** -23 * lp.abs() + 2.0 ** -24 * lse) * (size + (torch.arange(x.shape[1])[None] == tokens.cpu()[:, None]) * dlp.cpu().double().abs()[:, None]) + 1e-37
    assert ((got_d - ref).abs() <= bound).all(), float(((got_d - ref).abs() / bound).max())


@DTYPES
@pytest.mark.parametrize("N,V", [(1, 1), (3, 7), (2, 257), (5, 32003), (40, 16384), (7, 20001)])
@pytest.mark.parametrize("entropy", [False, True], ids=["logprob", "entropy"])
def test_gradient(la, N, V, entropy, dtype):
    x, tokens = make(N, V, dtype, N + V)
    _, ent, lse, _, _ = la.token_logprobs(x, tokens)
    g = torch.Generator().manual_seed(9)
    dlp, dent = torch.randn(N, generator=g).cuda(), torch.randn(N, generator=g).cuda() if entropy else None
    d = la.token_logprobs_backward(x, tokens, lse, ent if entropy else None, dlp, dent)
    check_grad(d, x, tokens, dlp, dent)
    if N > 2:
        assert not d[1].any()
    place = x.clone()
    assert la.token_logprobs_backward(place, tokens, lse, ent, dlp, dent, dlogits=place) is place and torch.equal(place, d)
    wide = torch.full((N, V + 3), 5.0, device="cuda", dtype=dtype)
    la.token_logprobs_backward(x, tokens, lse, ent, dlp, dent, dlogits=wide[:, :V])
    assert (wide[:, V:] == 5.0).all()
    check_grad(wide[:, :V], x, tokens, dlp, dent)


@DTYPES
def test_rows_past_32_bits(la, dtype):
    """Rows whose elements lie more than 2^31 behind the first."""
    V, far = 1000, (1 << 31) + 24
    x, tokens = make(3, V, dtype, 31)
    tokens[1] = 7
    buf = torch.empty(2 * far + V, dtype=dtype, device="cuda")
    rows = buf.as_strided((3, V), (far, 1))
    rows.copy_(x)
    want, got = la.token_logprobs(x, tokens, top=3), la.token_logprobs(rows, tokens, top=3)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    dlp = torch.ones(3, device="cuda")
    d = la.token_logprobs_backward(x, tokens, want[2], None, dlp)
    la.token_logprobs_backward(rows, tokens, want[2], None, dlp, dlogits=rows)
    assert torch.equal(rows, d)


def test_gradient_differences(la):
    x, tokens = make(6, 50, torch.float32, 4, sd=1.0)
    g = torch.Generator().manual_seed(2)
    dlp, dent, d = torch.randn(6, generator=g), torch.randn(6, generator=g), torch.randn((6, 50), generator=g)

    def loss(z):
        lp, ent, _, _, _ = la.token_logprobs(z, tokens)
        return float((lp.double().cpu() * dlp.double()).sum() + (ent.double().cpu() * dent.double()).sum())

    _, ent, lse, _, _ = la.token_logprobs(x, tokens)
    got = la.token_logprobs_backward(x, tokens, lse, ent, dlp.cuda(), dent.cuda())
    h = 2.0 ** -6
    slope = (loss(x + h * d.cuda()) - loss(x - h * d.cuda())) / (2 * h)
    want = float((got.cpu().double() * d.double()).sum())
    # h^2 / 6 of the third derivative: at most a few units per row times |d|^3 averaged over p, and 2^-20 / h of the outputs
    assert abs(slope - want) <= 2.0 ** -12 * 6 * 10 + 2.0 ** -13 * 6


def test_streams_graphs_and_no_rows(la):
    x, tokens = make(50, 3000, torch.bfloat16, 21)
    new, _ = make(50, 3000, torch.bfloat16, 22)

    def calls():
        lp, ent, lse, best, which = la.token_logprobs(x, tokens, top=5)
        return [lp, ent, lse, best, which, la.token_logprobs_backward(x, tokens, lse, ent, lp, ent)]

    calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = calls()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(on_side, calls()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    x.copy_(new)
    graph.replay()
    for a, b in zip(held, calls()):
        assert torch.equal(a, b)
    empty = la.token_logprobs(x[:0], tokens[:0], top=3)
    assert empty[3].shape == (0, 3)
    assert la.token_logprobs_backward(x[:0], tokens[:0], empty[2], empty[1], empty[0]).shape == (0, 3000)


def test_scores_agree_with_the_beam_choice(la):
    """One beam's best continuations are the row's best alternatives."""
    x, _ = make(6, 5000, torch.float32, 31)
    scores = torch.zeros((6, 1), device="cuda")
    nxt, _, tok, _ = la.beam_select(x.view(6, 1, 5000), scores)
    lp, _, _, best, which = la.token_logprobs(x, tok.view(6).contiguous(), top=1)
    assert torch.equal(which, tok) and torch.allclose(best, nxt, atol=1e-5) and torch.allclose(lp, nxt[:, 0], atol=1e-5)
