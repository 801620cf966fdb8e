"""A row's scores among other numbers of rows: the number decides how many CTAs share a row, so bits may differ and the bounds are those of
test_gpu_logprobs; which tokens are best, and in which order, may not."""
import pytest
import torch

from test_gpu_logprobs import DTYPES, check_grad, la, make, near  # noqa: F401  (la: the fixture)

pytestmark = pytest.mark.gpu


@DTYPES
@pytest.mark.parametrize("V,top", [(3001, 5), (32000, 32), (500, 0)])
def test_a_row_among_others(la, V, top, dtype):  # noqa: F811
    x, tokens = make(400, V, dtype, V)
    tokens[tokens < 0] = 3
    full = la.token_logprobs(x, tokens, top=top)
    for n in (1, 2, 30, 60, 80, 151, 153, 200, 303, 305):          # eight CTAs per row down to one
        some = la.token_logprobs(x[:n], tokens[:n], top=top)
        again = la.token_logprobs(x[:n].flip(0).contiguous(), tokens[:n].flip(0).contiguous(), top=top)
        for a, b in zip(some, again):
            assert torch.equal(a, b.flip(0)), n                     # (the same number of rows: the same bits in any order)
        assert torch.equal(some[4], full[4][:n]), n
        for got, want, tol, what in zip(some[:4], full[:4], (2.0 ** -20, 2.0 ** -19, 2.0 ** -20, 2.0 ** -20), ("logprob", "entropy", "lse", "alternatives")):
            near(got, want[:n].cpu().double(), 2 * tol, f"{what} of {n}")     # (each is off by as much from the exact one)
    assert la.last_device_status() == 0


@DTYPES
@pytest.mark.parametrize("N,V,left", [(1, 32003, 7), (600, 20000, 40), (5, 9000, 1)])
def test_mostly_masked_rows(la, N, V, left, dtype):  # noqa: F811
    """Rows of which a few tokens are allowed, anywhere in them, the others -infinity: scores, alternatives and gradient."""
    import gdelta_reference as R
    x, tokens = make(N, V, dtype, 51)
    g = torch.Generator().manual_seed(6)
    keep = torch.stack([torch.randperm(V, generator=g)[:left] for _ in range(N)]).cuda()
    mask = torch.ones((N, V), dtype=torch.bool, device="cuda").scatter_(1, keep, False)
    x[mask] = -float("inf")
    tokens[:] = keep[:, 0].int()
    got = la.token_logprobs(x, tokens, top=8)
    assert la.last_device_status() == 0
    ref = R.score(x, tokens.cpu(), 8)
    for a, b, tol, what in zip(got[:4], ref[:4], (2.0 ** -20, 2.0 ** -19, 2.0 ** -20, 2.0 ** -20), ("logprob", "entropy", "lse", "alternatives")):
        near(a, b, tol, what)
    assert torch.equal(got[4].cpu(), ref[4])
    few = slice(0, min(N, 20))
    dlp, dent = torch.randn(N, generator=g).cuda(), torch.randn(N, generator=g).cuda()
    d = la.token_logprobs_backward(x, tokens, got[2], got[1], dlp, dent)
    check_grad(d[few], x[few], tokens[few], dlp[few], dent[few])
    assert not d[mask].any()
