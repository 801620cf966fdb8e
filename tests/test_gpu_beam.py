"""Beam selection and state reordering on the GPU against plain references.

Choices are whole numbers and have to be equal: the reference ranks candidates in 64 bits,
equal ones by the lower beam, then the lower token.  Scores are FP32 results of 64-bit sums
whose log-sum-exp carries the FP32 exponentials' error: 4 U32 relative in the sum (2 ulp
each and its argument's rounding up to |x - max| <= 64: 64 U32 absolute in the worst term), so
they are held to 80 U32 + U32 |score|."""
import pytest
import torch

import decay_reference as R

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def la():
    from recurrent_state_02_gb300 import build
    build.build()
    import recurrent_state_02_gb300 as la_mod
    assert torch.cuda.is_available()
    return la_mod


def check(la, logits, scores, done=None, eos=-1):
    got = la.beam_select(logits, scores, done=done, eos=eos)
    ref = R.select(logits, scores, None if done is None else done.cpu(), eos)
    for g, r, name in zip(got[1:], ref[1:], ("parents", "tokens", "done")):
        assert torch.equal(g.cpu(), r), (name, g, r)
    fine = torch.isfinite(ref[0])
    s = got[0].cpu().double()
    assert torch.equal(torch.isfinite(s), fine) and (s[~fine] == -INF).all()
    assert ((s - ref[0]).abs()[fine] <= 80 * R.U32 + R.U32 * ref[0].abs()[fine]).all()
    return got


def make(B, K, V, dtype, seed, sd=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn((B, K, V), generator=g) * sd).to(dtype).cuda()
    scores = (-5 - 3 * torch.rand((B, K), generator=g)).cuda()
    return logits, scores


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 1, 5), (2, 4, 3), (1, 3, 17), (3, 2, 1000), (1, 5, 32003), (2, 4, 8192),
                                  (200, 3, 257), (2, 32, 500), (1, 12, 2049), (2, 7, 4095), (1, 31, 9)],
                         ids=lambda s: "x".join(map(str, s)))
def test_select(la, size, dtype):
    check(la, *make(*size, dtype, sum(size)))


@pytest.mark.parametrize("K", [1, 5, 32])
@pytest.mark.parametrize("B", [33, 38, 44, 53, 66, 88, 89, 153])
def test_select_batches(la, B, K):
    """Batches on every number of CTAs per request (8 to 2), with as many parts per row as fit or one."""
    check(la, *make(B, K, 300 if K < 32 else 70, torch.bfloat16, B + K))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
def test_select_padded_and_misaligned_rows(la, offset, dtype):
    """Rows of a padded vocabulary at every alignment; what lies between them is NaN."""
    B, K, V, ld = 2, 3, 1501, 1501 + 2 * offset + 3
    x, scores = make(B, K, V, dtype, 20 + offset)
    buf = torch.full((B * K * ld + offset,), float("nan"), device="cuda", dtype=dtype)
    rows = buf[offset:].view(B, K, ld)
    rows[..., :V] = x
    got = check(la, rows[..., :V], scores)
    want = la.beam_select(x, scores)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_select_ties(la, dtype):
    """Equal candidates go to the lower beam, then the lower token, whatever the order of the work."""
    B, K, V = 3, 5, 3001
    logits = torch.zeros((B, K, V), device="cuda", dtype=dtype)
    scores = torch.full((B, K), -2.0, device="cuda")
    _, parents, tokens, _ = check(la, logits, scores)
    assert (parents == 0).all() and torch.equal(tokens.cpu(), torch.arange(K, dtype=torch.int32).expand(B, K))
    logits[:, :, ::7] = 1.5      # few distinct values, far apart and in several beams
    logits[:, 2, 2990:] = 2.0
    logits[:, 4, 2990:] = 2.0
    check(la, logits, scores)
    logits = torch.where(torch.rand((B, K, V), generator=torch.Generator().manual_seed(3)).cuda() < 0.5, 0.0, -0.0).to(dtype)
    check(la, logits, scores)   # -0 and +0 are equal
    up = torch.arange(V, device="cuda").float().expand(B, K, V).to(dtype).contiguous() / 64
    check(la, up, scores)       # ascending: every block beats the last


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_select_masks(la, dtype):
    """Masked tokens, rows with nothing left, the type's lowest value, infinities and NaN."""
    B, K, V = 2, 4, 700
    low = torch.finfo(dtype).min
    x, scores = make(B, K, V, dtype, 31)
    x[:, :, 5:] = -INF                     # five tokens left in every beam
    check(la, x, scores)
    x[0, 1] = -INF                         # a beam with none
    x[1, :, 1:] = -INF                     # fewer candidates than slots once beams drop out
    x[1, 2, 0] = -INF
    got = check(la, x, scores)
    assert got[0][1, 3] == -INF and got[1][1, 3] == 3 and got[2][1, 3] == 0
    x[:] = -INF
    got = check(la, x, scores)
    assert (got[0] == -INF).all() and torch.equal(got[1].cpu(), torch.arange(K, dtype=torch.int32).expand(B, K))
    x, scores = make(B, K, V, dtype, 32)
    x[0, 0, 3] = float("nan")
    x[0, 1, 9] = INF
    x[1, 2, 690] = float("nan")
    got = check(la, x, scores)             # beams with a NaN or +inf drop out
    assert (got[1][0] >= 2).all() and (got[1][1] != 2).all()
    x, scores = make(B, K, V, dtype, 33)
    x[:, :, 100:] = low                    # masks of the lowest finite value
    check(la, x, scores)
    x, scores = make(B, K, V, dtype, 34)
    scores[0, 1:] = -INF                   # the first step: one live beam
    scores[1, 0] = float("nan")
    got = check(la, x, scores)
    assert (got[1][0] == 0).all() and (got[1][1] > 0).all()


def test_select_ended_beams(la):
    B, K, V = 4, 4, 900
    x, scores = make(B, K, V, torch.bfloat16, 41)
    done = torch.zeros((B, K), dtype=torch.uint8, device="cuda")
    done[0, 1] = 1
    done[1] = 1
    done[2, 0] = done[2, 3] = 3            # any non-zero value
    x[3, :, 7] = 30.0                      # eos wins everywhere
    x[2, 0] = float("nan")                 # an ended beam's logits are not read
    got = check(la, x, scores, done=done, eos=7)
    assert (got[2][1] == 7).all() and (got[3][1] == 1).all() and torch.equal(got[0][1], scores[1].sort(descending=True).values)
    assert (got[3][3] == 1).all()
    # in place: scores and done may be their own outputs
    s, d = scores.clone(), done.clone()
    out = la.beam_select(x, s, done=d, eos=7, next_scores=s, done_out=d)
    assert torch.equal(out[0], got[0]) and torch.equal(out[3], got[3]) and out[0].data_ptr() == s.data_ptr()


def test_select_refusals(la):
    x, scores = make(2, 3, 50, torch.float32, 51)
    with pytest.raises(ValueError):
        la.beam_select(x.transpose(0, 1), scores)
    with pytest.raises(ValueError):
        la.beam_select(x[..., ::2], scores)
    with pytest.raises(ValueError):
        la.beam_select(x.double(), scores)
    with pytest.raises(ValueError):
        la.beam_select(x, scores[:, :2])
    with pytest.raises(la.LinAttnError):
        la.beam_select(x, scores, eos=50)
    with pytest.raises(la.LinAttnError):
        la.beam_select(x, scores, done=torch.zeros((2, 3), dtype=torch.uint8, device="cuda"))
    with pytest.raises(la.LinAttnError):
        la.beam_select(torch.zeros((1, 33, 50), device="cuda"), torch.zeros((1, 33), device="cuda"))


@pytest.mark.parametrize("norm", [False, True], ids=["S", "Sz"])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1), (1, 4, 2, 64, 64), (3, 5, 3, 33, 7), (2, 9, 2, 128, 128), (2, 17, 1, 16, 20),
                                  (1, 32, 2, 8, 3), (5, 4, 16, 128, 64)], ids=lambda s: "x".join(map(str, s)))
def test_reorder(la, size, norm):
    B, K, H, r, dv = size
    g = torch.Generator().manual_seed(sum(size))
    S = torch.randn((B * K, H, r, dv), generator=g).cuda()
    z = torch.randn((B * K, H, r), generator=g).cuda() if norm else None
    for parents in (torch.randint(0, K, (B, K), generator=g), torch.arange(K).expand(B, K),
                    torch.arange(K).roll(1).expand(B, K), torch.full((B, K), K - 1)):
        parents = parents.int().contiguous().cuda()
        at = (torch.arange(B, device="cuda")[:, None] * K + parents).reshape(-1).long()
        So, zo = la.state_reorder(S, parents, z=z, S_out=torch.full_like(S, 3.0))
        assert torch.equal(So, S[at]) and (z is None or torch.equal(zo, z[at]))
        S2, z2 = S.clone(), None if z is None else z.clone()
        out = la.state_reorder(S2, parents, z=z2)
        assert out[0] is S2 and torch.equal(S2, S[at]) and (z is None or torch.equal(z2, z[at]))
        # off its 16-byte boundary
        S3 = torch.empty(S.numel() + 1, device="cuda")[1:].view(S.shape).copy_(S)
        la.state_reorder(S3, parents)
        assert torch.equal(S3, S[at])
    assert la.last_device_status() == 0


def test_reorder_bad_parents_are_recorded(la):
    S = torch.randn((4, 2, 8, 8), device="cuda")
    parents = torch.tensor([[1, 4, -1, 0]], dtype=torch.int32, device="cuda")
    out = S.clone()
    la.state_reorder(out, parents)
    assert la.last_device_status() == 2 and la.last_device_status() == 0
    assert torch.equal(out, torch.stack([S[1], S[1], S[2], S[0]]))


def test_reorder_refusals(la):
    S, z = torch.zeros((4, 2, 8, 8), device="cuda"), torch.zeros((4, 2, 8), device="cuda")
    parents = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        la.state_reorder(S, parents.long())
    with pytest.raises(ValueError):
        la.state_reorder(S, parents[:, :3].contiguous())
    with pytest.raises(ValueError):
        la.state_reorder(S, parents, z_out=z)
    with pytest.raises(ValueError):
        la.state_reorder(S, parents, z=z, z_out=z)
    with pytest.raises(la.LinAttnError):
        la.state_reorder(torch.zeros((33, 1, 2, 2), device="cuda"), torch.zeros((1, 33), dtype=torch.int32, device="cuda"))


def test_graph_replay(la):
    """Captured and replayed on new logits; two graphs share nothing."""
    x, scores = make(3, 4, 5000, torch.bfloat16, 61)
    S = torch.randn((12, 2, 16, 16), device="cuda")
    first = S.clone()
    la.beam_select(x, scores)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = la.beam_select(x, scores)
            la.state_reorder(S, o[1])
        graphs.append(g)
        outs.append(o)
    for seed in (62, 63):
        x.copy_(make(3, 4, 5000, torch.bfloat16, seed)[0])
        want = R.select(x, scores, None, -1)
        for g, o in zip(graphs, outs):
            S.copy_(first)
            g.replay()
            torch.cuda.synchronize()
            at = (torch.arange(3)[:, None] * 4 + want[1]).reshape(-1).long().cuda()
            assert torch.equal(o[1].cpu(), want[1]) and torch.equal(o[2].cpu(), want[2]) and torch.equal(S, first[at])


@pytest.mark.parametrize("kind", ["decay", "normalised"])
def test_beam_search(la, kind):
    """Prompt, then a beam search: decode, logits, choose, move the states.  Each chosen sequence's score equals the sum
    of log-probabilities along it, recomputed by the prefill of prompt and answer together (so the states
    followed their beams), and no slot appears twice."""
    B, K, H, d, V, P, steps = 2, 4, 2, 128, 211, 40, 6
    g = torch.Generator().manual_seed(71)
    table = (torch.randn((3, V, H, d), generator=g)).cuda()            # q, k, v of every token
    head = (torch.randn((H * d, V), generator=g) * 0.3).cuda()
    decay = torch.tensor([0.9, 0.99]).cuda()
    prompt = torch.randint(0, V, (B, P), generator=g).cuda()

    def qkv(tokens):                                                    # [N, T] -> [N,H,T,d]
        return [table[i][tokens].transpose(1, 2).contiguous() for i in range(3)]

    def run(tokens):
        q, k, v = qkv(tokens)
        if kind == "decay":
            return la.decay_prefill(q, k, v, decay, scale=d ** -0.5) + (None,)
        y, S, z = la.prefill_chunked(q, k, v)
        return y, S, z

    def logits_of(y):                                                   # [N,H,1,d]
        return (y.reshape(y.shape[0], -1) @ head)

    y, S, z = run(prompt)
    x = logits_of(y[:, :, -1:])[:, None].expand(B, K, V).contiguous()
    scores = torch.full((B, K), -INF, device="cuda")
    scores[:, 0] = 0.0                                                  # one live beam at first
    S = S.repeat_interleave(K, 0)
    z = None if z is None else z.repeat_interleave(K, 0)
    beams = torch.zeros((B, K, 0), dtype=torch.long, device="cuda")
    for _ in range(steps):
        scores, parents, tokens, _ = la.beam_select(x, scores)
        la.state_reorder(S, parents, z=z)
        beams = torch.cat([beams.gather(1, parents.long()[..., None].expand(-1, -1, beams.shape[2])), tokens.long()[..., None]], 2)
        q, k, v = qkv(tokens.reshape(B * K, 1).long())
        if kind == "decay":
            y = la.decay_decode_step(q, k, v, decay, S, scale=d ** -0.5)
        else:
            y = la.decode_step(q, k, v, S, z)
        x = logits_of(y).view(B, K, V)
    assert la.last_device_status() == 0
    assert all(len({tuple(r) for r in rows.tolist()}) == K for rows in beams)
    whole = torch.cat([prompt[:, None].expand(B, K, P), beams], 2).reshape(B * K, -1)
    y, _, _ = run(whole)
    lp = torch.log_softmax((y.transpose(1, 2).reshape(B * K, P + steps, H * d).double() @ head.double()), -1)
    total = lp[:, P - 1:-1].gather(2, beams.reshape(B * K, steps, 1)).sum((1, 2)).view(B, K)
    # FP32 throughout: logits are sums of H d products of size about 1, each carrying about 1e-5
    assert ((total - scores.double()).abs() <= steps * 1e-3).all()
    assert (scores[:, :-1] >= scores[:, 1:]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("level", ["low", "high", -1e30, 1e25, 1e9])
def test_select_rows_of_huge_logits(la, level, dtype):
    """Rows whose logits all lie near one huge value, masks of the type's lowest among them: their log-probabilities are
    those of the differences, log(1 / V) for a constant row, and do not vanish next to the value.  (Bound: the
    module's; the differences here are 0 or beyond the exponential's range.)"""
    B, K, V = 2, 3, 611
    level = {"low": torch.finfo(dtype).min, "high": torch.finfo(dtype).max}.get(level, level)
    x, scores = make(B, K, V, dtype, 71)
    x[0, 1] = level                            # one beam of three
    x[1] = level                               # every beam
    scores[0, 1] = scores[0].max() + 6.0       # log 611 = 6.4: near the other beams' best
    scores[1] = torch.tensor([-3.0, -1.0, -1.0], device="cuda")
    next_scores, parents, tokens, _ = la.beam_select(x, scores)
    lp = torch.log_softmax(x.double().cpu(), 2)
    cand = (scores.double().cpu()[..., None] + lp).reshape(B, -1)
    best = torch.sort(cand, dim=1, descending=True, stable=True)
    assert torch.equal(parents.cpu().long() * V + tokens.cpu(), best.indices[:, :K])
    want = best.values[:, :K]
    assert ((next_scores.double().cpu() - want).abs() <= 80 * R.U32 + R.U32 * want.abs()).all()
    assert parents[1].tolist() == [1, 1, 1] and tokens[1].tolist() == [0, 1, 2]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [1, 3, 7, 8, 9, 250, 2049, 2050, 2051, 2052, 2053, 2054, 2055, 2056, 40961])
def test_select_rows_that_end_inside_a_granule(la, V, dtype):
    """Rows that start on 16-byte boundaries and end anywhere, the last one with the buffer: the padding between them would
    win, and the best tokens are a row's last ones."""
    B, K = 2, 3
    ld = (V + 8) // 8 * 8
    buf = torch.full(((B * K - 1) * ld + V,), 99.0, device="cuda", dtype=dtype)
    rows = buf.as_strided((B, K, V), (K * ld, ld, 1))
    x, scores = make(B, K, V, dtype, 80 + V)
    x[..., -3:] += 9.0
    rows.copy_(x)
    got = check(la, rows, scores)
    want = la.beam_select(x, scores)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_select_many_beams_over_a_large_vocabulary(la, dtype):
    """32 beams whose candidates fill every warp's buffer again and again: ascending rows, where each block beats the
    last, rows of few distinct values, and random ones."""
    B, K, V = 2, 32, 32768
    x, scores = make(B, K, V, dtype, 90)
    scores[:] = -5.0 - torch.arange(K, device="cuda") * 0.25
    up = torch.arange(V, device="cuda").float() / 64        # BF16: runs of equal values
    x[0, ::2] = up.to(dtype)
    x[1, 1::2] = (torch.arange(V, device="cuda") % 5).to(dtype)
    got = la.beam_select(x, scores)
    cand = (scores.double()[..., None] + torch.log_softmax(x.double(), 2)).reshape(B, -1)
    # 64-bit scores of equal candidates differ in their last bits by the row: the choice is compared by score
    best = torch.sort(cand, dim=1, descending=True).values[:, :K]
    mine = cand.gather(1, got[1].long() * V + got[2].long())
    assert ((mine - best).abs() <= 80 * R.U32).all()
    assert ((got[0].double() - best).abs() <= 80 * R.U32 + R.U32 * best.abs()).all()
    for b in range(B):
        chosen = list(zip(got[1][b].tolist(), got[2][b].tolist()))
        assert len(set(chosen)) == K
        for k in range(K):      # within a beam: its best logits, equal ones by the lower token
            mine_k = [t for p, t in chosen if p == k]
            order = torch.sort(x[b, k].double(), descending=True, stable=True).indices[:len(mine_k)].tolist()
            assert sorted(mine_k) == sorted(order)
