"""The gated delta rule over ranges that test_gpu_gated_delta does not reach: packed batches on both sides of what plans itself and of what the plan
ranks, skipped sequences among them, gradients of many more chunks than SMs, write strengths up to beta |k|^2 = 2 and keys of any length, and
long sequences of few heads at full width."""
import pytest
import torch

import gdelta_reference as R
from test_gpu_gated_delta import DTYPES, ids, la, make  # noqa: F401  (la: the fixture)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def bh(x, s):
    return x[s].transpose(0, 1)[None]


def packed(lens, H, Hk, r, dv, seed, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q, k, v, _, alpha, beta, _, _ = make(1, H, Hk, cu[-1], r, dv, dtype, False, seed, layout="tok")
    S0 = torch.randn((len(lens), H, r, dv), generator=g).mul(0.3).cuda()
    return (q, k, v, alpha, beta, S0), cu


def check_packed(args, cu, y, S, which, scale, dtype=BF):
    q, k, v, alpha, beta, S0 = args
    for b in which:
        s = slice(cu[b], cu[b + 1])
        ref_y, ref_S, _, _ = R.prefill(*(bh(x, s) for x in (q, k, v, alpha, beta)), S0[b:b + 1], scale)
        R.check(S[b:b + 1], ref_S, dtype, f"S {b}", cu[b + 1] - cu[b])
        R.check(bh(y, s), ref_y, dtype, f"y {b}", cu[b + 1] - cu[b])


def lengths(B, seed):
    """Lengths of every kind: none, one token, equal ones in a row, chunks that are full and not."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 41 if B > 100 else 150, (B,), generator=g)
    lens[::5] = 0
    lens[1::7] = 64
    lens[2::9] = 1
    lens[B // 2] = 333
    lens[-1] = 65
    return lens.tolist()


@pytest.mark.parametrize("B", [31, 32, 33, 48, 1023, 1024, 1025])
def test_packed_plans(la, B):  # noqa: F811
    """Batches that plan themselves, that the plan ranks, and that it does not; every sequence whatever its rank."""
    lens = lengths(B, B)
    (q, k, v, alpha, beta, S0), cu = packed(lens, 4, 2, 64, 64, B)
    S_in = S0.clone()
    y, S = la.gated_delta_prefill_varlen(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), alpha, beta, S0=S_in, scale=0.3, S_out=S_in)
    assert la.last_device_status() == 0
    some = range(B) if B <= 64 else sorted({0, 1, 2, 5, 7, 31, 32, 33, B // 2, B // 2 + 1, 1000, 1022, B - 2, B - 1})
    check_packed((q, k, v, alpha, beta, S0), cu, y, S, some, 0.3)
    empty = torch.tensor([n == 0 for n in lens]).cuda()
    assert torch.equal(S[empty], S0[empty])
    # the others by comparison: sequences run alone have the same bits
    for b in range(0, B, 1 + B // 40):
        s = slice(cu[b], cu[b + 1])
        if lens[b]:
            one = torch.tensor([0, lens[b]], dtype=torch.int32, device="cuda")
            y1, S1 = la.gated_delta_prefill_varlen(*(x[s].contiguous() for x in (q, k, v)), one, *(x[s].contiguous() for x in (alpha, beta)),
                                                   S0=S0[b:b + 1].contiguous(), scale=0.3)
            assert torch.equal(y[s], y1) and torch.equal(S[b:b + 1], S1), b


@pytest.mark.parametrize("B", [5, 32, 33, 40, 1100])
def test_skipped_sequences(la, B):  # noqa: F811
    """Sequences outside the batch or of negative length, first, in the middle and last: skipped and recorded, the others as without them."""
    n, H, r, dv = 70, 2, 64, 64
    total = B * n
    q, k, v, _, alpha, beta, _, _ = make(1, H, H, total, r, dv, BF, False, 17, layout="tok")
    cu = [b * n for b in range(B + 1)]
    cu[0] = -3                                  # the first begins before the batch
    cu[B // 2] = cu[B // 2 + 1] + 1             # the one before it reaches into its neighbour, and it has a negative length
    cu[B] = total + 1                           # the last ends behind the batch
    bad = [0, B // 2, B - 1]
    at = torch.tensor(cu, dtype=torch.int32, device="cuda")
    S = torch.full((B, H, r, dv), 3.0, device="cuda")
    y = torch.full((total, H, dv), 7.0, device="cuda", dtype=BF)
    la.gated_delta_prefill_varlen(q, k, v, at, alpha, beta, y=y, S_out=S)
    assert la.last_device_status() == 2 and la.last_device_status() == 0
    S0 = torch.zeros_like(S)
    for b in bad:
        assert (S[b] == 3.0).all()
    assert (y[:n] == 7.0).all() and (y[(B - 1) * n:] == 7.0).all()
    near = [B // 2 - 1, B // 2 + 1]             # (both write the row that they share)
    check_packed((q, k, v, alpha, beta, S0), cu, y, S, [b for b in sorted({1, B - 2, *range(2, B - 1, 1 + B // 10)}) if b not in bad + near], 1.0)
    for b in near:
        s = slice(cu[b], cu[b + 1])
        _, ref_S, _, _ = R.prefill(*(bh(x, s) for x in (q, k, v, alpha, beta)), None, 1.0)
        R.check(S[b:b + 1], ref_S, BF, f"S {b}", cu[b + 1] - cu[b])


@pytest.mark.parametrize("B", [4, 64, 2000])
def test_overlapping_sequences_stay_inside_the_workspace(la, B):  # noqa: F811
    """Every other bound goes back to 0: sequences that overlap, more chunks than the workspace holds.  What does not fit is left out and
    recorded; the first sequence, the memory behind the workspace and the next call are as they were."""
    T, H, r, dv = 1000, 1, 64, 64
    q, k, v, _, alpha, beta, _, _ = make(1, H, H, T, r, dv, BF, False, 19, layout="tok")
    cu = torch.tensor([(b % 2) * T for b in range(B + 1)], dtype=torch.int32, device="cuda")
    need = la.gated_delta_prefill_varlen_workspace_bytes(B, H, H, T, r, dv)
    room = torch.full((need + (1 << 20),), 90, dtype=torch.uint8, device="cuda")
    S = torch.full((B, H, r, dv), 3.0, device="cuda")
    y, S = la.gated_delta_prefill_varlen(q, k, v, cu, alpha, beta, S_out=S, workspace=room[:need])
    assert la.last_device_status() == 2
    assert (room[need:] == 90).all()
    assert (S[1::2] == 3.0).all()
    one = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y1, S1 = la.gated_delta_prefill_varlen(q, k, v, one, alpha, beta)
    assert la.last_device_status() == 0
    assert torch.equal(S[:1], S1) and torch.equal(y, y1)        # (all that run have the same tokens)


def test_nan_neighbours_of_planned_batches(la):  # noqa: F811
    lens = lengths(40, 3)
    (q, k, v, alpha, beta, S0), cu = packed(lens, 2, 2, 128, 128, 23)
    at = torch.tensor(cu, dtype=torch.int32, device="cuda")
    want_y, want_S = la.gated_delta_prefill_varlen(q, k, v, at, alpha, beta, S0=S0)
    bad = [b for b in (1, 8, 20, 39) if lens[b]]
    for x in (q, k, v, alpha, beta):
        for b in bad:
            x[cu[b]:cu[b + 1]] = float("nan")
    y, S = la.gated_delta_prefill_varlen(q, k, v, at, alpha, beta, S0=S0)
    for b in range(40):
        if b not in bad:
            assert torch.equal(S[b], want_S[b]) and torch.equal(y[cu[b]:cu[b + 1]], want_y[cu[b]:cu[b + 1]]), b


@pytest.mark.parametrize("size", [(2, 16, 16, 1001, 128, 128), (2, 16, 8, 1001, 128, 64), (3, 16, 16, 801, 64, 128), (2, 32, 8, 600, 64, 64),
                                  (1, 3, 3, 7001, 128, 128)], ids=ids)
def test_gradients_of_many_chunks(la, size):  # noqa: F811
    """More than twice as many chunks as SMs, and no multiple of them: every key head's gradients against the head alone (one chunk per
    CTA, the same bits), some of them against 64 bits, a poisoned workspace and a replayed graph."""
    B, H, Hk, T, r, dv = size
    q, k, v, dy, alpha, beta, S0, dS_T = make(*size, BF, True, 29)
    alpha[:, :, ::97] = 1e-10
    run = lambda ws=None: la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, scale=0.2, workspace=ws)  # noqa: E731
    first = run()
    ws = torch.full((la.gated_delta_backward_workspace_bytes(*size),), 255, dtype=torch.uint8, device="cuda")
    for a, b in zip(first, run(ws)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(ws)
    ws.fill_(255)
    graph.replay()
    for a, b in zip(first, held):
        assert torch.equal(a, b)
    assert la.last_device_status() == 0
    for b in range(B):
        for hk in range(Hk):
            one = lambda x: None if x is None else x[b:b + 1, hk * (x.shape[1] // Hk):(hk + 1) * (x.shape[1] // Hk)].contiguous()  # noqa: E731
            got = [one(x) for x in first]
            alone = la.gated_delta_backward(one(q), one(k), one(v), one(dy), one(alpha), one(beta), S0=one(S0), dS_T=one(dS_T), scale=0.2)
            for x, z, name in zip(got, alone, R.NAMES):
                assert torch.equal(x, z), (b, hk, name)
            if (b, hk) in ((0, 0), (B - 1, Hk - 1)):
                args = (one(q), one(k), one(v), one(dy), one(alpha), one(beta), one(S0), one(dS_T))
                ref, terms = R.backward(*args, 0.2)
                R.check_all(got, (ref, terms), BF, T)


@DTYPES
@pytest.mark.parametrize("size", [(1, 2, 1, 200, 128, 128), (1, 2, 2, 150, 64, 192), (1, 2, 2, 90, 33, 20)], ids=ids)
@pytest.mark.parametrize("norm,strength", [(1.0, 1.9), (0.25, 8.0), (3.0, 0.15), (1.0, 2.0)], ids=lambda x: str(x))
def test_write_strengths_and_key_lengths(la, size, norm, strength, dtype):  # noqa: F811
    """Write strengths up to beta |k|^2 = 2 and keys (and queries) of any length: a step is then a reflection at most, errors do not grow."""
    q, k, v, dy, alpha, beta, S0, dS_T = make(*size, dtype, True, 37)
    k, q = ((x.float() * norm).to(dtype) for x in (k, q))
    beta = beta * strength
    beta[:, 0, ::3] = strength * (0.99 if dtype == BF else 1.0)      # (BF16 keys are up to 2^-8 longer than their norm says)
    T = size[3]
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0, scale=0.3)
    ref_y, ref_S, _, _ = R.prefill(q, k, v, alpha, beta, S0, 0.3)
    R.check(S, ref_S, dtype, "S", T)
    R.check(y, ref_y, dtype, "y", T)
    got = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, scale=0.3)
    R.check_all(got, R.backward(q, k, v, dy, alpha, beta, S0, dS_T, 0.3), dtype, T)
    assert la.last_device_status() == 0


@pytest.mark.parametrize("size", [(1, 8, 4, 10000, 128, 128), (1, 4, 4, 20000, 64, 192), (1, 2, 1, 40000, 128, 256)], ids=ids)
def test_long_sequences_in_two_parts(la, size):  # noqa: F811
    """Few heads of full width and of several column tiles go in two parts: the bits of the same call packed, which goes in one, and
    the last tokens against 64 bits from the state before them."""
    B, H, Hk, T, r, dv = size
    q, k, v, _, alpha, beta, S0, _ = make(*size, BF, True, 43)
    S = S0.clone()
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S, scale=0.2, S_out=S)
    tok = [x[0].transpose(0, 1).contiguous() for x in (q, k, v, alpha, beta)]
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y2, S2 = la.gated_delta_prefill_varlen(*tok[:3], cu, *tok[3:], S0=S0, scale=0.2)
    assert la.last_device_status() == 0
    assert torch.equal(S, S2) and torch.equal(y[0].transpose(0, 1), y2)
    cut = T - 150
    part = lambda a, b: [x[:, :, a:b].contiguous() for x in (q, k, v, alpha, beta)]  # noqa: E731
    _, before = la.gated_delta_prefill(*part(0, cut), S0=S0)
    ref_y, ref_S, _, _ = R.prefill(*part(cut, T), before, 0.2)
    R.check(S, ref_S, BF, "S", 150)
    R.check(y[:, :, cut:], ref_y, BF, "y", 150)


@pytest.mark.parametrize("size", [(1, 4, 2, 500, 128, 128), (2, 2, 2, 333, 64, 64), (1, 2, 2, 300, 128, 64), (1, 2, 1, 260, 64, 128)], ids=ids)
def test_roundings_of_bf16_results(la, size):  # noqa: F811
    """The 2-norms of the errors of y, dq, dk and dv in chunks, by counting their roundings.  Rounding to BF16 is off by at most 2^-8 of a value and, spread
    evenly over a step, by 2^-8 / sqrt(3) in the 2-norm.  y: its own, and S's, or A's and V's, whichever product a term comes from: at most three,
    together 2^-8.  dq: its own, and dP's: two.  dk: its own, and dP's or dL's: two.  dv: its own.  What goes in two parts adds 2^-16, the sums in FP32
    less."""
    T = size[3]
    q, k, v, dy, alpha, beta, S0, dS_T = make(*size, BF, True, 61)
    y, S = la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0, scale=0.2)
    got = la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T, scale=0.2)
    ref_y, _, _, _ = R.prefill(q, k, v, alpha, beta, S0, 0.2)
    ref, _ = R.backward(q, k, v, dy, alpha, beta, S0, dS_T, 0.2)
    rounding = 2.0 ** -8 / 3 ** 0.5
    for x, z, n, name in ((y, ref_y, 3, "y"), (got[0], ref[0], 2, "dq"), (got[1], ref[1], 2, "dk"), (got[2], ref[2], 1, "dv")):
        rel = float((R.f64(x) - z).norm() / z.norm())
        print(f"[roundings] {name} {size}: {rel:.2e} of {n ** 0.5 * rounding + 2.0 ** -15:.2e}")
        assert rel <= n ** 0.5 * rounding + 2.0 ** -15, (name, rel)


def test_calls_at_once(la):  # noqa: F811
    """Calls of every kind on four streams at the same time, each waiting for parts of its own while the others hold SMs: the bits of the
    calls alone."""
    jobs = []
    for seed, size in ((1, (2, 8, 4, 1500, 128, 128)), (2, (4, 8, 8, 700, 64, 64)), (3, (1, 8, 8, 10000, 128, 128)), (4, (2, 4, 4, 900, 64, 128))):
        q, k, v, dy, alpha, beta, S0, dS_T = make(*size, BF, True, seed)
        tok = [x[0].transpose(0, 1).contiguous() for x in (q, k, v, alpha, beta)]
        n = size[3] // 40
        cu = torch.tensor([min(i * n, size[3]) for i in range(41)], dtype=torch.int32, device="cuda")

        def job(q=q, k=k, v=v, dy=dy, alpha=alpha, beta=beta, S0=S0, dS_T=dS_T, tok=tok, cu=cu):
            out = [*la.gated_delta_prefill(q, k, v, alpha, beta, S0=S0)]
            out += la.gated_delta_backward(q, k, v, dy, alpha, beta, S0=S0, dS_T=dS_T)
            out += la.gated_delta_prefill_varlen(*tok[:3], cu, *tok[3:], y=torch.zeros_like(tok[2]))
            return out
        jobs.append(job)
    alone = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        held = []
        for job, stream in zip(jobs, streams):
            with torch.cuda.stream(stream):
                held.append(job())
        torch.cuda.synchronize()
        for a, b in zip(alone, held):
            for x, z in zip(a, b):
                assert torch.equal(x, z)
    assert la.last_device_status() == 0


@DTYPES
def test_gradients_past_32_bits(la, dtype):  # noqa: F811
    """Arrays of more than 2^31 elements: the last heads' gradients have the bits of those heads alone."""
    H, T, r, dv = (17, 1 << 20, 128, 128) if dtype == BF else (8704, 2048, 128, 128)
    g = torch.Generator(device="cuda").manual_seed(5)
    normal = lambda sd: torch.randn((1, H, T, r), generator=g, device="cuda", dtype=dtype).mul_(sd)  # noqa: E731
    q, k, v, dy = normal(r ** -0.5), normal(r ** -0.5), normal(1.0), normal(1.0)
    assert v.numel() > 1 << 31
    alpha, beta = (torch.rand((1, H, T), generator=g, device="cuda").mul_(0.3).add_(c) for c in (0.7, 0.1))
    alpha[:, :, ::1000] = 1e-9
    got = la.gated_delta_backward(q, k, v, dy, alpha, beta, scale=0.1)
    assert la.last_device_status() == 0
    for h in (H - 1, 0):
        one = lambda x: x[:, h:h + 1].contiguous()  # noqa: E731
        for x, z, name in zip(got, la.gated_delta_backward(*(one(x) for x in (q, k, v, dy, alpha, beta)), scale=0.1), R.NAMES):
            assert torch.isfinite(z).all() and z.any(), name
            assert torch.equal(one(x), z), (h, name)
    del q, k, v, dy, got
    torch.cuda.empty_cache()
