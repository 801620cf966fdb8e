"""The wrappers of the gated delta rule and of the token log-probabilities call the library with the tensors' device current
and that device's stream, whichever device is current outside, and refuse what does not fit before they call it.  On
the CPU: library, guard and streams are recorders."""
import pytest
import torch

import recurrent_state_02_gb300 as la
from test_binding_device import DEV, FakeTensor
from test_decay_binding import calls  # noqa: F401

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
B, H, Hk, T, r, dv, N, V = 2, 4, 2, 70, 128, 64, 5, 500


class Rows(FakeTensor):
    """A matrix with rows `ld` apart."""

    def __init__(self, shape, dtype, ld):
        super().__init__(shape, dtype)
        self.ld = ld

    def is_contiguous(self):
        return self.ld == self.shape[1]

    def stride(self, dim):
        return (self.ld, 1)[dim]


def dense(**other):
    t = dict(q=FakeTensor((B, Hk, T, r), BF), k=FakeTensor((B, Hk, T, r), BF), v=FakeTensor((B, H, T, dv), BF),
             alpha=FakeTensor((B, H, T), F32), beta=FakeTensor((B, H, T), F32), S=FakeTensor((B, H, r, dv), F32))
    t.update(other)
    return t


def test_wrappers_use_the_tensors_device(calls):  # noqa: F811
    t = dense()
    la.gated_delta_prefill(t["q"], t["k"], t["v"], t["alpha"], t["beta"], S0=t["S"])
    la.gated_delta_backward(t["q"], t["k"], t["v"], t["v"], t["alpha"], t["beta"], S0=t["S"], dS_T=t["S"])
    la.gated_delta_prefill_varlen(*(FakeTensor((T, h, n), BF) for h, n in ((Hk, r), (Hk, r), (H, dv))), FakeTensor((B + 1,), I32),
                                  FakeTensor((T, H), F32), None, S0=t["S"])
    la.gated_delta_decode_step(*(FakeTensor((B, h, 1, n), BF) for h, n in ((Hk, r), (Hk, r), (H, dv))), t["S"],
                               FakeTensor((B, H), F32))
    for fn, args in ((la.gated_delta_prefill_workspace_bytes, (B, H, Hk, T, r, dv)),
                     (la.gated_delta_prefill_varlen_workspace_bytes, (B, H, Hk, T, r, dv)),
                     (la.gated_delta_backward_workspace_bytes, (B, H, Hk, T, r, dv))):
        fn(*args, device=DEV)
    logits, tokens, row = Rows((N, V), BF, V + 8), FakeTensor((N,), I32), FakeTensor((N,), F32)
    la.token_logprobs(logits, tokens, top=3)
    la.token_logprobs_backward(logits, tokens, row, row, row, row, dlogits=Rows((N, V), BF, V))
    assert {name for name, _, _ in calls} == {
        "la_gated_delta_prefill", "la_gated_delta_prefill_varlen", "la_gated_delta_decode_step", "la_gated_delta_backward",
        "la_gated_delta_prefill_workspace_bytes", "la_gated_delta_prefill_varlen_workspace_bytes",
        "la_gated_delta_backward_workspace_bytes", "la_token_logprobs", "la_token_logprobs_backward"}
    for name, dev, last in calls:
        assert dev == 1, name
        if not name.endswith("_bytes"):
            assert last == 1001, name


@pytest.mark.parametrize("wrong", [
    dict(k=FakeTensor((B, H, T, r), BF)), dict(v=FakeTensor((B, 3, T, dv), BF)), dict(q=FakeTensor((B, Hk, T, r), torch.float16)),
    dict(k=FakeTensor((B, Hk, T, r), F32)), dict(alpha=FakeTensor((B, H), F32)), dict(beta=FakeTensor((B, H, T), BF)),
    dict(S=FakeTensor((B, Hk, r, dv), F32)), dict(alpha=FakeTensor((B, H, T), F32, torch.device("cuda", 0))),
    dict(v=FakeTensor((B, H, T, dv), BF, torch.device("cpu"))),
], ids=["k heads", "H", "dtype", "mixed", "alpha shape", "beta dtype", "S heads", "device", "cpu"])
def test_wrappers_refuse(calls, wrong):  # noqa: F811
    t = dense(**wrong)
    with pytest.raises(ValueError):
        la.gated_delta_prefill(t["q"], t["k"], t["v"], t["alpha"], t["beta"], S0=t["S"])
    with pytest.raises(ValueError):
        la.gated_delta_backward(t["q"], t["k"], t["v"], t["v"], t["alpha"], t["beta"], S0=t["S"])
    assert not calls


def test_score_wrappers_refuse(calls):  # noqa: F811
    tokens, row = FakeTensor((N,), I32), FakeTensor((N,), F32)
    for logits, which in ((FakeTensor((N, 1, V), BF), tokens), (Rows((N, V), BF, V - 1), tokens), (Rows((N, V), torch.float16, V), tokens),
                          (Rows((N, V), BF, V), FakeTensor((N + 1,), I32)), (Rows((N, V), BF, V), FakeTensor((N,), torch.int64))):
        with pytest.raises(ValueError):
            la.token_logprobs(logits, which)
        with pytest.raises(ValueError):
            la.token_logprobs_backward(logits, which, row, row, row)
    assert not calls
