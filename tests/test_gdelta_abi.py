"""Host checks of the gated delta rule's and the token log-probabilities' entry points: refusals return before anything is
enqueued, so these run without a GPU."""
import pytest

from test_decay_abi import FAKE, call, native  # noqa: F401  (native: the fixture)

PREFILL = "q k v dtype alpha beta S0 B H Hk T r dv scale y S_out ws ws_bytes stream"
VARLEN = "q k v dtype alpha beta S0 cu B H Hk T r dv scale y S_out ws ws_bytes stream"
DECODE = "q k v dtype alpha beta S B H Hk r dv scale y stream"
BACKWARD = "q k v dtype alpha beta S0 B H Hk T r dv scale dy dS_T dq dk dv_out dalpha dbeta dS0 ws ws_bytes stream"
BASE = dict(q=FAKE, k=FAKE, v=FAKE, dtype=0, alpha=FAKE, beta=FAKE, S0=None, S=FAKE, cu=FAKE, B=2, H=4, Hk=2, T=64, r=128, dv=128,
            scale=1.0, y=FAKE, S_out=FAKE, dy=FAKE, dS_T=None, dq=FAKE, dk=FAKE, dv_out=FAKE, dalpha=FAKE, dbeta=FAKE, dS0=FAKE,
            ws=FAKE, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("entry,names,outs", [("la_gated_delta_prefill", PREFILL, "y S_out"),
                                              ("la_gated_delta_prefill_varlen", VARLEN, "y S_out cu"),
                                              ("la_gated_delta_decode_step", DECODE, "y S"),
                                              ("la_gated_delta_backward", BACKWARD, "dy dq dk dv_out dS0")])
def test_gated_delta_refusals(native, entry, names, outs):  # noqa: F811
    N = native
    f = lambda **kw: call(N, entry, names, {n: BASE[n] for n in names.split()}, **kw)  # noqa: E731
    for n in ("q k v " + outs).split():
        assert f(**{n: None}) == N.LA_ERR_NULL, n
    for n in "B H Hk r dv".split():
        assert f(**{n: 0}) == N.LA_ERR_SHAPE, n
    assert f(Hk=3) == N.LA_ERR_SHAPE and f(Hk=8) == N.LA_ERR_SHAPE
    if "T" in names.split():
        assert f(T=-1) == N.LA_ERR_SHAPE and f(T=(1 << 30) + 1, H=1, Hk=1) == N.LA_ERR_UNSUPPORTED
    assert f(scale=float("nan")) == N.LA_ERR_SHAPE and f(scale=float("inf")) == N.LA_ERR_SHAPE
    assert f(dtype=5) == N.LA_ERR_DTYPE
    assert f(r=257) == N.LA_ERR_UNSUPPORTED and f(dv=257) == N.LA_ERR_UNSUPPORTED
    assert f(B=65536) == N.LA_ERR_UNSUPPORTED and f(H=65536) == N.LA_ERR_UNSUPPORTED
    for n in "q k v".split():
        assert f(**{n: FAKE + 1}) == N.LA_ERR_ALIGN, n
        assert f(dtype=1, **{n: FAKE + 2}) == N.LA_ERR_ALIGN, n
    for n in "alpha beta S0 S S_out cu dS_T dalpha dbeta dS0".split():
        if n in names.split():
            assert f(**{n: FAKE + 2}) == N.LA_ERR_ALIGN, n
    if entry == "la_gated_delta_prefill_varlen":
        assert f(T=1 << 30, H=4) == N.LA_ERR_SHAPE


def test_gated_delta_workspaces(native):  # noqa: F811
    N, L = native, native.lib()
    sizes = [BASE[n] for n in "B H Hk T r dv dtype".split()]
    need = L.la_gated_delta_backward_workspace_bytes(*sizes)
    assert need > 0
    f = lambda **kw: call(N, "la_gated_delta_backward", BACKWARD, {n: BASE[n] for n in BACKWARD.split()}, **kw)  # noqa: E731
    assert f(ws=None) == N.LA_ERR_WORKSPACE and f(ws_bytes=need - 1) == N.LA_ERR_WORKSPACE and f(ws=FAKE + 64) == N.LA_ERR_ALIGN
    for entry, names in (("la_gated_delta_prefill", PREFILL), ("la_gated_delta_prefill_varlen", VARLEN)):
        need = getattr(L, entry + "_workspace_bytes")(*sizes)
        g = lambda **kw: call(N, entry, names, {n: BASE[n] for n in names.split()}, **kw)  # noqa: E731
        if need:
            assert g(ws=None) == N.LA_ERR_WORKSPACE and g(ws_bytes=need - 1) == N.LA_ERR_WORKSPACE and g(ws=FAKE + 64) == N.LA_ERR_ALIGN
    for fn in (L.la_gated_delta_prefill_workspace_bytes, L.la_gated_delta_prefill_varlen_workspace_bytes,
               L.la_gated_delta_backward_workspace_bytes):
        for args in ((0, 1, 1, 64, 128, 128, 0), (1, 1, 1, -1, 128, 128, 0), (1, 1, 1, 64, 0, 128, 0), (1, 3, 2, 64, 128, 128, 0),
                     (1, 1, 1, 64, 128, 300, 0), (1, 1, 1, 64, 128, 128, 7), (1, 1, 1, 0, 128, 128, 1)):
            assert fn(*args) == 0, args


def test_many_packed_sequences(native):  # noqa: F811
    """total_T counts the tokens of all sequences: their number times that is no size of anything."""
    L = native.lib()
    sizes = (4096, 16, 8, 1 << 20, 128, 128, BASE["dtype"])
    assert L.la_gated_delta_prefill_workspace_bytes(*sizes) == 0            # B sequences of that length each
    assert L.la_gated_delta_prefill_varlen_workspace_bytes(*sizes) > 0


SCORE = "logits dtype ld tokens N V top lp ent lse tlp ttok stream"
GRAD = "logits dtype ld tokens lse ent dlp dent N V out gd stream"
ROWS = dict(logits=FAKE, dtype=0, ld=1000, tokens=FAKE, N=4, V=1000, top=5, lp=FAKE, ent=FAKE, lse=FAKE, tlp=FAKE, ttok=FAKE, dlp=FAKE,
            dent=FAKE, out=FAKE + 4096, gd=1000, stream=None)


@pytest.mark.parametrize("entry,names,outs", [("la_token_logprobs", SCORE, "lp tlp ttok"),
                                              ("la_token_logprobs_backward", GRAD, "lse ent dlp out")])
def test_logprob_refusals(native, entry, names, outs):  # noqa: F811
    N = native
    f = lambda **kw: call(N, entry, names, {n: ROWS[n] for n in names.split()}, **kw)  # noqa: E731
    for n in ("logits tokens " + outs).split():
        assert f(**{n: None}) == N.LA_ERR_NULL, n
    assert f(N=-1) == N.LA_ERR_SHAPE and f(V=0) == N.LA_ERR_SHAPE and f(ld=999) == N.LA_ERR_SHAPE and f(ld=1 << 61) == N.LA_ERR_SHAPE
    assert f(dtype=4) == N.LA_ERR_DTYPE and f(V=(1 << 30) + 1, ld=1 << 31, **({"gd": 1 << 31} if "gd" in names else {})) == N.LA_ERR_UNSUPPORTED
    assert f(logits=FAKE + 1) == N.LA_ERR_ALIGN and f(dtype=1, logits=FAKE + 2) == N.LA_ERR_ALIGN
    for n in "tokens lse ent lp tlp ttok dlp dent".split():
        if n in names.split():
            assert f(**{n: FAKE + 2}) == N.LA_ERR_ALIGN, n
    if entry == "la_token_logprobs":
        assert f(top=-1) == N.LA_ERR_SHAPE and f(top=33) == N.LA_ERR_UNSUPPORTED
    else:
        assert f(gd=999) == N.LA_ERR_SHAPE and f(out=FAKE + 1) == N.LA_ERR_ALIGN
        assert f(out=FAKE, gd=1001) == N.LA_ERR_SHAPE      # in place, but at another stride
        assert f(N=1 << 30, V=1 << 20, ld=1 << 20, gd=1 << 20) == N.LA_ERR_UNSUPPORTED
    assert f(N=0, logits=None, tokens=None, **({"out": None} if "gd" in names else {"lp": None})) == N.LA_OK
