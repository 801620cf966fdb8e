"""Host checks of the decayed linear attention, beam selection and state reordering entry
points: refusals return before anything is enqueued, so these run without a GPU."""
import pytest

FAKE = 1 << 20  # a 256-byte aligned non-null address; never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def native():
    from recurrent_state_02_gb300 import build, _native
    build.build()
    return _native


def call(native, entry, names, defaults, **kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return getattr(native.lib(), entry)(*[a[n] for n in names.split()])


PREFILL = "q k v dtype decay S0 B H T r dv scale y S_out ws ws_bytes stream"
VARLEN = "q k v dtype decay S0 cu B H T r dv scale y S_out stream"
DECODE = "q k v dtype decay S B H r dv scale y stream"
BACKWARD = "q k v dtype decay S0 B H T r dv scale dy dS_T dq dk dv_out dS0 ws ws_bytes stream"
BASE = dict(q=FAKE, k=FAKE, v=FAKE, dtype=0, decay=FAKE, S0=None, S=FAKE, cu=FAKE, B=2, H=3, T=64, r=128, dv=128,
            scale=1.0, y=FAKE, S_out=FAKE, dy=FAKE, dS_T=None, dq=FAKE, dk=FAKE, dv_out=FAKE, dS0=FAKE, ws=None,
            ws_bytes=0, stream=None)


@pytest.mark.parametrize("entry,names,outs", [("la_decay_prefill", PREFILL, "y S_out"),
                                              ("la_decay_prefill_varlen", VARLEN, "y S_out cu"),
                                              ("la_decay_decode_step", DECODE, "y S"),
                                              ("la_decay_backward", BACKWARD, "dy dq dk dv_out dS0")])
def test_decay_refusals(native, entry, names, outs):
    N = native
    f = lambda **kw: call(N, entry, names, {n: BASE[n] for n in names.split()}, **kw)  # noqa: E731
    for n in ("q k v decay " + outs).split():
        assert f(**{n: None}) == N.LA_ERR_NULL, n
    for n in "B H r dv".split():
        assert f(**{n: 0}) == N.LA_ERR_SHAPE, n
    if "T" in names.split():
        assert f(T=-1) == N.LA_ERR_SHAPE and f(T=(1 << 30) + 1, H=1) == N.LA_ERR_UNSUPPORTED
    assert f(scale=float("nan")) == N.LA_ERR_SHAPE and f(scale=float("inf")) == N.LA_ERR_SHAPE
    assert f(dtype=5) == N.LA_ERR_DTYPE
    assert f(r=257) == N.LA_ERR_UNSUPPORTED and f(dv=257) == N.LA_ERR_UNSUPPORTED
    assert f(B=65536) == N.LA_ERR_UNSUPPORTED and f(H=65536) == N.LA_ERR_UNSUPPORTED
    assert f(q=FAKE + 1) == N.LA_ERR_ALIGN and f(decay=FAKE + 2) == N.LA_ERR_ALIGN
    assert f(dtype=1, k=FAKE + 2) == N.LA_ERR_ALIGN
    if entry == "la_decay_prefill_varlen":
        assert f(cu=FAKE + 2) == N.LA_ERR_ALIGN and f(T=1 << 30, H=4) == N.LA_ERR_SHAPE


def test_workspace_queries(native):
    L = native.lib()
    for fn in (L.la_decay_prefill_workspace_bytes, L.la_decay_backward_workspace_bytes):
        for args in ((0, 1, 64, 128, 128, 0), (1, 1, -1, 128, 128, 0), (1, 1, 64, 0, 128, 0), (1, 1, 64, 128, 300, 0),
                     (1, 1, 64, 128, 128, 7), (1, 1, 0, 128, 128, 0), (1, 1, 1 << 16, 128, 128, 1)):
            assert fn(*args) == 0, args


SELECT = "logits dtype ld scores done B K V eos next parents tokens done_out stream"
SELECT_BASE = dict(logits=FAKE, dtype=0, ld=1000, scores=FAKE, done=None, B=2, K=4, V=1000, eos=-1, next=FAKE,
                   parents=FAKE, tokens=FAKE, done_out=None, stream=None)


def test_select_refusals(native):
    N = native
    f = lambda **kw: call(N, "la_beam_select", SELECT, SELECT_BASE, **kw)  # noqa: E731
    for n in "logits scores next parents tokens".split():
        assert f(**{n: None}) == N.LA_ERR_NULL, n
    for n in "B K V".split():
        assert f(**{n: 0}) == N.LA_ERR_SHAPE, n
    assert f(ld=999) == N.LA_ERR_SHAPE and f(eos=1000) == N.LA_ERR_SHAPE and f(eos=-2) == N.LA_ERR_SHAPE
    assert f(done=FAKE) == N.LA_ERR_SHAPE          # an ended beam's candidate needs its token
    assert f(ld=1 << 62) == N.LA_ERR_SHAPE
    assert f(dtype=3) == N.LA_ERR_DTYPE
    assert f(K=33) == N.LA_ERR_UNSUPPORTED and f(B=65536) == N.LA_ERR_UNSUPPORTED
    assert f(V=(1 << 30) + 1, ld=1 << 31) == N.LA_ERR_UNSUPPORTED
    assert f(logits=FAKE + 1) == N.LA_ERR_ALIGN and f(dtype=1, logits=FAKE + 2) == N.LA_ERR_ALIGN
    assert f(parents=FAKE + 2) == N.LA_ERR_ALIGN and f(next=FAKE + 1) == N.LA_ERR_ALIGN


REORDER = "S z parents B K H r dv S_out z_out stream"
REORDER_BASE = dict(S=FAKE, z=None, parents=FAKE, B=2, K=4, H=2, r=128, dv=128, S_out=FAKE, z_out=None, stream=None)


def test_reorder_refusals(native):
    N = native
    f = lambda **kw: call(N, "la_state_reorder", REORDER, REORDER_BASE, **kw)  # noqa: E731
    for n in "S parents S_out".split():
        assert f(**{n: None}) == N.LA_ERR_NULL, n
    assert f(z=FAKE) == N.LA_ERR_NULL and f(z_out=FAKE) == N.LA_ERR_NULL
    for n in "B K H r dv".split():
        assert f(**{n: 0}) == N.LA_ERR_SHAPE, n
    assert f(K=33) == N.LA_ERR_UNSUPPORTED and f(B=65536) == N.LA_ERR_UNSUPPORTED
    assert f(H=1 << 20, r=1 << 20, dv=1 << 10) == N.LA_ERR_UNSUPPORTED
    assert f(S=FAKE + 2) == N.LA_ERR_ALIGN and f(z=FAKE + 1, z_out=FAKE) == N.LA_ERR_ALIGN
