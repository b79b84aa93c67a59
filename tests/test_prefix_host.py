"""Host-only checks of the shared-prefix calls: argument errors of the C ABI (before any CUDA call)
and the tests' 64-bit references against the oracle's per-token recurrence."""
import ctypes

import numpy as np
import pytest
import torch

import glasynth as gs
import linear_attention_recurrence_simple_gb300 as gla
import oracle
from tests.prefix_helpers import SCALE, Tails, ref_decode, ref_fold

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS = 0, -1, -2, -3, -4, -5, -6
A, MIS = 0x10000, 0x10004  # fake device addresses, never dereferenced
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return gla.load_library()


def tail(k=A, v=A, ks=None, vs=None, rows=8, cap=32, fmt=0):
    return ctypes.byref(gla._CTail(k, v, ks, vs, rows, cap, fmt))


def _decode(lib, q=A, k=A, v=A, ll=A, pool=A, rows=3, pr=A, t=None, slot=None, tl=A, o=A, N=4, H=2, dk=96, dv=192, dt=0,
            **kw):
    return lib.gla_prefix_decode_step(P(q), P(k), P(v), P(ll), 0.1, P(pool), rows, P(pr), t or tail(**kw), P(slot),
                                      P(tl), P(o), N, H, dk, dv, dt, None)


def _append(lib, k=A, v=A, t=None, slot=None, pos=A, cu=A, n=3, T=9, H=2, dk=96, dv=192, dt=0, read=False, **kw):
    if read:
        return lib.gla_tail_read(t or tail(**kw), P(slot), P(pos), P(cu), P(k), P(v), n, T, H, dk, dv, dt, None)
    return lib.gla_tail_append(P(k), P(v), t or tail(**kw), P(slot), P(pos), P(cu), n, T, H, dk, dv, dt, None)


def _fold(lib, ll=A, pool=A, rows=3, pr=A, t=None, slot=None, tl=A, out=A, orows=4, orow=None, N=4, H=2, dk=96, dv=192,
          dt=0, **kw):
    return lib.gla_tail_fold(P(ll), P(pool), rows, P(pr), t or tail(**kw), P(slot), P(tl), P(out), orows, P(orow), N, H,
                             dk, dv, dt, None)


def _check_tail_errors(call):
    assert call(fmt=2) == DTYPE
    assert call(fmt=-1) == DTYPE
    assert call(rows=-1, t=tail(rows=-1)) == SHAPE
    assert call(cap=0) == SHAPE
    assert call(cap=24) == SHAPE                        # a multiple of 16
    assert call(t=tail(rows=2 ** 31 - 1, cap=2 ** 30)) == SHAPE  # byte offsets past 64 bits
    assert call(t=tail(k=None)) == NULL
    assert call(t=tail(v=None)) == NULL
    assert call(fmt=1) == NULL                          # MXFP8 needs both scale arrays
    assert call(fmt=1, ks=A) == NULL
    assert call(t=tail(k=MIS)) == ALIGN
    assert call(t=tail(v=MIS)) == ALIGN
    assert call(fmt=1, ks=MIS, vs=A) == ALIGN
    assert call(fmt=1, ks=A, vs=MIS) == ALIGN
    assert call(dt=5) == DTYPE
    assert call(dk=64) == UNSUP
    assert call(dv=128) == UNSUP
    assert call(H=0) == SHAPE


def test_decode_argument_errors(lib):
    _check_tail_errors(lambda **kw: _decode(lib, **kw) if "rows" not in kw else _decode(lib, t=kw["t"]))
    assert lib.gla_prefix_decode_step(P(A), P(A), P(A), P(A), 0.1, P(A), 3, P(A), None, None, P(A), P(A), 4, 2, 96, 192,
                                      0, None) == NULL
    for name in ("q", "k", "v", "ll", "pool", "pr", "tl", "o"):
        assert _decode(lib, **{name: None}) == NULL, name
    for name in ("q", "k", "v", "ll", "pool", "o"):
        assert _decode(lib, **{name: MIS}) == ALIGN, name
    for name in ("pr", "tl", "slot"):
        assert _decode(lib, **{name: A + 2}) == ALIGN, name
    assert _decode(lib, N=-1) == SHAPE
    assert _decode(lib, N=9) == SHAPE                   # nine sequences, eight tail rows, no slots
    assert _decode(lib, N=2 ** 30, H=2, slot=A) == SHAPE
    assert _decode(lib, N=0, q=None, k=None, v=None, o=None) == OK


def test_append_and_read_argument_errors(lib):
    for read in (False, True):
        call = lambda **kw: _append(lib, read=read, **kw)  # noqa: E731
        _check_tail_errors(lambda **kw: call(**kw) if "rows" not in kw else call(t=kw["t"]))
        for name in ("k", "v", "pos", "cu"):
            assert call(**{name: None}) == NULL, name
        for name in ("k", "v"):
            assert call(**{name: MIS}) == ALIGN, name
        for name in ("pos", "cu", "slot"):
            assert call(**{name: A + 1}) == ALIGN, name
        assert call(n=-1) == SHAPE
        assert call(T=-1) == SHAPE
        assert call(T=2 ** 31 - 63) == SHAPE
        assert call(T=2 ** 30, H=200) == SHAPE
        assert call(n=9) == SHAPE
        assert call(n=0, k=None, v=None, pos=None, cu=None) == OK
        assert call(T=0, k=None, v=None, pos=None, cu=None) == OK


def test_fold_argument_errors(lib):
    _check_tail_errors(lambda **kw: _fold(lib, **kw) if "rows" not in kw else _fold(lib, t=kw["t"]))
    for name in ("ll", "pool", "pr", "tl", "out"):
        assert _fold(lib, **{name: None}) == NULL, name
    for name in ("ll", "pool", "out"):
        assert _fold(lib, **{name: MIS}) == ALIGN, name
    for name in ("pr", "tl", "slot", "orow"):
        assert _fold(lib, **{name: A + 2}) == ALIGN, name
    assert _fold(lib, N=-1) == SHAPE
    assert _fold(lib, rows=-1, t=tail()) == SHAPE
    assert _fold(lib, orows=-1, orow=A) == SHAPE
    assert _fold(lib, orows=3) == SHAPE                 # four sequences, three rows, no out_row
    assert _fold(lib, N=9, orows=9) == SHAPE
    assert _fold(lib, N=0, pool=None, out=None) == OK


def _fwd(lib, q=A, k=A, v=A, ll=A, pool=A, rows=3, pr=A, o=A, hT=None, cu=A, n=2, T=8, H=2, dk=96, dv=192, dt=0, ws=A,
         wsb=4096):
    return lib.gla_prefix_fwd(P(q), P(k), P(v), P(ll), P(pool), rows, P(pr), 0.1, P(o), P(hT), P(cu), n, T, H, dk, dv, dt,
                              P(ws), wsb, None)


def _bwd(lib, q=A, k=A, v=A, ll=A, pool=A, rows=3, pr=A, dO=A, dhT=None, dq=A, dk_=A, dv_=A, dpool=A, cu=A, n=2, T=8, H=2,
         dk=96, dv=192, dt=0, ws=A, wsb=1 << 30):
    return lib.gla_prefix_bwd(P(q), P(k), P(v), P(ll), P(pool), rows, P(pr), 0.1, P(dO), P(dhT), P(dq), P(dk_), P(dv_),
                              P(dpool), P(cu), n, T, H, dk, dv, dt, P(ws), wsb, None)


def test_fwd_and_bwd_argument_errors(lib):
    for call, ptrs in ((_fwd, ("q", "k", "v", "o")), (_bwd, ("q", "k", "v", "dO", "dq", "dk_", "dv_"))):
        for name in ptrs + ("ll", "pool"):
            assert call(lib, **{name: None}) == NULL, name
            assert call(lib, **{name: MIS}) == ALIGN, name
        assert call(lib, pr=None) == NULL
        assert call(lib, cu=None) == NULL
        assert call(lib, pr=A + 2) == ALIGN
        assert call(lib, cu=A + 2) == ALIGN
        assert call(lib, dt=3) == DTYPE
        assert call(lib, dk=64) == UNSUP
        assert call(lib, n=-1) == SHAPE
        assert call(lib, T=-1) == SHAPE
        assert call(lib, H=0) == SHAPE
        assert call(lib, rows=-1) == SHAPE
        assert call(lib, ws=None) == WS
        assert call(lib, wsb=16) == WS
        assert call(lib, ws=MIS) == ALIGN
    assert _fwd(lib, hT=MIS) == ALIGN
    assert _fwd(lib, n=0, cu=None) == OK
    assert _bwd(lib, dhT=MIS) == ALIGN
    assert _bwd(lib, dpool=MIS) == ALIGN
    assert _bwd(lib, n=0, dpool=None) == OK
    assert _bwd(lib, n=0, rows=0) == OK
    need = gla.gla_prefix_bwd_workspace_bytes(2, 8, 2, 0)
    assert need >= gla.gla_bwd_workspace_bytes(2, 8, 2, True, 0) + 2 * 2 * 96 * 192 * 4
    assert _bwd(lib, wsb=need - 1) == WS
    assert gla.gla_prefix_bwd_workspace_bytes(-1, 8, 2, 0) == 0
    assert gla.gla_prefix_bwd_workspace_bytes(2, 8, 2, 9) == 0


def test_binding_refuses_tensors_that_are_not_on_a_device_or_have_other_shapes():
    t = gla.gla_tail_alloc(2, 3, 20, device="cpu")
    assert t.k.shape == (2, 3, 32, 96) and t.v.shape == (2, 3, 32, 192) and t.k.dtype == torch.bfloat16
    m = gla.gla_tail_alloc(2, 3, 16, torch.float8_e4m3fn, device="cpu")
    assert m.k.dtype == torch.uint8 and m.k_scales.shape == (2, 3, 16, 3) and m.v_scales.shape == (2, 3, 16, 6)
    with pytest.raises(TypeError):
        gla.gla_tail_alloc(2, 3, 16, torch.float16, device="cpu")
    z = torch.zeros
    i = z(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gla.gla_prefix_decode_step(z(2, 3, 96), z(2, 3, 96), z(2, 3, 192), z(3), z(1, 3, 96, 192), i, t, i)
    with pytest.raises(TypeError):
        gla.gla_prefix_decode_step(z(2, 3, 96).half(), z(2, 3, 96).half(), z(2, 3, 192).half(), z(3),
                                   z(1, 3, 96, 192), i, t, i)
    with pytest.raises(ValueError):
        gla.gla_tail_append(z(2, 3, 96), z(2, 3, 192), t, i, z(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        gla.gla_tail_fold(z(3), z(1, 3, 96, 192), i, t, i)


@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
def test_references_equal_the_recurrence(fmt):
    """The written-out sums against the oracle's recurrence over the same tokens, started from the
    shared state: 64-bit sums in two orders, 2^-40 of the terms' magnitude apart at most."""
    lens, H, rows = [0, 1, 5, 18], 2, [1, 0, 1, 1]
    t = Tails(3, 6, H, 32, fmt, True)
    slots = [4, 0, 5, 2]
    ll = np.array([np.log(0.9), -np.inf], np.float32)
    pool = gs.normal(3, 4, (2, H, 96, 192), 0.1)
    q, k = (gs.bf16_round(gs.normal(3, 5 + i, (4, H, 96), 0.1)) for i in range(2))
    v = gs.bf16_round(gs.normal(3, 7, (4, H, 192)))
    o, mag = ref_decode(q, k, v, ll, SCALE, pool, rows, t.k, t.v, slots, lens)
    s, smag = ref_fold(ll, pool, rows, t.k, t.v, slots, lens)
    for n, L in enumerate(lens):
        K, V = t.k[slots[n], :, :L].transpose(1, 0, 2), t.v[slots[n], :, :L].transpose(1, 0, 2)
        state = pool[rows[n]][None].astype(np.float64)
        if L:
            _, hT = oracle.fwd(np.zeros_like(K), K, V, ll, SCALE, h0=pool[rows[n]][None])
            state = hT.copy()
        assert np.all(np.abs(s[n] - state[0]) <= 2.0 ** -40 * smag[n])
        on = oracle.decode_step(q[n:n + 1], k[n:n + 1], v[n:n + 1], ll, SCALE, state.copy())
        assert np.all(np.abs(o[n] - on[0]) <= 2.0 ** -40 * mag[n])
