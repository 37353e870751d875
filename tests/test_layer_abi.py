"""The layer operators' C ABI and binding refuse bad arguments before the GPU
is touched (no compute call is made here)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from linear_attention_sequence_falcon_b200 import build
    build.build()
    from linear_attention_sequence_falcon_b200 import _lib
    return _lib.load()


P = 0x1000  # a pointer that no refused call may follow
OK, NULL, ENUM, SHAPE, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3, -9, -11


def _scan(lib, dtype=1, x=P, f=P, N=2, L=3, D=64, ldx=64, ldf=64, out=P):
    return lib.falcon_scan(dtype, x, f, None, None, N, L, D, ldx, ldf, out, None, None, None)


def test_scan_codes(lib):
    assert _scan(lib, dtype=2) == ENUM
    assert _scan(lib, N=-1) == SHAPE and _scan(lib, L=-1) == SHAPE and _scan(lib, D=-1) == SHAPE
    assert _scan(lib, ldx=63) == SHAPE and _scan(lib, ldf=0) == SHAPE
    assert _scan(lib, ldx=1 << 60) == SHAPE                       # offsets beyond 63 bits
    assert _scan(lib, ldx=(1 << 21) + 1) == SHAPE and _scan(lib, N=1, L=1, D=(1 << 21) + 1) == SHAPE
    assert _scan(lib, L=(1 << 30) + 1) == SHAPE
    assert _scan(lib, N=2 ** 30, D=4096, ldx=4096, ldf=4096) == SHAPE
    assert _scan(lib, x=None) == NULL and _scan(lib, f=None) == NULL and _scan(lib, out=None) == NULL
    assert _scan(lib, N=0) == OK and _scan(lib, D=0) == OK and _scan(lib, L=0, x=None, f=None, out=None) == OK


def _scan_bwd(lib, dtype=1, x=P, dout=P, dx=P, N=2, L=3, D=64, ldx=64, lddx=64, marks=P, ws=None, ws_bytes=0):
    return lib.falcon_scan_bwd_ws(dtype, x, P, None, None, marks, N, L, D, ldx, 64, dout, None, dx, lddx, P, 64, None,
                                  ws, ws_bytes, None)


def test_scan_bwd_codes(lib):
    assert _scan_bwd(lib, dtype=-1) == ENUM
    assert _scan_bwd(lib, ldx=1) == SHAPE and _scan_bwd(lib, lddx=1) == SHAPE and _scan_bwd(lib, L=-2) == SHAPE
    assert _scan_bwd(lib, x=None) == NULL and _scan_bwd(lib, dout=None) == NULL and _scan_bwd(lib, dx=None) == NULL
    n = ctypes.c_size_t(1)
    assert lib.falcon_scan_bwd_workspace_size(1, 2, 300, 64, 0, ctypes.byref(n)) == OK
    need = n.value
    assert need >= 2 * 3 * 64 * 4
    assert _scan_bwd(lib, L=300, marks=None) == WORKSPACE
    assert _scan_bwd(lib, L=300, marks=None, ws=0x10000, ws_bytes=need - 1) == WORKSPACE
    assert _scan_bwd(lib, L=300, marks=None, ws=0x10010, ws_bytes=need) == WORKSPACE
    assert lib.falcon_scan_bwd_workspace_size(1, 2, 300, 64, 1, ctypes.byref(n)) == OK and n.value == 0
    assert lib.falcon_scan_bwd_workspace_size(3, 2, 300, 64, 1, ctypes.byref(n)) == ENUM
    assert lib.falcon_scan_bwd_workspace_size(1, 2, 300, 64, 1, None) == NULL


def test_scan_step_codes(lib):
    step = lambda dt=1, x=P, N=2, D=64, ld=64, s=P: lib.falcon_scan_step(dt, x, P, s, N, D, ld, 64, P, P, None)  # noqa: E731
    assert step(dt=5) == ENUM and step(D=-1) == SHAPE and step(ld=10) == SHAPE
    assert step(x=None) == NULL and step(s=None) == NULL and step(N=0) == OK


def _gate(lib, dtype=1, o=P, sb=1, sh=1, sl=64, gate=P, ldg=128, eps=1e-6, B=1, H=2, L=3, d=64, out=P):
    return lib.falcon_norm_gate(dtype, o, sb, sh, sl, gate, ldg, P, 0, eps, B, H, L, d, out, None)


def test_norm_gate_codes(lib):
    assert _gate(lib, dtype=9) == ENUM
    assert _gate(lib, d=0) == SHAPE and _gate(lib, d=16385) == SHAPE and _gate(lib, H=-1) == SHAPE
    assert _gate(lib, ldg=127) == SHAPE and _gate(lib, sl=-64) == SHAPE and _gate(lib, sl=1 << 61) == SHAPE
    assert _gate(lib, eps=-1.0) == UNSUPPORTED and _gate(lib, eps=float("nan")) == UNSUPPORTED
    assert _gate(lib, o=None) == NULL and _gate(lib, out=None) == NULL
    assert _gate(lib, L=0) == OK and _gate(lib, gate=None, ldg=0, B=0) == OK


def test_norm_gate_bwd_codes(lib):
    n = ctypes.c_size_t(1)
    assert lib.falcon_norm_gate_bwd_workspace_size(1, 1, 2, 3, 64, ctypes.byref(n)) == OK
    need = n.value

    def bwd(gate=P, dgate=P, dout=P, lddg=128, ws=0x10000, ws_bytes=need, d=64):
        return lib.falcon_norm_gate_bwd_ws(1, P, 1, 1, 64, gate, 128, P, 0, 1e-6, 1, 2, 3, d, dout, P, 1, 1, 64, dgate,
                                           lddg, P, ws, ws_bytes, None)
    assert bwd(dgate=None) == NULL and bwd(gate=None) == NULL and bwd(dout=None) == NULL
    assert bwd(lddg=100) == SHAPE and bwd(d=20000) == SHAPE
    if need:
        assert bwd(ws=None) == WORKSPACE and bwd(ws_bytes=need - 1) == WORKSPACE and bwd(ws=0x10020) == WORKSPACE
    assert lib.falcon_norm_gate_bwd_workspace_size(1, 1, 2, 3, 0, ctypes.byref(n)) == SHAPE
    assert lib.falcon_norm_gate_bwd_workspace_size(1, 1, 2, 3, 64, None) == NULL


def test_residual_norm_codes(lib):
    fwd = lambda dt=1, r=P, h=P, R=2, D=64, eps=1e-6: lib.falcon_residual_norm(dt, r, P, P, P, eps, R, D, P, h, None)  # noqa: E731
    assert fwd(dt=2) == ENUM and fwd(R=-1) == SHAPE and fwd(D=0) == SHAPE and fwd(D=16385) == SHAPE
    assert fwd(eps=-1e-6) == UNSUPPORTED and fwd(r=None) == NULL and fwd(h=None) == NULL and fwd(R=0) == OK
    n = ctypes.c_size_t(1)
    assert lib.falcon_residual_norm_bwd_workspace_size(1, 5, 64, ctypes.byref(n)) == OK
    need = n.value

    def bwd(r=P, y=P, dh=P, dr=P, ws=0x10000, ws_bytes=need):
        return lib.falcon_residual_norm_bwd_ws(1, r, y, P, P, dh, None, 1e-6, 5, 64, dr, P, P, P, ws, ws_bytes, None)
    assert bwd(r=None) == NULL and bwd(dh=None) == NULL and bwd(dr=None) == NULL and bwd(y=None) == NULL
    if need:
        assert bwd(ws=None) == WORKSPACE and bwd(ws_bytes=need - 1) == WORKSPACE and bwd(ws=0x10080) == WORKSPACE


def test_short_way_is_built_and_hands_over(lib):
    """The module behind layer.py's short way is there, and answers None to what
    it does not take (here: tensors that are not on a GPU, and no tensors)."""
    from linear_attention_sequence_falcon_b200 import layer
    q = layer._quick
    assert q is not None
    x, s, w = torch.zeros(2, 5, 8), torch.zeros(2, 8), torch.zeros(8)
    o, r = torch.zeros(2, 3, 5, 8), torch.zeros(4, 8)
    for t in (x, None, 3):
        assert q.scan(t, x, None, None, None, None, None, True, False) is None
        assert q.scan_bwd(t, x, x, None, None, None, None, None, None, None) is None
        assert q.scan_step(t, s, s, None, None) is None
        assert q.norm_gate(t, None, w, 1e-6, None) is None
        assert q.norm_gate_bwd(t, None, w, 1e-6, x, True) is None
        assert q.residual_norm(t, w, 1e-6, None, None) is None
        assert q.residual_norm_bwd(t, w, 1e-6, r, None, None, None) is None
    assert q.norm_gate(o, None, w, "eps", None) is None
    with pytest.raises(TypeError):
        q.scan(x)


# ---------------------------------------------------------------- the binding (CPU tensors: refused before any pointer)

def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _refused(call, *args, match=None, **kw):
    import linear_attention_sequence_falcon_b200 as F
    with pytest.raises(F.FalconError, match=match):
        call(*args, **kw)


def test_binding_refuses_scan():
    import linear_attention_sequence_falcon_b200 as F
    x, s = _t(2, 5, 8), _t(2, 8, dtype=torch.float32)
    both = _t(2, 5, 16)
    assert F.check_scan_shapes(both[..., :8], both[..., 8:]) == (2, 5, 8, 16, 16)
    assert F.check_scan_shapes(both[:, -1:, :8], both[:, -1:, 8:])[3:] == (80, 80)  # one token of each sequence
    _refused(F.scan, x, x, match="no CPU path")
    _refused(F.scan, x[0], x[0])                                       # not [N,L,D]
    _refused(F.scan, x, _t(2, 5, 9))
    _refused(F.scan, x, x.float())
    _refused(F.scan, x.half(), x.half())
    _refused(F.scan, x.transpose(1, 2), x.transpose(1, 2))            # the last axis strided
    _refused(F.scan, _t(5, 2, 8).transpose(0, 1), x)                  # tokens not evenly spaced
    _refused(F.scan, _t(2, 1, 8).expand(2, 5, 8), x)                  # rows that overlap
    _refused(F.scan, x, x, reset=_t(2, 5))
    _refused(F.scan, x, x, reset=torch.zeros(2, 6, dtype=torch.bool))
    _refused(F.scan, x, x, initial_state=s.bfloat16())
    _refused(F.scan, x, x, initial_state=_t(2, 9, dtype=torch.float32))
    _refused(F.scan, x, x, marks=_t(2, 2, 8, dtype=torch.float32))
    _refused(F.scan, x, x, out=both[..., :8])
    _refused(F.scan_bwd, x, x, x.float())
    _refused(F.scan_bwd, x, x, x, dstate=_t(2, 8))
    _refused(F.scan_bwd, x, x, x, dx=_t(2, 5, 7))
    _refused(F.scan_step, x, x, s)
    _refused(F.scan_step, x[:, 0], x[:, 0], _t(2, 8))
    _refused(F.scan_step, x[:, 0], x[:, 0], s, state_out=_t(3, 8, dtype=torch.float32))


def test_binding_refuses_norm_gate():
    import linear_attention_sequence_falcon_b200 as F
    o, g, w = _t(2, 3, 5, 8), _t(2, 5, 24), _t(8, dtype=torch.float32)
    _refused(F.norm_gate, o, g, w, 1e-6, match="no CPU path")
    _refused(F.norm_gate, o[0], g, w, 1e-6)
    _refused(F.norm_gate, o, _t(2, 5, 23), w, 1e-6)
    _refused(F.norm_gate, o, g.float(), w, 1e-6)
    _refused(F.norm_gate, o, g, w.bfloat16(), 1e-6)
    _refused(F.norm_gate, o, g, _t(2, 8, dtype=torch.float32), 1e-6)
    _refused(F.norm_gate, o, g, w, -1.0, match="eps")
    _refused(F.norm_gate, o.transpose(2, 3), _t(2, 8, 15), _t(5, dtype=torch.float32), 1e-6)
    _refused(F.norm_gate, _t(1, 1, 1, 16385), None, None, 1e-6)
    _refused(F.norm_gate, o, g, w, 1e-6, out=_t(2, 3, 5, 8))
    _refused(F.norm_gate_bwd, o, g, w, 1e-6, _t(2, 5, 23))
    _refused(F.norm_gate_bwd, o, None, w, 1e-6, g, dgate=g)
    _refused(F.norm_gate_bwd, o, g, w, 1e-6, g, do=_t(2, 3, 1, 8).expand(2, 3, 5, 8), match="overlap")


def test_binding_refuses_residual_norm():
    import linear_attention_sequence_falcon_b200 as F
    r, w = _t(4, 8), _t(8, dtype=torch.float32)
    _refused(F.residual_norm, r, w, 1e-6, match="no CPU path")
    _refused(F.residual_norm, r, w, 1e-6, y=_t(5, 8))
    _refused(F.residual_norm, r, w, 1e-6, y=r.float())
    _refused(F.residual_norm, r, w, 1e-6, scale=w)                     # nothing to scale
    _refused(F.residual_norm, r, _t(9, dtype=torch.float32), 1e-6)
    _refused(F.residual_norm, r.t(), _t(4, dtype=torch.float32), 1e-6)
    _refused(F.residual_norm, r, w, float("nan"), match="eps")
    same = _t(4, 8)
    _refused(F.residual_norm, r, w, 1e-6, y=r, r_out=same, h=same)
    _refused(F.residual_norm_bwd, r, w, 1e-6, _t(4, 9))
    _refused(F.residual_norm_bwd, r, w, 1e-6, r, y=r, dy=same)         # without a scale dy is dr
    _refused(F.residual_norm_bwd, r, w, 1e-6, r, y=r, scale=w, dr=same, dy=same)


def test_binding_refuses_norm_over_the_stream_it_returns():
    """Without y the stream that residual_norm returns is r itself: h may not be
    written over it (with an r_out of its own, or with y, it may)."""
    import linear_attention_sequence_falcon_b200 as F
    r, w = _t(4, 8), _t(8, dtype=torch.float32)
    _refused(F.residual_norm, r, w, 1e-6, h=r, match="same array")
    _refused(F.residual_norm, r, w, 1e-6, h=r.view(4, 8), match="same array")
    _refused(F.residual_norm, r, w, 1e-6, r_out=r, h=r, match="same array")
    for kw in (dict(r_out=_t(4, 8), h=r), dict(y=_t(4, 8), h=r), dict(h=_t(4, 8))):
        _refused(F.residual_norm, r, w, 1e-6, **kw, match="no CPU path")  # taken
