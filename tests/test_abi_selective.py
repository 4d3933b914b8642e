"""Refusals of the selective scan, its step, the conv1d step and the verification, before any launch (CPU only)."""
import ctypes

import pytest
import torch

import mamba2_ssd_varlen_gb300 as m
import workloads

_FAKE = 0x7F0000000000
_P = ctypes.c_void_p(_FAKE)


@pytest.fixture(scope="module")
def lib():
    from mamba2_ssd_varlen_gb300 import build
    build.build()
    return m.load_library()


def _fill(cls, base, kw):
    base = dict(base, **kw)
    return cls(*[base[n] for n, _ in cls._fields_])


def _dims(**kw):
    return _fill(m.ssd_selective_dims, dict(T=8, R=2, D=64, N=16, G=1, dtype=m.DTYPE_BF16, num_slots=4, block_size=0,
                                            block_table_width=0, softplus=1, reserved=0, u_stride=0, delta_stride=0,
                                            B_stride=0, C_stride=0, z_stride=0, y_stride=0), kw)


def _scan_io(**kw):
    base = {n: _P for n, _ in m.ssd_selective_io._fields_}
    base.update(block_table=None, workspace_bytes=1 << 40)
    return _fill(m.ssd_selective_io, base, kw)


def _step_io(**kw):
    return _fill(m.ssd_selective_step_io, {n: _P for n, _ in m.ssd_selective_step_io._fields_}, kw)


def _scan(lib, d, io, cu=_P):
    return lib.ssd_varlen_selective_scan(ctypes.byref(d), cu, ctypes.byref(io), None)


def _step(lib, d, io, cu=_P):
    return lib.ssd_varlen_selective_step(ctypes.byref(d), cu, ctypes.byref(io), None)


def test_struct_sizes():
    assert ctypes.sizeof(m.ssd_selective_dims) == 96
    assert ctypes.sizeof(m.ssd_selective_io) == 18 * 8
    assert ctypes.sizeof(m.ssd_selective_step_io) == 13 * 8
    assert ctypes.sizeof(m.ssd_verify_dims) == 40
    assert ctypes.sizeof(m.ssd_verify_io) == 10 * 8


BAD_DIMS = [(dict(R=0), -2), (dict(T=-1), -2), (dict(D=0), -2), (dict(N=0), -2), (dict(G=0), -2), (dict(reserved=1), -2),
            (dict(num_slots=-1), -2), (dict(G=3), -4), (dict(dtype=5), -6), (dict(N=257), -11), (dict(u_stride=63), -2),
            (dict(delta_stride=-64), -2), (dict(B_stride=15), -2), (dict(C_stride=1 << 40), -2), (dict(z_stride=10), -2),
            (dict(y_stride=63), -2)]


@pytest.mark.parametrize("kw,code", BAD_DIMS + [(dict(block_size=-16), -2), (dict(block_table_width=-1), -2)])
def test_scan_rejects_bad_dims(lib, kw, code):
    assert _scan(lib, _dims(**kw), _scan_io()) == code


@pytest.mark.parametrize("kw,code", BAD_DIMS + [(dict(num_slots=0), -2)])
def test_step_rejects_bad_dims(lib, kw, code):
    assert _step(lib, _dims(**kw), _step_io()) == code


@pytest.mark.parametrize("field", ["u", "delta", "A", "B", "C", "y", "device_err", "state_pool"])
def test_scan_and_step_reject_null(lib, field):
    assert _scan(lib, _dims(), _scan_io(**{field: None})) == -1
    assert _step(lib, _dims(), _step_io(**{field: None})) == -1
    assert _scan(lib, _dims(), _scan_io(), None) == -1
    assert _step(lib, _dims(), _step_io(), None) == -1
    assert _step(lib, _dims(), _step_io(read_slots=None)) == -1


@pytest.mark.parametrize("field,by", [("u", 1), ("delta", 1), ("B", 1), ("C", 1), ("z", 1), ("y", 1), ("A", 2),
                                      ("D", 2), ("delta_bias", 2), ("state_pool", 2), ("device_err", 2)])
def test_scan_and_step_reject_misaligned(lib, field, by):
    bad = ctypes.c_void_p(_FAKE + by)
    assert _scan(lib, _dims(), _scan_io(**{field: bad})) == -7
    assert _step(lib, _dims(), _step_io(**{field: bad})) == -7
    if by == 1:
        assert _scan(lib, _dims(dtype=m.DTYPE_F32), _scan_io(**{field: ctypes.c_void_p(_FAKE + 2)})) == -7


def test_scan_block_table_and_pool(lib):
    for bs in (0, 8, 24):
        assert _scan(lib, _dims(block_size=bs, block_table_width=2), _scan_io(block_table=_P)) == -5
    for field in ("init_slots", "final_slots"):
        only = dict(init_slots=None, final_slots=None, state_pool=None)
        only[field] = _P
        assert _scan(lib, _dims(), _scan_io(**only)) == -1
    assert _scan(lib, _dims(num_slots=0), _scan_io()) == -1


def test_scan_workspace(lib):
    d = _dims(T=1 << 17, R=1, D=256)
    need = m.ssd_varlen_selective_scan_workspace(d)
    if need:
        assert _scan(lib, d, _scan_io(workspace=None)) == -8
        assert _scan(lib, d, _scan_io(workspace_bytes=need - 1)) == -8
        assert _scan(lib, d, _scan_io(workspace=ctypes.c_void_p(_FAKE + 4))) == -8
    assert m.ssd_varlen_selective_scan_workspace(_dims(D=0)) == 0


def _conv_io(**kw):
    return _fill(m.ssd_conv_io, {n: _P for n, _ in m.ssd_conv_io._fields_}, kw)


def _conv(lib, d, io, cu=_P):
    return lib.ssd_varlen_conv1d_step(ctypes.byref(d), cu, ctypes.byref(io), None)


@pytest.mark.parametrize("kw,code", [(dict(R=0), -2), (dict(T=-1), -2), (dict(D=0), -2), (dict(num_slots=-1), -2),
                                     (dict(dtype=9), -6), (dict(W=1), -11), (dict(W=5), -11), (dict(num_slots=0), -1)])
def test_conv_step_rejects_bad_dims(lib, kw, code):
    d = _fill(m.ssd_conv_dims, dict(T=8, R=2, D=65, W=4, dtype=m.DTYPE_BF16, num_slots=4, silu=1), kw)
    assert _conv(lib, d, _conv_io()) == code


def test_conv_step_rejects_bad_pointers(lib):
    d = m.ssd_conv_dims(8, 2, 65, 4, m.DTYPE_BF16, 4, 1)
    for field in ("x", "y", "weight", "device_err", "conv_pool"):
        assert _conv(lib, d, _conv_io(**{field: None})) == -1
    assert _conv(lib, d, _conv_io(), None) == -1
    for field, by in [("x", 1), ("y", 1), ("conv_pool", 1), ("weight", 2), ("bias", 2), ("read_slots", 2)]:
        assert _conv(lib, d, _conv_io(**{field: ctypes.c_void_p(_FAKE + by)})) == -7


def _verify_dims(**kw):
    return _fill(m.ssd_verify_dims, dict(T=8, R=2, V=100, dtype=m.DTYPE_F32, reserved=0, target_stride=0,
                                         draft_stride=0), kw)


def _verify_io(**kw):
    return _fill(m.ssd_verify_io, {n: _P for n, _ in m.ssd_verify_io._fields_}, kw)


def _verify(lib, d, io, cu=_P):
    return lib.ssd_varlen_verify(ctypes.byref(d), cu, ctypes.byref(io), None)


@pytest.mark.parametrize("kw,code", [(dict(R=0), -2), (dict(T=-1), -2), (dict(V=0), -2), (dict(V=(1 << 22) + 1), -2),
                                     (dict(reserved=1), -2), (dict(dtype=3), -6), (dict(target_stride=99), -2),
                                     (dict(draft_stride=-100), -2)])
def test_verify_rejects_bad_dims(lib, kw, code):
    assert _verify(lib, _verify_dims(**kw), _verify_io()) == code


def test_verify_rejects_bad_pointers(lib):
    for field in ("target", "tokens", "accept_u", "sample_u", "accepted", "out_tokens", "device_err", "write_slots",
                  "next_slots"):
        assert _verify(lib, _verify_dims(), _verify_io(**{field: None})) == -1
    assert _verify(lib, _verify_dims(), _verify_io(), None) == -1
    for field in ("target", "draft", "tokens", "accept_u", "sample_u", "next_slots"):
        assert _verify(lib, _verify_dims(), _verify_io(**{field: ctypes.c_void_p(_FAKE + 2)})) == -7
    assert _verify(lib, _verify_dims(dtype=m.DTYPE_BF16), _verify_io(target=ctypes.c_void_p(_FAKE + 1))) == -7


def test_binding_refuses_wrong_tensors(lib):
    good = workloads.make_selective_problem([4, 3], D=8, N=4)
    m.SelectiveScanCall(good)
    for name, bad in [("delta", good["delta"].float()), ("delta", good["delta"][:, :4]), ("delta", good["delta"][:5]),
                      ("z", good["z"][:1].expand(7, 8)), ("u", good["u"].half()), ("A", good["A"].double()),
                      ("B", good["B"][:, :, ::2]), ("D", good["D"][:4]), ("state_pool", good["state_pool"][:, :, :3])]:
        with pytest.raises(ValueError):
            m.SelectiveScanCall(dict(good, **{name: bad}))
    v = workloads.make_verify_problem([3, 2], V=20)
    m.VerifyCall(v)
    for name, bad in [("draft", v["draft"][:3]), ("draft", v["draft"].bfloat16()), ("tokens", v["tokens"].long()),
                      ("target", v["target"][:1].expand(5, 20)), ("sample_u", v["sample_u"].double()),
                      ("write_slots", v["write_slots"][:2])]:
        with pytest.raises(ValueError):
            m.VerifyCall(dict(v, **{name: bad}))
