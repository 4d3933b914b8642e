"""GPU parity of the conv1d step with the fp64 oracle of the conv1d: every window as a request of its own, its
state after every token.  The states are raw inputs and must match bit for bit.

y: W fused multiply-adds and the bias, each rounding once (W + 2 units of 2^-24 of the sum of magnitudes), a
SiLU whose exponential and quotient are good to 2^-21 relative (and whose slope is at most 1.1); a bf16 y lies
between the bf16 roundings of the reference minus and plus that."""
import numpy as np
import pytest
import torch

import mamba2_ssd_varlen_gb300 as m
import workloads
from oracle.conv1d import conv1d

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mamba2_ssd_varlen_gb300 import build
    build.build()
    m.load_library()


def check(scale=1.0, **kw):
    prob = workloads.make_conv_step_problem(device="cuda", **kw)
    prob["x"].mul_(scale)
    before = prob["conv_pool"].clone()
    host = workloads.to_oracle_plain(prob)
    ref = conv1d(dict(host, write_slots=None))["y"]
    sizes = conv1d(dict(host, write_slots=None, silu=False, x=np.abs(host["x"]), weight=np.abs(host["weight"]),
                        bias=None if host["bias"] is None else np.abs(host["bias"]),
                        conv_pool=np.abs(host["conv_pool"])))["y"]
    call = m.run_conv1d_step(prob)
    torch.cuda.synchronize()
    assert call.status() == 0
    tol = 1.1 * (kw.get("W", 4) + 2) * 2.0 ** -24 * sizes + 2.0 ** -21 * np.abs(ref) + 1e-30
    lo, hi = ref - tol, ref + tol
    if prob["dtype"] == "bf16":
        lo, hi = (torch.from_numpy(v).to(torch.bfloat16).double().numpy() for v in (lo, hi))
    got = call.y.double().cpu().numpy()
    assert np.all((got >= lo) & (got <= hi))
    pool, W = prob["conv_pool"], prob["W"]
    want = before.clone()
    cu, read, write = host["cu_seqlens"], host["read_slots"], host["write_slots"]
    for i in range(prob["R"]):
        seq = before[read[i]] if read[i] >= 0 else torch.zeros_like(before[0])
        for t in range(cu[i], cu[i + 1]):
            seq = torch.cat([seq, prob["x"][t][:, None]], 1)[:, -(W - 1):]
            if write[t] >= 0:
                want[write[t]] = seq
    assert torch.equal(pool.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D", [1, 3, 8, 20, 64, 100, 264, 1030])
def test_widths(D, W, dtype):
    check(windows=[1, 4, 0, 2, 9, 1, 3], D=D, W=W, dtype=dtype, seed=D)


@pytest.mark.parametrize("silu,bias", [(False, True), (True, False), (False, False)])
def test_options(silu, bias):
    check(windows=[1, 4, 3], D=40, silu=silu, bias=bias)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_silu_over_a_wide_range(dtype):
    check(windows=[3, 4, 5], D=264, dtype=dtype, scale=25.0)


def test_many_windows():
    check(windows=[i % 4 for i in range(600)], D=24)


@pytest.mark.parametrize("D", [64, 33])
def test_without_slots_with_bad_slots_and_on_another_stream(D):
    kw = dict(windows=[2, 1], D=D, device="cuda", zero_every=0, skip_every=0)
    clean = m.run_conv1d_step(workloads.make_conv_step_problem(**kw))
    prob = workloads.make_conv_step_problem(**kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call = m.ConvStepCall(prob, stream=side)
    call()
    side.synchronize()
    assert call.status() == 0 and torch.equal(call.y, clean.y)
    prob = workloads.make_conv_step_problem(**kw)
    free = dict(prob, read_slots=None, write_slots=None)
    call = m.run_conv1d_step(free)
    zero = m.run_conv1d_step(dict(prob, read_slots=torch.full_like(prob["read_slots"], -1), write_slots=None))
    torch.cuda.synchronize()
    assert call.status() == 0 and torch.equal(call.y, zero.y)
    for field, bit in [("read_slots", "INIT_SLOT"), ("write_slots", "FINAL_SLOT")]:
        prob = workloads.make_conv_step_problem(**kw)
        prob[field][0] = 100
        call = m.run_conv1d_step(prob)
        assert call.status() == m.DEVERR[bit]
        assert torch.equal(call.y[2:], clean.y[2:])
    for cu in ([1, 2, 3], [0, 4, 3], [0, 2, 2]):
        prob = workloads.make_conv_step_problem(**kw)
        prob["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        assert m.run_conv1d_step(prob).status() & m.DEVERR["CU_SEQLENS"]
    prob = workloads.make_conv_step_problem([0, 0], D=D, device="cuda")
    assert m.run_conv1d_step(prob).status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 33])
def test_states_keep_every_bit_pattern(D, dtype):
    """Negative and payload-carrying NaN, infinities, zeros of both signs and subnormals pass through a slot."""
    prob = workloads.make_conv_step_problem(windows=[1, 3, 2], D=D, W=4, dtype=dtype, seed=2, device="cuda")
    words = [0x7FC0, 0xFFC0, 0x7F81, 0xFFFF, 0x7F80, 0xFF80, 0x0000, 0x8000, 0x0001, 0x8001, 0x3F80]
    words = [w - 0x10000 if w >= 0x8000 else w for w in words]
    for name in ("x", "conv_pool"):
        flat = prob[name].view(torch.int16).reshape(-1)
        fill = torch.tensor(words, dtype=torch.int16, device="cuda").repeat(flat.numel() // len(words) + 1)
        flat.copy_(fill[:flat.numel()])
    before = prob["conv_pool"].clone()
    call = m.run_conv1d_step(prob)
    torch.cuda.synchronize()
    assert call.status() == 0
    cu, read, write = (prob[k].tolist() for k in ("cu_seqlens", "read_slots", "write_slots"))
    want = before.clone()
    for i in range(prob["R"]):
        seq = before[read[i]] if read[i] >= 0 else torch.zeros_like(before[0])
        for t in range(cu[i], cu[i + 1]):
            seq = torch.cat([seq, prob["x"][t][:, None]], 1)[:, -3:]
            if write[t] >= 0:
                want[write[t]] = seq
    assert torch.equal(prob["conv_pool"].view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("moved", ["x", "conv_pool", "weight"])
def test_pointers_off_the_vector_boundary(moved, dtype):
    """The same problem with one tensor an element further on gives the same bits."""
    def problem():
        return workloads.make_conv_step_problem(windows=[1, 4, 2], D=64, W=4, dtype=dtype, seed=8, device="cuda")
    plain, off = problem(), problem()
    room = torch.empty(off[moved].numel() + 1, dtype=off[moved].dtype, device="cuda")
    view = room[1:].view(off[moved].shape)
    view.copy_(off[moved])
    off[moved] = view
    a, b = m.run_conv1d_step(plain), m.run_conv1d_step(off)
    torch.cuda.synchronize()
    assert a.status() == 0 and b.status() == 0
    assert torch.equal(a.y, b.y) and torch.equal(plain["conv_pool"], off["conv_pool"])
