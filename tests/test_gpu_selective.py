"""GPU parity of the selective scan (prefill and windows) with the fp64 oracle, through the C ABI.

Every value is held to the oracle's running bound of one fp32 evaluation of the formulas (oracle.selective): a
bf16 y lies between the bf16 roundings of the reference minus and plus that bound (rounding is monotonic).  Slots
that a call does not write keep their bits.
"""
import numpy as np
import pytest
import torch

import mamba2_ssd_varlen_gb300 as m
import workloads
from oracle.selective import selective_scan, selective_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mamba2_ssd_varlen_gb300 import build
    build.build()
    m.load_library()


def held(got, ref, tol, what):
    got = got.detach().float().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, what
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    over = np.abs(got - ref) / (tol + 1e-30)
    k = int(np.argmax(over)) if over.size else 0
    assert over.size == 0 or over.flat[k] <= 1.0, (
        f"{what}: |err| is {over.flat[k]:.3f} of its bound at {np.unravel_index(k, over.shape)}")


def bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double()


def check(prob, call, ref, before):
    torch.cuda.synchronize()
    assert call.status() == 0
    if prob["dtype"] == "bf16":
        got, lo, hi = call.y.double().cpu(), bf16(ref["y"] - ref["y_tol"]), bf16(ref["y"] + ref["y_tol"])
        assert bool(((got >= lo) & (got <= hi)).all()), "y"
    else:
        held(call.y, ref["y"], ref["y_tol"], "y")
    pool = prob["state_pool"].cpu()
    for s, v in ref["writes"].items():
        held(pool[s], v, ref["writes_tol"][s], f"state_pool[{s}]")
    rest = [s for s in range(pool.shape[0]) if s not in ref["writes"]]
    assert torch.equal(pool[rest], before.cpu()[rest])


def scan(**kw):
    prob = workloads.make_selective_problem(device="cuda", canary=-7.0, **kw)
    before, ref = prob["state_pool"].clone(), selective_scan(workloads.to_oracle_plain(prob))
    call = m.run_selective_scan(prob)
    check(prob, call, ref, before)
    held(call.final_states, ref["final_states"], ref["final_tol"], "final_states")
    return prob, call


def step(**kw):
    prob = workloads.make_selective_step_problem(device="cuda", **kw)
    before, ref = prob["state_pool"].clone(), selective_step(workloads.to_oracle_plain(prob))
    check(prob, m.run_selective_step(prob), ref, before)


EDGES = [5, 0, 1, 17, 42, 16, 15, 33]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 9, 12, 16, 17, 24, 31, 32, 33, 48, 64, 65, 100, 128, 200, 256])
def test_state_sizes(N, dtype):
    scan(lengths=EDGES, D=40, N=N, dtype=dtype, seed=N)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 31, 32, 33, 64, 72, 200])
def test_widths_and_layouts(D, layout, dtype):
    scan(lengths=EDGES, D=D, layout=layout, dtype=dtype, seed=D)


@pytest.mark.parametrize("N", [5, 16, 20])
@pytest.mark.parametrize("D,G", [(64, 2), (96, 4), (36, 4), (24, 8), (15, 5), (6, 6), (256, 2)])
def test_groups(D, G, N):
    scan(lengths=[19, 40, 3], D=D, G=G, N=N, seed=G)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("bias,softplus", [(True, True), (False, True), (True, False), (False, False)])
def test_options(z, skip, bias, softplus, dtype):
    scan(lengths=[30, 1, 50], D=48, z=z, skip=skip, bias=bias, softplus=softplus, dtype=dtype)


@pytest.mark.parametrize("block", [16, 64, 144])
@pytest.mark.parametrize("N", [16, 13])
def test_block_checkpoints_at_absolute_positions(block, N):
    scan(lengths=[200, 0, 1, 33, 160, 16], D=40, N=N, block_size=block, num_computed=[0, 5, 15, 47, 128, 16],
         init_every=1, seed=block)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths,D", [([3000], 40), ([1, 2500, 700], 24), ([1025] * 3, 64), ([4097], 8)])
def test_long_requests(lengths, D, dtype):
    # few rows and a long axis: where the scan may split a request over the time
    scan(lengths=lengths, D=D, dtype=dtype, init_every=1)


def test_long_request_with_block_checkpoints():
    scan(lengths=[3000, 700], D=33, N=20, block_size=256, num_computed=[100, 999], init_every=1)


@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("lengths", [[0, 3000, 0, 5], [0, 0, 2100], [2049, 0, 1]])
def test_long_and_empty_requests(lengths, layout):
    scan(lengths=lengths, D=41, layout=layout, init_every=1, block_size=512, num_computed=[7] * len(lengths))


def test_long_requests_with_bad_arguments():
    kw = dict(lengths=[3000, 1200], D=40, device="cuda", init_every=1, block_size=256, num_computed=[0, 0])
    clean = m.run_selective_scan(workloads.make_selective_problem(**kw))
    assert m.ssd_varlen_selective_scan_workspace(clean.dims) > 0  # split over the time
    for cu in ([0, 4300, 4200], [5, 3000, 4200], [0, 3000, 4100], [0, -7, 4200]):
        prob = workloads.make_selective_problem(**kw)
        prob["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        assert m.run_selective_scan(prob).status() & m.DEVERR["CU_SEQLENS"]
    for field, bit in [("init_slots", "INIT_SLOT"), ("final_slots", "FINAL_SLOT"), ("block_table", "BLOCK_SLOT")]:
        prob = workloads.make_selective_problem(**kw)
        prob[field].view(-1)[-1 if field != "init_slots" else 0] = 5000
        if field == "block_table":
            prob[field][0, 10] = 5000
        assert m.run_selective_scan(prob).status() == m.DEVERR[bit]


def test_many_short_requests():
    scan(lengths=[(7 * i) % 23 for i in range(300)], D=40)


@pytest.mark.parametrize("steps", [20.0, 90.0])
def test_steps_far_outside_the_usual(steps):
    # softplus where exp(v) overflows fp32 on one side and is lost on the other; decays that underflow
    prob = workloads.make_selective_problem([64, 9], D=40, dtype="fp32", device="cuda", seed=9, init_every=1)
    prob["delta"].mul_(steps)
    ref = selective_scan(workloads.to_oracle_plain(prob))
    call = m.run_selective_scan(prob)
    torch.cuda.synchronize()
    tiny = 1e-35 * (1 + np.max(np.abs(ref["y"])))  # terms below fp32's normal range may be lost
    held(call.y, ref["y"], ref["y_tol"] + tiny, "y")
    held(call.final_states, ref["final_states"], ref["final_tol"] + tiny, "final_states")


def test_gate_far_outside_the_usual():
    prob = workloads.make_selective_problem([40], D=40, dtype="fp32", device="cuda", seed=3)
    prob["z"].mul_(60.0)
    ref = selective_scan(workloads.to_oracle_plain(prob))
    call = m.run_selective_scan(prob)
    torch.cuda.synchronize()
    held(call.y, ref["y"], ref["y_tol"] + 1e-30, "y")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["u", "z", "delta"])
def test_a_bad_value_stays_in_its_request_and_channel(name, bad):
    kw = dict(lengths=[20, 21, 22], D=40, N=16, dtype="bf16", device="cuda", seed=6)
    clean = m.run_selective_scan(workloads.make_selective_problem(**kw))
    prob = workloads.make_selective_problem(**kw)
    prob[name][20 + 5, 3] = bad
    call = m.run_selective_scan(prob)
    torch.cuda.synchronize()
    same = call.y.view(torch.int16) == clean.y.view(torch.int16)
    hit = torch.zeros_like(same)
    hit[25:41, 3] = True
    assert bool(same[~hit].all())
    assert not bool(torch.isfinite(call.y[25, 3]))
    ok = torch.ones_like(call.final_states, dtype=torch.bool)
    ok[1, 3] = False
    assert torch.equal(call.final_states[ok], clean.final_states[ok])


def test_all_requests_empty():
    prob = workloads.make_selective_problem([0, 0, 0], D=40, device="cuda", init_every=2, seed=1, canary=3.0)
    before = prob["state_pool"].clone()
    call = m.run_selective_scan(prob)
    torch.cuda.synchronize()
    assert call.status() == 0
    for i, (r, w) in enumerate(zip(prob["init_slots"].tolist(), prob["final_slots"].tolist())):
        want = before[r] if r >= 0 else torch.zeros_like(before[0])
        assert torch.equal(prob["state_pool"][w], want)
        assert torch.equal(call.final_states[i], want)


def test_device_errors_skip_what_is_bad():
    kw = dict(lengths=[20, 30], D=40, block_size=16, num_computed=[0, 0], init_every=1, device="cuda", seed=2)
    clean = m.run_selective_scan(workloads.make_selective_problem(**kw))
    for field, value, bit in [("init_slots", 1000, "INIT_SLOT"), ("final_slots", 1000, "FINAL_SLOT"),
                              ("block_table", 1000, "BLOCK_SLOT"), ("num_computed", -5, "NUM_COMPUTED")]:
        prob = workloads.make_selective_problem(**kw)
        prob[field].view(-1)[0] = value
        call = m.run_selective_scan(prob)
        torch.cuda.synchronize()
        assert call.status() == m.DEVERR[bit], field
        assert torch.equal(call.y[20:], clean.y[20:])
    prob = workloads.make_selective_problem(**kw)
    prob["block_table"] = prob["block_table"][:, :1].contiguous()
    narrow = m.run_selective_scan(prob)
    torch.cuda.synchronize()
    # 20 tokens cross one boundary, 30 tokens one: a table of one column is enough
    assert narrow.status() == 0 and torch.equal(narrow.y, clean.y)
    prob = workloads.make_selective_problem(**kw)
    prob["num_computed"][1] = 400
    call = m.run_selective_scan(prob)
    assert call.status() == m.DEVERR["BLOCK_TABLE"] and torch.equal(call.y, clean.y)
    for cu in ([1, 20, 50], [0, 51, 50], [0, 20, 49], [0, -1, 50]):
        prob = workloads.make_selective_problem(**kw)
        prob["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        assert m.run_selective_scan(prob).status() & m.DEVERR["CU_SEQLENS"]


@pytest.mark.parametrize("lengths,D,N", [([300, 5, 70], 72, 16), ([3000], 40, 16), ([100], 33, 20)])
def test_calls_repeat_bit_for_bit_on_any_stream(lengths, D, N):
    kw = dict(lengths=lengths, D=D, N=N, device="cuda", seed=8)
    a = m.run_selective_scan(workloads.make_selective_problem(**kw))
    prob = workloads.make_selective_problem(**kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = m.SelectiveScanCall(prob, stream=side)
    for _ in range(3):
        b()
    side.synchronize()
    assert torch.equal(a.y, b.y) and torch.equal(a.final_states, b.final_states)
    g = torch.cuda.CUDAGraph()
    prob = workloads.make_selective_problem(**kw)
    c = m.SelectiveScanCall(prob)
    c()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c()
    c.y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.y, c.y) and torch.equal(a.final_states, c.final_states)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 3, 4, 8, 13, 16, 20, 32, 50, 64, 128, 256])
def test_step_state_sizes(N, dtype):
    step(windows=[1, 4, 0, 2, 9, 1], D=40, N=N, dtype=dtype, seed=N)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("D", [1, 7, 32, 33, 64, 200, 520])
def test_step_widths_and_layouts(D, layout, dtype):
    step(windows=[1, 4, 0, 2], D=D, layout=layout, dtype=dtype, seed=D)


@pytest.mark.parametrize("D,G", [(64, 2), (36, 4), (24, 8), (15, 5)])
@pytest.mark.parametrize("N", [5, 16])
def test_step_groups(D, G, N):
    step(windows=[1, 3], D=D, G=G, N=N)


@pytest.mark.parametrize("z,skip,bias,softplus", [(False, True, True, True), (True, False, False, True),
                                                  (True, True, True, False), (False, False, False, False)])
def test_step_options(z, skip, bias, softplus):
    step(windows=[1, 3, 8], D=48, z=z, skip=skip, bias=bias, softplus=softplus)


def test_step_many_windows():
    step(windows=[i % 3 for i in range(700)], D=24, N=4)


def test_step_without_write_slots_and_device_errors():
    kw = dict(windows=[2, 1], D=40, device="cuda", zero_every=0, skip_every=0)
    clean = m.run_selective_step(workloads.make_selective_step_problem(**kw))
    prob = workloads.make_selective_step_problem(**kw)
    prob["write_slots"] = None
    before = prob["state_pool"].clone()
    call = m.run_selective_step(prob)
    torch.cuda.synchronize()
    assert call.status() == 0 and torch.equal(call.y, clean.y) and torch.equal(prob["state_pool"], before)
    for field, bit in [("read_slots", "INIT_SLOT"), ("write_slots", "FINAL_SLOT")]:
        prob = workloads.make_selective_step_problem(**kw)
        prob[field][0] = 100
        call = m.run_selective_step(prob)
        assert call.status() == m.DEVERR[bit]
        assert torch.equal(call.y[2:], clean.y[2:])
    for cu in ([1, 2, 3], [0, 4, 3], [0, 2, 2]):
        prob = workloads.make_selective_step_problem(**kw)
        prob["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        assert m.run_selective_step(prob).status() & m.DEVERR["CU_SEQLENS"]


def test_state_pool_past_32_bit_offsets():
    # the last slot of a pool of 2^31 + elements: its offset does not fit 32 bits
    D, N = 4096, 64
    slots = 2 ** 31 // (D * N) + 3
    prob = workloads.make_selective_step_problem([1, 1], D=D, N=N, device="cuda", seed=5, zero_every=0, skip_every=0)
    small = prob["state_pool"]
    small_out = m.run_selective_step(dict(prob, state_pool=small.clone()))
    pool = torch.zeros((slots, D, N), dtype=torch.float32, device="cuda")
    at = torch.tensor([slots - 4, slots - 3, slots - 2, slots - 1], device="cuda")
    pool[at] = small
    big = dict(prob, state_pool=pool, read_slots=at[prob["read_slots"].long()].int(),
               write_slots=at[prob["write_slots"].long()].int())
    call = m.run_selective_step(big)
    torch.cuda.synchronize()
    ref = dict(prob, state_pool=small)
    m.run_selective_step(ref)
    torch.cuda.synchronize()
    assert call.status() == 0 and torch.equal(call.y, small_out.y)
    assert torch.equal(pool[at], ref["state_pool"])
