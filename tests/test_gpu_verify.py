"""GPU parity of the draft verification with the whole-number oracle: every result equal, bit for bit."""
import numpy as np
import pytest
import torch

import mamba2_ssd_varlen_gb300 as m
import workloads
from oracle.verify import verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mamba2_ssd_varlen_gb300 import build
    build.build()
    m.load_library()


def check(prob, bits=0):
    prob = dict(prob)
    R = prob["cu_seqlens"].shape[0] - 1
    prob["next_slots"] = torch.arange(1000, 1000 + R, dtype=torch.int32, device="cuda")
    ref = verify(workloads.to_oracle_plain(prob))
    call = m.run_verify(prob)
    torch.cuda.synchronize()
    assert call.status() == bits
    np.testing.assert_array_equal(call.accepted.cpu().numpy(), ref["accepted"])
    np.testing.assert_array_equal(call.out_tokens.cpu().numpy(), ref["out_tokens"])
    np.testing.assert_array_equal(call.next_slots.cpu().numpy(), ref["next_slots"])
    return ref


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("V", [1, 2, 7, 100, 257, 1000, 1024, 4099])
def test_vocabularies_and_layouts(V, layout, dtype):
    check(workloads.make_verify_problem([4, 1, 0, 6, 2, 9], V, dtype=dtype, seed=V, device="cuda", layout=layout))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [32003, 70000, 131072])
def test_large_vocabularies(V, dtype):
    check(workloads.make_verify_problem([4, 1, 3], V, dtype=dtype, seed=V, device="cuda", scale=3.0))


@pytest.mark.parametrize("keep", [0, 1, 5])
@pytest.mark.parametrize("draft", [True, False])
def test_masked_targets_and_drafts_without_a_distribution(keep, draft):
    ref = check(workloads.make_verify_problem([5] * 30, 300, seed=keep, device="cuda", draft=draft, keep=keep,
                                              near=0.2))
    assert np.all(ref["out_tokens"].reshape(30, 5)[np.arange(30), ref["accepted"]] >= 0)


def test_many_windows():
    check(workloads.make_verify_problem([i % 6 for i in range(400)], 500, seed=1, device="cuda"))


def test_every_draft_accepted_and_none():
    prob = workloads.make_verify_problem([6] * 8, 200, seed=2, device="cuda")
    prob["draft"] = prob["target"].clone()
    prob["accept_u"] *= 0.999
    assert np.all(check(prob)["accepted"] == 5)
    prob["accept_u"] = torch.full_like(prob["accept_u"], 2.0)
    # rejected with target == draft: no residual is positive, so the target's own row is drawn from
    ref = check(prob)
    assert np.all(ref["accepted"] == 0) and np.all(ref["out_tokens"][::6] >= 0)


@pytest.mark.parametrize("u", [0.0, 1e-30, 0.5, 1.0 - 2 ** -24, 1.0, -1.0, float("nan"), float("inf")])
def test_edges_of_the_random_number(u):
    prob = workloads.make_verify_problem([1, 3, 4], 777, seed=3, device="cuda")
    prob["sample_u"].fill_(u)
    check(prob)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), -1.0, 1e30, 1e-40])
def test_values_that_are_no_probabilities(bad):
    prob = workloads.make_verify_problem([1, 3, 4], 300, seed=4, device="cuda")
    prob["target"][:, 5::7] = bad
    prob["target"][2] = bad
    check(prob)
    prob["draft"][:, 3::11] = bad
    check(prob)


def test_rows_without_a_weight():
    prob = workloads.make_verify_problem([1, 3], 90, seed=5, device="cuda")
    prob["target"].zero_()
    ref = check(prob)
    assert ref["out_tokens"][0] == -1 and ref["out_tokens"][1] == -1


def test_drafts_outside_the_vocabulary():
    prob = workloads.make_verify_problem([3, 3], 90, seed=6, device="cuda")
    prob["tokens"][1], prob["tokens"][4] = 90, -3
    check(prob, m.DEVERR["TOKEN"])
    prob["draft"] = None
    check(prob, m.DEVERR["TOKEN"])


def test_bad_windows_and_no_windows():
    prob = workloads.make_verify_problem([2, 3], 90, seed=7, device="cuda")
    for cu in ([1, 2, 5], [0, 6, 5], [0, 2, 4], [0, -1, 5]):
        bad = dict(prob, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert m.run_verify(bad).status() & m.DEVERR["CU_SEQLENS"]
    prob = workloads.make_verify_problem([0, 0], 90, seed=7, device="cuda")
    assert np.all(check(prob)["accepted"] == -1)


def test_without_slots_in_place_on_another_stream_and_in_a_graph():
    prob = workloads.make_verify_problem([4, 0, 2], 3000, seed=8, device="cuda")
    ref = check(prob)
    bare = m.run_verify(dict(prob, write_slots=None))
    assert bare.next_slots is None
    anchors = torch.tensor([70, 71, 72], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call = m.VerifyCall(dict(prob, next_slots=anchors), stream=side)
    call()
    side.synchronize()
    assert anchors[1].item() == 71 and anchors[0].item() == ref["next_slots"][0]
    torch.cuda.synchronize()
    g, c = torch.cuda.CUDAGraph(), m.VerifyCall(prob)
    with torch.cuda.graph(g):
        c()
    g.replay()
    torch.cuda.synchronize()
    for got in (bare, call, c):
        np.testing.assert_array_equal(got.out_tokens.cpu().numpy(), ref["out_tokens"])
