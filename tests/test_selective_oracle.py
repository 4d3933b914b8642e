"""The oracles of the selective scan and of the draft verification, pinned by independent forms (CPU)."""
import numpy as np
import pytest
import torch

import workloads
from oracle.selective import selective_scan, selective_step
from oracle.verify import draw, verify


def _prob(**kw):
    return workloads.to_oracle_plain(workloads.make_selective_problem(dtype="fp32", **kw))


@pytest.mark.parametrize("G", [1, 2])
def test_scan_equals_the_materialised_sum(G):
    # y_t = sum_s C_t . (exp(A (S_t - S_s)) dt_s u_s B_s), every pair of tokens written out
    p = _prob(lengths=[9], D=4, N=3, G=G, init_every=0, seed=G)
    r = selective_scan(p)
    dt = np.logaddexp(p["delta"] + p["delta_bias"], 0.0)
    S = np.cumsum(dt, 0)
    rep = 4 // G
    for t in range(9):
        y = np.zeros(4)
        for s in range(t + 1):
            w = np.exp(p["A"] * (S[t] - S[s])[:, None]) * (dt[s] * p["u"][s])[:, None] * np.repeat(p["B"][s], rep, 0)
            y += (np.repeat(p["C"][t], rep, 0) * w).sum(1)
        z = p["z"][t]
        y = (y + p["D"] * p["u"][t]) * z / (1 + np.exp(-z))
        np.testing.assert_allclose(r["y"][t], y, rtol=1e-12, atol=1e-12)


def test_scan_without_decay_is_a_cumulative_sum():
    p = _prob(lengths=[7], D=3, N=2, z=False, skip=False, init_every=0)
    p["A"] = np.zeros_like(p["A"])
    dt = np.logaddexp(p["delta"] + p["delta_bias"], 0.0)
    h = np.cumsum((dt * p["u"])[:, :, None] * p["B"], 0)
    np.testing.assert_allclose(selective_scan(p)["y"], (h * p["C"]).sum(2), rtol=1e-12)


def test_packed_equals_separate_and_split_equals_whole():
    p = _prob(lengths=[6, 0, 11], D=5, N=4, init_every=1, final_slots=True, seed=4)
    whole = selective_scan(p)
    cut = dict(p, cu_seqlens=np.array([0, 6, 6, 10]), u=p["u"][:10], delta=p["delta"][:10], B=p["B"][:10],
               C=p["C"][:10], z=p["z"][:10])
    head = selective_scan(cut)
    np.testing.assert_array_equal(head["y"], whole["y"][:10])
    pool = p["state_pool"].copy()
    for s, v in head["writes"].items():
        pool[s] = v
    tail = dict(p, cu_seqlens=np.array([0, 7]), u=p["u"][10:], delta=p["delta"][10:], B=p["B"][10:], C=p["C"][10:],
                z=p["z"][10:], state_pool=pool, init_slots=p["final_slots"][2:], final_slots=None)
    r = selective_scan(tail)
    np.testing.assert_allclose(r["y"], whole["y"][10:], rtol=1e-12)
    np.testing.assert_allclose(r["final_states"][0], whole["final_states"][2], rtol=1e-12)


def test_step_equals_scan():
    p = _prob(lengths=[4, 3], D=3, N=2, init_every=1, seed=2)
    s = dict(p, read_slots=p["init_slots"], write_slots=np.array([-1, -1, -1, 0, -1, -1, 1]))
    a, b = selective_scan(p), selective_step(s)
    np.testing.assert_array_equal(a["y"], b["y"])
    np.testing.assert_array_equal(b["writes"][0], a["final_states"][0])
    np.testing.assert_array_equal(b["writes"][1], a["final_states"][1])


def test_fp32_arithmetic_stays_inside_the_bound():
    # the bound is meant for any fp32 evaluation in the written order: torch's is one
    prob = workloads.make_selective_problem([200], D=16, N=16, dtype="fp32", seed=5, init_every=1)
    ref = selective_scan(workloads.to_oracle_plain(prob))
    h = prob["state_pool"][prob["init_slots"].long()][0].clone()
    v = prob["delta"] + prob["delta_bias"]
    dt = torch.log1p(torch.exp(v))
    for t in range(200):
        h = torch.exp(dt[t, :, None] * prob["A"]) * h + (dt[t] * prob["u"][t])[:, None] * prob["B"][t]
        z = prob["z"][t]
        y = ((h * prob["C"][t]).sum(1) + prob["D"] * prob["u"][t]) * (z / (1 + torch.exp(-z)))
        assert np.all(np.abs(y.double().numpy() - ref["y"][t]) <= ref["y_tol"][t])
    assert np.all(np.abs(h.double().numpy() - ref["final_states"][0]) <= ref["final_tol"][0])
    assert np.max(ref["final_tol"]) < 1e-3 * np.max(np.abs(ref["final_states"]))  # and it bounds something


def test_verify_draws_the_target_distribution():
    # speculative sampling's property: whatever the draft's distribution, the first token after the window's own
    # follows the target's.  20000 windows over 5 tokens: a count's deviation is below 5 sqrt(n p)
    rng = np.random.default_rng(0)
    n, p, q = 20000, np.array([0.4, 0.3, 0.2, 0.1, 0.0]), np.array([0.1, 0.2, 0.3, 0.2, 0.2])
    tokens = np.zeros((n, 2), np.int32)
    tokens[:, 1] = rng.choice(5, n, p=q)
    row = lambda v: np.tile(v.astype(np.float32), (2 * n, 1))  # noqa: E731
    r = verify({"target": row(p), "draft": row(q), "tokens": tokens.reshape(-1), "cu_seqlens": np.arange(n + 1) * 2,
                "accept_u": rng.random(2 * n, dtype=np.float32), "sample_u": rng.random(n, dtype=np.float32)})
    first = r["out_tokens"].reshape(n, 2)[:, 0]
    for v in range(5):
        assert abs(np.sum(first == v) - n * p[v]) <= 5 * np.sqrt(n * p[v])


def test_draw_edges():
    assert draw([0, 0, 0], 0.5) == -1
    assert draw([0, 3, 0, 1], 0.0) == 1
    assert draw([0, 3, 0, 1], 0.74) == 1
    assert draw([0, 3, 0, 1], 0.75) == 3
    assert draw([0, 3, 0, 1], 1.0) == 3
    assert draw([0, 3, 0, 1], float("nan")) == 1
    assert draw([2, 0], -1.0) == 0
