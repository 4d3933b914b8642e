"""Plain fp64 selective scan (S6), token by token: the oracle of ssd_varlen_selective_scan and
ssd_varlen_selective_step, with a running bound of what fp32 arithmetic may be off by.

    dt' = softplus(delta + bias)                        (or delta + bias)
    h   = exp(dt' A) h + dt' u B ;  y = (C . h + D u) silu(z)

The bound follows one fp32 evaluation of these formulas.  With eps = 2^-24 (half a unit in the last
place), dt' is off by a relative TAU, exp(x) by a relative 2^-22 (the documented error of the hardware's
2^x) + |x| (TAU + 4 eps) (the rounding of its argument), dt' u B by TAU + 4 eps, and each state update
rounds twice.  So with e the bound of the state before the token,
    e <- a (e + |h| rho) + |b| (TAU + 4 eps) + 2 eps |h_new|
and y is off by sum |C| e + (N + 4) eps sum |C h| + ... , times the gate and its own error.
"""
import numpy as np

EPS = 2.0 ** -24
TAU = 2.0 ** -21   # the step: an exponential, a logarithm and their sum, each good to a few units
RHO = 2.0 ** -22


def _softplus(v):
    return np.logaddexp(v, 0.0)


def _walk(p, t0, t1, h, after):
    """Tokens t0..t1-1 from state h (D,N); after(t, h, e) sees the state after each. Returns y, its bound, h, e."""
    A, D, N, G = p["A"], p["A"].shape[0], p["A"].shape[1], p["B"].shape[1]
    e = np.zeros_like(h)
    y, ye = np.zeros((t1 - t0, D)), np.zeros((t1 - t0, D))
    for t in range(t0, t1):
        v = p["delta"][t] + (0.0 if p["delta_bias"] is None else p["delta_bias"])
        if p["softplus"]:
            dt = _softplus(v)
            # v rounds once before the softplus, whose slope is the sigmoid
            off = dt * TAU + EPS * np.abs(v) / (1.0 + np.exp(-v))
        else:
            dt, off = v, EPS * np.abs(v)
        dt, off = dt[:, None], off[:, None]
        u = p["u"][t][:, None]
        B = np.repeat(p["B"][t], D // G, 0)
        C = np.repeat(p["C"][t], D // G, 0)
        x = dt * A
        a, b = np.exp(x), dt * u * B
        ae = a * (RHO + off * np.abs(A) + 4 * EPS * np.abs(x))
        be = np.abs(off * u * B) + 4 * EPS * np.abs(b)
        new = a * h + b
        e = a * e + ae * (np.abs(h) + e) + be + 2 * EPS * np.abs(new)
        h = new
        s = (C * h).sum(1)
        se = (np.abs(C) * e).sum(1) + (N + 4) * EPS * (np.abs(C * h)).sum(1)
        if p["D"] is not None:
            s = s + p["D"] * p["u"][t]
            se = se + 4 * EPS * np.abs(p["D"] * p["u"][t])
        if p["z"] is not None:
            z = p["z"][t]
            gate = z / (1.0 + np.exp(-z))
            se = se * np.abs(gate) + np.abs(s * gate) * (8 * EPS + RHO * (1.0 + np.abs(z)))
            s = s * gate
        y[t - t0], ye[t - t0] = s, se + EPS * np.abs(s)
        after(t, h, e)
    return y, ye, h, e


def selective_scan(p):
    """p: fp64 arrays u, delta, z (T,D); B, C (T,G,N); A (D,N); D, delta_bias (D) or None; softplus; cu_seqlens;
    num_computed, init_slots, final_slots, block_table, state_pool or None; block_size.
    Returns y, final_states, writes {slot: state} and their bounds (*_tol)."""
    D, N = p["A"].shape
    cu = [int(v) for v in p["cu_seqlens"]]
    R = len(cu) - 1
    y, yt = np.zeros((cu[-1], D)), np.zeros((cu[-1], D))
    fin, ft, writes, wt = np.zeros((R, D, N)), np.zeros((R, D, N)), {}, {}
    for i in range(R):
        h = np.zeros((D, N))
        if p.get("init_slots") is not None and 0 <= int(p["init_slots"][i]) < p["state_pool"].shape[0]:
            h = p["state_pool"][int(p["init_slots"][i])].copy()
        s = 0 if p.get("num_computed") is None else int(p["num_computed"][i])

        def after(t, h, e, i=i, s=s):
            pos = s + t - cu[i] + 1
            if p.get("block_table") is None or pos % p["block_size"]:
                return
            col = pos // p["block_size"] - 1
            if col < p["block_table"].shape[1] and 0 <= int(p["block_table"][i][col]) < p["state_pool"].shape[0]:
                slot = int(p["block_table"][i][col])
                writes[slot], wt[slot] = h.copy(), e.copy()

        y[cu[i]:cu[i + 1]], yt[cu[i]:cu[i + 1]], h, e = _walk(p, cu[i], cu[i + 1], h, after)
        fin[i], ft[i] = h, e
        if p.get("final_slots") is not None and 0 <= int(p["final_slots"][i]) < p["state_pool"].shape[0]:
            writes[int(p["final_slots"][i])], wt[int(p["final_slots"][i])] = h, e
    return {"y": y, "y_tol": yt, "final_states": fin, "final_tol": ft, "writes": writes, "writes_tol": wt}


def selective_step(p):
    """The same over windows: read_slots (R), write_slots (T) or None. Returns y and writes, with bounds."""
    D, N = p["A"].shape
    cu = [int(v) for v in p["cu_seqlens"]]
    y, yt, writes, wt = np.zeros((cu[-1], D)), np.zeros((cu[-1], D)), {}, {}
    for i in range(len(cu) - 1):
        h, r = np.zeros((D, N)), int(p["read_slots"][i])
        if 0 <= r < p["state_pool"].shape[0]:
            h = p["state_pool"][r].copy()

        def after(t, h, e):
            w = -1 if p.get("write_slots") is None else int(p["write_slots"][t])
            if 0 <= w < p["state_pool"].shape[0]:
                writes[w], wt[w] = h.copy(), e.copy()

        y[cu[i]:cu[i + 1]], yt[cu[i]:cu[i + 1]], _, _ = _walk(p, cu[i], cu[i + 1], h, after)
    return {"y": y, "y_tol": yt, "writes": writes, "writes_tol": wt}
