"""Plain verification of drafted tokens (speculative sampling): the oracle of ssd_varlen_verify, in Python
whole numbers and Fractions, so that it rounds nowhere but where the definition does.

The acceptance compares accept_u * q (rounded to fp32) with p; the residual p - q is rounded to fp32; the
weights are whole multiples of 2^-40; the mark is floor(sample_u * S), the product rounded to fp64."""
import math
from fractions import Fraction

import numpy as np


def _fixed(w):
    """floor(2^40 min(max(w, 0), 1)) of an fp32 value, 0 for a NaN."""
    w = float(w)
    if not w > 0.0:
        return 0
    return int(Fraction(min(w, 1.0)) * (1 << 40))


def draw(weights, u):
    """The first v with f_0 + ... + f_v > mark; -1 where no weight is positive."""
    total = sum(weights)
    if total == 0:
        return -1
    f = float(np.float64(np.float32(u)) * np.float64(total))
    mark = 0 if not f >= 1.0 else (total if math.isinf(f) else int(math.floor(f)))
    mark = min(mark, total - 1)
    run = 0
    for v, f in enumerate(weights):
        run += f
        if run > mark:
            return v
    raise AssertionError


def verify(p):
    """p: target, draft (T,V) fp32 (draft or None), tokens (T), accept_u (T), sample_u (R), cu_seqlens,
    write_slots (T) or None, next_slots (R) or None (values before the call)."""
    cu = [int(v) for v in p["cu_seqlens"]]
    R, V = len(cu) - 1, p["target"].shape[1]
    accepted, out = np.full(R, -1, np.int32), np.full(cu[-1], -1, np.int32)
    nxt = None if p.get("next_slots") is None else np.array(p["next_slots"], np.int32).copy()
    for i in range(R):
        a, b = cu[i], cu[i + 1]
        if a == b:
            continue
        n, k = 0, b - a - 1
        while n < k:
            t, x = a + n, int(p["tokens"][a + n + 1])
            if not 0 <= x < V:
                break
            q = np.float32(1.0) if p["draft"] is None else np.float32(p["draft"][t, x])
            with np.errstate(invalid="ignore"):
                ok = np.float32(p["accept_u"][t + 1]) * q < np.float32(p["target"][t, x])
            if not ok:
                break
            n += 1
        r = a + n
        full = np.asarray(p["target"][r], np.float32)
        w = full
        if n < k:
            q = p["draft"][r] if p["draft"] is not None else (np.arange(V) == int(p["tokens"][r + 1]))
            with np.errstate(invalid="ignore"):
                w = full - np.asarray(q, np.float32)
        f = [_fixed(v) for v in w]
        if sum(f) == 0:
            f = [_fixed(v) for v in full]
        accepted[i] = n
        out[a:a + n] = p["tokens"][a + 1:a + 1 + n]
        out[r] = draw(f, p["sample_u"][i])
        if nxt is not None:
            nxt[i] = p["write_slots"][r]
    return {"accepted": accepted, "out_tokens": out, "next_slots": nxt}
