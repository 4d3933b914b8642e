"""Cases of the selective-scan (S6) layer and of speculative decoding's verification.

Four operators, as one speculative decoding loop over a selective state space layer
uses them:

  scan    the selective scan over a packed batch of prompts (varlen, state slots,
          block checkpoints)
  step    the same recurrence for windows of single or drafted tokens, with a read
          slot for each request and a write slot for each token
  conv    the short causal convolution over such windows, its state kept after every
          token (the prompts' convolution is ssd_varlen_conv1d)
  verify  drafted tokens against the target's probabilities from given random
          numbers; the token that follows, and the slot that the next step reads

listed() and draw() give cases, prepare() their inputs, run() one pass: in elementary
torch operations, or where `own` is true through the package's entry points.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CHUNK = 64  # tokens of a chunk in the plain form of the scan


# ---------------------------------------------------------------------------- cases
def listed():
    scan = {"op": "scan", "dtype": "bf16", "N": 16, "G": 1, "z": True, "skip": True, "softplus": True,
            "init": "none", "block": 0, "sliced": True}
    step = {"op": "step", "dtype": "bf16", "N": 16, "G": 1, "z": True, "skip": True, "softplus": True, "sliced": True}
    return [
        # three short prompts, one of them continued: the smallest prefill, all latency
        dict(scan, name="scan_tiny_fp32", dtype="fp32", R=3, kind="given", lens="5,17,42", D=64, z=False, init="last",
             sliced=False),
        # an ordinary prefill batch at a 2560-wide model's inner size (80 heads of 64)
        dict(scan, name="scan_uniform_8x2048", R=8, kind="same", L=2048, D=5120),
        # mixed prompt lengths, half of them continuing a cached prefix
        dict(scan, name="scan_lognormal_64", R=64, kind="lognormal", T=32768, D=8192, init="half"),
        # one long document: few rows, a long axis
        dict(scan, name="scan_long_131072", R=1, kind="same", L=131072, D=4096),
        # ragged prompts, every block's state kept for the prefix cache, an odd width and state size, fp32
        dict(scan, name="scan_blocks_odd_fp32", dtype="fp32", R=13, kind="spread", L=3000, D=1003, N=24, init="half",
             block=256, sliced=False),
        # a plain decode step of a busy server
        dict(step, name="step_256x1", R=256, K=1, D=5120),
        # a speculative step: three drafts after each request's last token, every state kept
        dict(step, name="step_spec_256x4", R=256, K=4, D=5120),
        # the convolution of the same two steps
        {"op": "conv", "name": "conv_256x1", "dtype": "bf16", "R": 256, "K": 1, "D": 5120, "W": 4, "bias": True},
        {"op": "conv", "name": "conv_spec_256x4", "dtype": "bf16", "R": 256, "K": 4, "D": 5120, "W": 4, "bias": True},
        # one user's speculative step: latency
        {"op": "verify", "name": "verify_1x8", "dtype": "fp32", "R": 1, "K": 8, "V": 131072, "draft": True, "topk": 0},
        # a busy server's, the whole vocabulary kept
        {"op": "verify", "name": "verify_256x4", "dtype": "fp32", "R": 256, "K": 4, "V": 131072, "draft": True,
         "topk": 0},
        # ragged windows of n-gram drafts (no draft probabilities) after top-k, an odd vocabulary, bf16
        {"op": "verify", "name": "verify_ngram_64_odd", "dtype": "bf16", "R": 64, "K": 6, "V": 32003, "draft": False,
         "topk": 50},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "step", "conv", "verify"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "verify":
        c = {"op": op, "dtype": rng.choice(["fp32", "fp32", "bf16"]), "R": _log(rng, 1, 512), "K": rng.randint(1, 9),
             "V": _log(rng, 1000, 262144), "draft": rng.random() < 0.75, "topk": rng.choice([0, 0, 50])}
        c["R"] = max(1, min(c["R"], 150_000_000 // (c["K"] * c["V"])))
        return c
    D = _log(rng, 16, 8192)
    if op == "conv":
        return {"op": op, "dtype": dtype, "R": _log(rng, 1, 512), "K": rng.randint(1, 8), "D": D, "W": rng.randint(2, 4),
                "bias": rng.random() < 0.7}
    G = rng.choice([1, 1, 1, 2, 4])
    c = {"op": op, "dtype": dtype, "D": D // G * G, "N": rng.choice([16, 16, 16, _log(rng, 1, 64)]), "G": G,
         "z": rng.random() < 0.7, "skip": rng.random() < 0.8, "softplus": rng.random() < 0.8,
         "sliced": rng.random() < 0.5}
    if op == "step":
        return dict(c, R=max(1, min(_log(rng, 1, 512), 40_000_000 // (D * c["N"]))), K=rng.randint(1, 8))
    R, L = _log(rng, 1, 64), _log(rng, 1, 8192)
    L = max(1, min(L, 130_000_000 // (R * D), 4_000_000_000 // (R * D * c["N"])))
    return dict(c, R=R, kind=rng.choice(["same", "spread"]), L=L, init=rng.choice(["none", "half", "all"]),
                block=rng.choice([0, 0, 128, 1024]))


def _lengths(c):
    """The case's prompt or window lengths: fixed by the case, the same for every seed."""
    r = random.Random(str(sorted((k, v) for k, v in c.items() if k != "name")))
    if c["op"] in ("step", "conv", "verify"):
        K = c["K"]
        if c["op"] != "verify" or K == 1 or c["draft"]:
            return [K] * c["R"]
        return [r.randint(1, K) for _ in range(c["R"])]
    if c["kind"] == "given":
        return [int(x) for x in c["lens"].split(",")]
    if c["kind"] == "same":
        return [c["L"]] * c["R"]
    if c["kind"] == "spread":
        return [r.randint(1, c["L"]) for _ in range(c["R"])]
    raw = [min(4096.0, max(1.0, math.exp(r.gauss(math.log(400.0), 1.0)))) for _ in range(c["R"])]  # lognormal
    lens = [max(1, int(x * c["T"] / sum(raw))) for x in raw]
    lens[max(range(len(lens)), key=lens.__getitem__)] += c["T"] - sum(lens)
    return lens


def _computed(c, lens):
    """Tokens already in each prompt's state (multiples of nothing in particular), and whether it starts from a slot."""
    start = [{"none": False, "all": True, "half": i % 2 == 0, "last": i == len(lens) - 1}[c["init"]]
             for i in range(len(lens))]
    return [(37 * (i + 1)) % 901 if s else 0 for i, s in enumerate(start)], start


# --------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"scan": _prepare_scan, "step": _prepare_step, "conv": _prepare_conv, "verify": _prepare_verify}[case["op"]](
        case, g)
    s["case"] = case
    if own:  # the call's handle: argument structs, output buffers and workspace
        import mamba2_ssd_varlen_gb300 as m
        s["call"] = {"scan": m.SelectiveScanCall, "step": m.SelectiveStepCall, "conv": m.ConvStepCall,
                     "verify": m.VerifyCall}[case["op"]](s["prob"])
    return s


def _randn(g, *shape, scale=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale + mean).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _selective_inputs(c, T, g):
    """u (the convolution's output), delta, B, C and z of one layer, and its weights: A near -(1..N), the bias such
    that softplus gives steps from 1e-3 to 1e-1, as such layers are initialised."""
    D, N, G, dt = c["D"], c["N"], c["G"], _DT[c["dtype"]]
    u = torch.nn.functional.silu(_randn(g, T, D)).to(dt)
    step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    if c["softplus"]:
        delta, bias = _randn(g, T, D, scale=0.5, dtype=dt), torch.log(torch.expm1(step))
    else:
        delta, bias = (step * torch.exp(_randn(g, T, D, scale=0.5))).to(dt), None
    if c["sliced"]:  # views of the two projections' outputs, as a layer has them
        low = (-(-D // 32) + 7) // 8 * 8
        dbc = _randn(g, T, low + 2 * G * N, dtype=dt)
        B, C = dbc[:, low:low + G * N].unflatten(1, (G, N)), dbc[:, low + G * N:].unflatten(1, (G, N))
        z = _randn(g, T, 2 * D, dtype=dt)[:, D:] if c["z"] else None
    else:
        B, C = _randn(g, T, G, N, dtype=dt), _randn(g, T, G, N, dtype=dt)
        z = _randn(g, T, D, dtype=dt) if c["z"] else None
    A = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(_randn(g, D, N, scale=0.1))
    return {"u": u, "delta": delta, "A": A.contiguous(), "B": B, "C": C, "z": z, "delta_bias": bias,
            "D": _randn(g, D, scale=0.1, mean=1.0) if c["skip"] else None, "softplus": c["softplus"]}


def _prepare_scan(c, g):
    lens = _lengths(c)
    cu = _cu(lens)
    R, D, N, bs = len(lens), c["D"], c["N"], c["block"]
    done, start = _computed(c, lens)
    p = _selective_inputs(c, cu[-1], g)
    p["cu_seqlens"], p["num_computed"] = _i32(cu), _i32(done)
    p["block_size"], p["block_table"], p["state_pool"], p["init_slots"] = bs, None, None, None
    slots = sum(start)
    blocks = [(i, kb) for i in range(R) for kb in range(1, (done[i] + lens[i]) // max(bs, 1) + 1)
              if bs and kb * bs > done[i]]
    if slots or blocks:
        p["state_pool"] = _randn(g, slots + len(blocks), D, N, scale=0.5)
    if slots:
        order = iter(torch.randperm(slots, generator=torch.Generator().manual_seed(1)).tolist())
        p["init_slots"] = _i32([next(order) if s else -1 for s in start])
    if blocks:
        table = [[-1] * max(kb for _, kb in blocks) for _ in range(R)]
        for k, (i, kb) in enumerate(blocks):
            table[i][kb - 1] = slots + k
        p["block_table"] = _i32(table)
    else:
        p["block_size"] = 0
    # the plain form's plan: chunks cut at absolute multiples of _CHUNK, a row of token indices for each
    rows, chunks, ends, kept = [], [[] for _ in range(R)], [], []
    for i in range(R):
        t, e = cu[i], cu[i + 1]
        while t < e:
            n = min(e - t, _CHUNK - (done[i] + t - cu[i]) % _CHUNK)
            chunks[i].append(len(rows))
            rows.append((t, n))
            t += n
            pos = done[i] + t - cu[i]
            if blocks and pos % bs == 0:
                kept.append((table[i][pos // bs - 1], len(rows) - 1))
    nch = len(rows)
    idx = torch.full((nch, _CHUNK), cu[-1], dtype=torch.int64)  # the row after the last holds zeros
    ar = torch.arange(_CHUNK)
    first, count = torch.tensor([r[0] for r in rows])[:, None], torch.tensor([r[1] for r in rows])[:, None]
    idx = torch.where(ar < count, first + ar, idx)
    flat = torch.empty(cu[-1] + 1, dtype=torch.int64)
    flat[idx.reshape(-1)] = torch.arange(nch * _CHUNK)
    depth = max(len(x) for x in chunks)
    chain = torch.tensor([x + [nch] * (depth - len(x)) for x in chunks]).T.contiguous()
    plan = {"idx": idx.cuda(), "flat": flat[:-1].cuda(), "chain": chain.cuda(), "kept": None}
    if kept:
        plan["kept"] = (torch.tensor([k[0] for k in kept]).cuda(), torch.tensor([k[1] for k in kept]).cuda())
    return {"prob": p, "plan": plan}


def _window_slots(g, R, T):
    """Read slots for R requests and write slots for T tokens of one pool, in no order."""
    perm = torch.randperm(R + T, generator=g, device="cuda").to(torch.int32)
    return perm[:R].contiguous(), perm[R:].contiguous()


def _prepare_step(c, g):
    R, K = c["R"], c["K"]
    p = _selective_inputs(c, R * K, g)
    p["cu_seqlens"] = _i32(_cu([K] * R))
    p["state_pool"] = _randn(g, R + R * K, c["D"], c["N"], scale=0.5)
    p["read_slots"], p["write_slots"] = _window_slots(g, R, R * K)
    return {"prob": p}


def _prepare_conv(c, g):
    R, K, D, W, dt = c["R"], c["K"], c["D"], c["W"], _DT[c["dtype"]]
    reads, writes = _window_slots(g, R, R * K)
    return {"prob": {"x": _randn(g, R * K, D, dtype=dt), "weight": _randn(g, D, W, scale=W ** -0.5),
                     "bias": _randn(g, D, scale=0.1) if c["bias"] else None, "silu": True,
                     "cu_seqlens": _i32(_cu([K] * R)), "conv_pool": _randn(g, R + R * K, D, W - 1, dtype=dt),
                     "read_slots": reads, "write_slots": writes}}


def _prepare_verify(c, g):
    lens, V, dt = _lengths(c), c["V"], _DT[c["dtype"]]
    cu, R = _cu(lens), len(lens)
    T = cu[-1]
    target, draft, tokens = torch.empty(T, V, dtype=dt, device="cuda"), None, torch.empty(T, dtype=torch.int32,
                                                                                          device="cuda")
    if c["draft"]:
        draft = torch.empty(T, V, dtype=dt, device="cuda")
    for a in range(0, T, 64):  # peaked distributions; the draft model's are near the target's
        b = min(T, a + 64)
        x = _randn(g, b - a, V, scale=3.0)
        pt = torch.softmax(x, -1)
        if c["topk"]:
            pt = torch.where(pt >= pt.topk(min(c["topk"], V), -1).values[:, -1:], pt, 0.0)
            pt /= pt.sum(-1, keepdim=True)
        target[a:b] = pt.to(dt)
        pd = torch.softmax(x + _randn(g, b - a, V, scale=0.5), -1) if c["draft"] else torch.softmax(x * 1.5, -1)
        if c["draft"]:
            draft[a:b] = pd.to(dt)
        tokens[a:b] = torch.multinomial(pd, 1, generator=g).reshape(-1).to(torch.int32)
    tokens = torch.roll(tokens, 1)  # row t's distribution is the one that token t + 1 was drafted from
    u = torch.rand(T, generator=g, device="cuda")
    return {"prob": {"target": target, "draft": draft, "tokens": tokens, "accept_u": u,
                     "sample_u": torch.rand(R, generator=g, device="cuda"), "cu_seqlens": _i32(cu),
                     "write_slots": torch.randperm(T, generator=g, device="cuda").to(torch.int32)},
            "K": max(lens)}


# ------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"scan": _scan, "step": _step, "conv": _conv, "verify": _verify}[op](s)
    call = s["call"]()
    if op == "scan":
        return _scan_outputs(s["prob"], call.y, call.final_states)
    if op == "step":
        return {"y": call.y, "pool": s["prob"]["state_pool"]}
    if op == "conv":
        return {"y": call.y, "pool": s["prob"]["conv_pool"]}
    return {"accepted": call.accepted, "out_tokens": call.out_tokens, "next_slots": call.next_slots}


def _scan_outputs(p, y, final):
    out = {"y": y, "final_states": final}
    if p["block_table"] is not None:
        out["pool"] = p["state_pool"]
    return out


def _steps(p):
    """dt' = softplus(delta + bias) where the layer has it, fp32."""
    v = p["delta"].float()
    if p["delta_bias"] is not None:
        v = v + p["delta_bias"]
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v))) if p["softplus"] else v


def _finish(p, y):
    """+ D u, * silu(z), rounded once."""
    if p["D"] is not None:
        y = y + p["D"] * p["u"].float()
    if p["z"] is not None:
        z = p["z"].float()
        y = y * (z / (1.0 + torch.exp(-z)))
    return y.to(p["u"].dtype)


def _scan(s):
    """Chunks of _CHUNK tokens side by side, a token of each at a time: their states from zero, the states that enter
    them (chunk by chunk), then their outputs."""
    p, plan = s["prob"], s["plan"]
    idx, chain = plan["idx"], plan["chain"]
    nch, (D, N), G = idx.shape[0], p["A"].shape, p["B"].shape[1]
    R, E = p["cu_seqlens"].shape[0] - 1, D // G

    def cut(x):  # token rows of each chunk, zeros where it has none
        return torch.cat([x, x.new_zeros(1, *x.shape[1:])])[idx]

    dt = _steps(p)
    du = cut(dt * p["u"].float()).view(nch, _CHUNK, G, E)
    dt = cut(dt).view(nch, _CHUNK, G, E)
    B, C = cut(p["B"].float()), cut(p["C"].float())
    A = p["A"].view(G, E, N)

    def advance(h, j):
        return torch.exp(dt[:, j, :, :, None] * A).mul_(h).add_(du[:, j, :, :, None] * B[:, j, :, None, :])

    h = torch.zeros(nch, G, E, N, device="cuda")
    for j in range(_CHUNK):
        h = advance(h, j)
    total = dt.sum(1)
    zero = torch.zeros(1, G, E, N, device="cuda")
    local, total = torch.cat([h, zero]), torch.cat([total, zero[..., 0]])
    enter = torch.empty(nch + 1, G, E, N, device="cuda")
    if p["init_slots"] is None:
        state = torch.zeros(R, G, E, N, device="cuda")
    else:
        state = p["state_pool"][p["init_slots"].long()].view(R, G, E, N)
        state = torch.where(p["init_slots"].view(R, 1, 1, 1) >= 0, state, 0.0)
    for k in range(chain.shape[0]):
        c = chain[k]
        enter[c] = state
        state = torch.exp(total[c][..., None] * A).mul_(state).add_(local[c])
    h = enter[:nch]
    y = torch.empty(nch, _CHUNK, D, device="cuda")
    for j in range(_CHUNK):
        h = advance(h, j)
        y[:, j] = (h * C[:, j, :, None, :]).sum(-1).view(nch, D)
    if plan["kept"] is not None:  # a chunk's last state is the one after its last token: the rest of it adds nothing
        slots, chunk = plan["kept"]
        p["state_pool"][slots] = h[chunk].view(-1, D, N)
    return _scan_outputs(p, _finish(p, y.view(-1, D)[plan["flat"]]), state.view(R, D, N))


def _step(s):
    p = s["prob"]
    (D, N), G, R = p["A"].shape, p["B"].shape[1], p["read_slots"].shape[0]
    K, E, A = s["case"]["K"], D // G, p["A"].view(G, D // G, N)
    dt = _steps(p)
    du = (dt * p["u"].float()).view(R, K, G, E, 1)
    dt = dt.view(R, K, G, E, 1)
    B, C = p["B"].float().reshape(R, K, G, 1, N), p["C"].float().reshape(R, K, G, 1, N)
    pool, writes = p["state_pool"], p["write_slots"].long().view(R, K)
    h = pool[p["read_slots"].long()].view(R, G, E, N)
    y = torch.empty(R, K, D, device="cuda")
    for j in range(K):
        h = torch.exp(dt[:, j] * A) * h + du[:, j] * B[:, j]
        y[:, j] = (h * C[:, j]).sum(-1).view(R, D)
        pool[writes[:, j]] = h.view(R, D, N)
    return {"y": _finish(p, y.view(R * K, D)), "pool": pool}


def _conv(s):
    p, c = s["prob"], s["case"]
    R, K, D, W, pool = c["R"], c["K"], c["D"], c["W"], p["conv_pool"]
    seq = torch.cat([pool[p["read_slots"].long()], p["x"].view(R, K, D).transpose(1, 2)], 2)  # (R, D, W - 1 + K)
    win = seq.unfold(2, W, 1)  # (R, D, K, W): a token's own input is the last
    v = (win.float() * p["weight"][:, None, :]).sum(-1).transpose(1, 2).reshape(R * K, D)
    if p["bias"] is not None:
        v = v + p["bias"]
    pool[p["write_slots"].long()] = win[..., 1:].transpose(1, 2).reshape(R * K, D, W - 1)
    return {"y": (v / (1.0 + torch.exp(-v))).to(p["x"].dtype), "pool": pool}


def _verify(s):
    p = s["prob"]
    cu = p["cu_seqlens"].long()
    V, first, n = p["target"].shape[1], cu[:-1], cu[1:] - cu[:-1]
    j = torch.arange(1, s["K"], device="cuda")  # the drafts' places in their windows
    at = torch.minimum(first[:, None] + j, cu[1:, None] - 1)
    token, row = p["tokens"][at].long(), at - 1
    row = row.clamp_min(0)
    pt = p["target"][row, token].float()
    qt = p["draft"][row, token].float() if p["draft"] is not None else torch.ones_like(pt)
    good = (p["accept_u"][at] * qt < pt) & (j < n[:, None])
    accepted = torch.cumprod(good.long(), 1).sum(1)
    last = first + accepted  # the row that gives the token that follows
    full = p["target"][last].float()
    w, rejected = full, accepted < n - 1
    if p["draft"] is not None:
        w = torch.where(rejected[:, None], full - p["draft"][last].float(), full)
    else:
        t = p["tokens"][torch.minimum(last + 1, cu[1:] - 1)].long()
        hit = rejected[:, None] & (torch.arange(V, device="cuda") == t[:, None])
        w = torch.where(hit, 0.0, full)

    def fixed(w):  # whole multiples of 2^-40: sums of these have no order
        return torch.floor(torch.where(w > 0, w, 0.0).clamp_max(1.0) * 2.0 ** 40).long()

    f = fixed(w)
    f = torch.where((f.sum(1) == 0)[:, None], fixed(full), f)
    run = torch.cumsum(f, 1)
    total = run[:, -1]
    mark = torch.minimum((p["sample_u"].double() * total.double()).floor().long(), total - 1)
    pick = torch.where(total > 0, (run <= mark[:, None]).sum(1), -1)
    t = torch.arange(p["tokens"].shape[0], device="cuda")
    i = torch.searchsorted(cu, t, right=True) - 1
    place = t - cu[i]
    nxt = torch.cat([p["tokens"][1:], p["tokens"][:1]]).long()
    out = torch.where(place < accepted[i], nxt, torch.where(place == accepted[i], pick[i], -1))
    return {"accepted": accepted.int(), "out_tokens": out.int(), "next_slots": p["write_slots"][last]}


# ----------------------------------------------------------------- what it comes to
def work(c):
    lens = _lengths(c)
    T, R, e = sum(lens), len(lens), 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "verify":
        # of each window: a row of the target's, of the draft's too where one is rejected (about half are); and the drafts' entries
        rows = R * (1.5 if c["draft"] and c["K"] > 1 else 1.0)
        return {"bytes": rows * c["V"] * e + T * 64 + R * 16, "flops": rows * c["V"] * 4}
    D = c["D"]
    if c["op"] == "conv":
        W = c["W"]
        return {"bytes": T * D * e * 2 + (R + T) * D * (W - 1) * e + D * (W + 1) * 4 + (R + T) * 4,
                "flops": T * D * (2 * W + 4)}
    N, G = c["N"], c["G"]
    tokens = T * e * (D * (3 + bool(c["z"])) + 2 * G * N) + D * (N + 2) * 4
    flops = T * D * (7 * N + 8)
    if c["op"] == "step":
        return {"bytes": tokens + (R + T) * (D * N * 4 + 4), "flops": flops}
    done, start = _computed(c, lens)
    kept = sum((d + n) // c["block"] - d // c["block"] for d, n in zip(done, lens)) if c["block"] else 0
    return {"bytes": tokens + (R + sum(start) + kept) * D * N * 4, "flops": flops}


# ------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The definition, token by token in fp64; nothing for verify, whose results are whole numbers."""
    if case["op"] == "verify":
        return None
    held = prepare(dict(case), seed)["prob"]
    p = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() and k not in ("state_pool", "conv_pool") else v
         for k, v in held.items()}
    if case["op"] == "conv":
        return _exact_conv(case, p)
    lens = _lengths(case)
    cu, R, (D, N) = _cu(lens), len(lens), p["A"].shape
    pool = p["state_pool"].double() if p["state_pool"] is not None else None
    slots = p["read_slots"] if case["op"] == "step" else p["init_slots"]
    h = torch.zeros(R, D, N, dtype=torch.float64, device="cuda")
    if slots is not None:
        for i, k in enumerate(slots.tolist()):
            if k >= 0:
                h[i] = pool[k]
    step = p["delta"] if p["delta_bias"] is None else p["delta"] + p["delta_bias"]
    if case["softplus"]:
        step = torch.logaddexp(step, torch.zeros_like(step))
    done = _computed(case, lens)[0] if case["op"] == "scan" else None
    writes = p["write_slots"].tolist() if case["op"] == "step" else None
    table = p["block_table"].tolist() if case["op"] == "scan" and p["block_table"] is not None else None
    order = sorted(range(R), key=lambda i: -lens[i])  # requests that still have a token come first
    h = h[order]
    y = torch.empty(cu[-1], D, dtype=torch.float64, device="cuda")
    starts, alive = torch.tensor([cu[i] for i in order], device="cuda"), R
    rep = D // p["B"].shape[1]
    for j in range(max(lens)):
        while lens[order[alive - 1]] <= j:
            alive -= 1
        t = starts[:alive] + j
        d, b, c = step[t], p["B"][t].repeat_interleave(rep, 1), p["C"][t].repeat_interleave(rep, 1)
        now = h[:alive]
        now.mul_(torch.exp(d[..., None] * p["A"])).addcmul_((d * p["u"][t])[..., None], b)
        y[t] = torch.einsum("rdn,rdn->rd", now, c)
        if writes is not None:
            for k in range(alive):
                pool[writes[cu[order[k]] + j]] = h[k]
        if table is not None:
            for k in range(alive):
                pos = done[order[k]] + j + 1
                if pos % case["block"] == 0:
                    pool[table[order[k]][pos // case["block"] - 1]] = h[k]
    if p["D"] is not None:
        y += p["D"] * p["u"]
    if p["z"] is not None:
        y *= p["z"] * torch.sigmoid(p["z"])
    if case["op"] == "step":
        return {"y": y, "pool": pool}
    final = torch.empty_like(h)
    final[order] = h
    return _scan_outputs(dict(p, state_pool=pool), y, final)


def _exact_conv(case, p):
    R, K, W, pool = case["R"], case["K"], case["W"], p["conv_pool"].double()
    y, reads, writes = torch.empty_like(p["x"]), p["read_slots"].tolist(), p["write_slots"].tolist()
    for i in range(R):
        held = pool[reads[i]].clone()
        for t in range(i * K, i * K + K):
            held = torch.cat([held, p["x"][t][:, None]], 1)
            v = (held * p["weight"]).sum(1) + (p["bias"] if p["bias"] is not None else 0.0)
            y[t] = v * torch.sigmoid(v)
            held = held[:, 1:]
            pool[writes[t]] = held
    return {"y": y, "pool": pool}
