"""Speculative decoding of a small selective-state-space (S6) language model, all of it on the library's
entry points: prompts through ssd_varlen_conv1d and ssd_varlen_selective_scan, then steps of drafted
windows through ssd_varlen_conv1d_step, ssd_varlen_selective_step and ssd_varlen_verify.

Every window token's state goes to a slot of its own, so a rejected draft costs nothing: the verification
hands out the slot of the last accepted token, which is the next step's read anchor, on the device.  A
request owns two sets of k + 1 slots and the steps write them in turn (a step never writes what it reads).

    python examples/speculative_s6.py            # on a GPU
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba2_ssd_varlen_gb300 as m  # noqa: E402


class S6Model:
    """Embedding, `layers` S6 blocks, head; random weights.  Its pools hold `slots` states a layer."""

    def __init__(self, vocab, width, layers, slots, dtype=torch.float32, N=16, W=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s, scale=1.0: torch.randn(s, generator=g, device=device) * scale  # noqa: E731
        D, rank = 2 * width, max(8, width // 16 // 8 * 8)
        self.N, self.D, self.rank, self.dtype, self.layers = N, D, rank, dtype, []
        self.embed = randn(vocab, width, scale=width ** -0.5).to(dtype)
        self.head = randn(width, vocab, scale=width ** -0.5).to(dtype)
        for _ in range(layers):
            self.layers.append({
                "in": randn(width, 2 * D, scale=width ** -0.5).to(dtype),
                "conv": randn(D, W, scale=W ** -0.5), "conv_bias": randn(D, scale=0.1),
                "x": randn(D, rank + 2 * N, scale=D ** -0.5).to(dtype),
                "dt": randn(rank, D, scale=rank ** -0.5).to(dtype),
                "dt_bias": torch.log(torch.expm1(torch.logspace(-3, -1, D, device=device))),
                "A": -torch.arange(1, N + 1, device=device, dtype=torch.float32).repeat(D, 1),
                "D": torch.ones(D, device=device), "out": randn(D, width, scale=D ** -0.5).to(dtype),
                "state": torch.zeros(slots, D, N, device=device),
                "conv_state": torch.zeros(slots, D, W - 1, dtype=dtype, device=device)})

    def __call__(self, tokens, cu, read, write, window):
        """Logits (T, V) of packed tokens.  window: slots in `write` are per token, else per request."""
        h = self.embed[tokens.long()]
        for p in self.layers:
            x, z = (torch.nn.functional.normalize(h.float(), dim=-1).to(self.dtype) @ p["in"]).chunk(2, -1)
            conv = {"x": x.contiguous(), "weight": p["conv"], "bias": p["conv_bias"], "silu": True, "cu_seqlens": cu,
                    "conv_pool": p["conv_state"], "read_slots": read, "write_slots": write}
            u = (m.run_conv1d_step if window else m.run_conv1d)(conv).y
            low = u @ p["x"]
            delta, B, C = low[:, :self.rank] @ p["dt"], low[:, None, self.rank:self.rank + self.N], \
                low[:, None, self.rank + self.N:]
            s = {"u": u, "delta": delta, "A": p["A"], "B": B, "C": C, "D": p["D"], "z": z, "softplus": True,
                 "delta_bias": p["dt_bias"], "state_pool": p["state"], "cu_seqlens": cu}
            if window:
                y = m.run_selective_step(dict(s, read_slots=read, write_slots=write)).y
            else:
                y = m.run_selective_scan(dict(s, init_slots=read, final_slots=write, final_dense=False)).y
            h = h + y @ p["out"]
        return (h @ self.head).float()


def _cu(lens, dev):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=dev)


def _probabilities(logits, temperature):
    """Softmax at a temperature; one-hot at temperature 0."""
    if temperature:
        return torch.softmax(logits / temperature, -1)
    return torch.nn.functional.one_hot(logits.argmax(-1), logits.shape[-1]).float()


def generate(target, draft, prompts, new_tokens, k, temperature=0.0, seed=0):
    """`new_tokens` tokens (at least) after each prompt, with k drafts a step (k = 0: one token a step, no draft
    model).  Returns the generated lists and the mean number of tokens a step."""
    dev, R = target.embed.device, len(prompts)
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=g, device=dev)  # noqa: E731
    pick = lambda p: torch.multinomial(p, 1, generator=g).reshape(-1).int()  # noqa: E731
    slot = torch.arange(2 * R * (k + 1), dtype=torch.int32, device=dev).view(2, R, k + 1)
    packed = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=dev)
    cu = _cu([len(p) for p in prompts], dev)
    none = torch.full((R,), -1, dtype=torch.int32, device=dev)
    read = slot[1, :, 0].contiguous()  # where the prompts' states go
    logits = target(packed, cu, none, read, False)[cu[1:].long() - 1]
    if k:
        draft(packed, cu, none, read, False)
    last = pick(_probabilities(logits, temperature))
    out, steps, made = [[int(t)] for t in last.tolist()], 0, 0
    one, window = _cu([1] * R, dev), _cu([k + 1] * R, dev)
    while min(len(o) for o in out) < new_tokens:
        write = slot[steps % 2]
        tokens, q = [last], []
        for j in range(k + 1 if k else 0):  # the last call only advances the draft model's state
            at = read if j == 0 else write[:, j - 1].contiguous()
            pj = _probabilities(draft(tokens[j], one, at, write[:, j].contiguous(), True), temperature)
            q.append(pj)
            if j < k:
                tokens.append(pick(pj))
        flat = torch.stack(tokens, 1).reshape(-1).contiguous()
        writes = write.reshape(-1).contiguous()
        p = _probabilities(target(flat, window, read, writes, True), temperature)
        call = m.run_verify({"target": p, "draft": torch.stack(q, 1).flatten(0, 1) if k else None, "tokens": flat,
                             "cu_seqlens": window, "accept_u": rand(R * (k + 1)), "sample_u": rand(R),
                             "write_slots": writes, "next_slots": read.clone()})
        read = call.next_slots
        new = call.out_tokens.view(R, k + 1)
        last = new.gather(1, call.accepted.long()[:, None]).reshape(-1)
        for o, row in zip(out, new.tolist()):
            o += [t for t in row if t >= 0]
        steps += 1
        made += int((new >= 0).sum())
    return out, made / max(steps, 1) / R


def main(vocab=512, width=256, layers=2, requests=4, prompt=50, new_tokens=40, k=3):
    m.load_library()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(vocab, (prompt + 7 * i,), generator=g).tolist() for i in range(requests)]
    model = lambda seed: S6Model(vocab, width, layers, 2 * requests * (k + 1), seed=seed)  # noqa: E731
    plain, _ = generate(model(0), None, prompts, new_tokens, 0)
    good, rate = generate(model(0), model(0), prompts, new_tokens, k)
    poor, low = generate(model(0), model(5), prompts, new_tokens, k)
    same = all(a[:new_tokens] == b[:new_tokens] == c[:new_tokens] for a, b, c in zip(plain, good, poor))
    print(f"greedy decoding of {requests} requests, {k} drafts a step: {rate:.2f} tokens a step with a draft model "
          f"that agrees, {low:.2f} with one that does not; the same tokens as without drafts: {same}")
    return same, rate, low


if __name__ == "__main__":
    main()
