"""A gated delta rule layer served: ragged prompts through the chunked path, then decoding steps on
cached states and windows, checked against the whole sequences through the chunked path.

    python examples/serve.py                # (16, 48) heads, 128 wide, 4 prompts, 64 decoding steps
    python examples/serve.py --steps 16 --graph

A prompt runs conv front-end -> q/k norms + rotation -> chunked rule; its last state and its last
W - 1 inputs go into the caches. A decoding step runs the same three on one token of every sequence:
gdn_conv_step -> gdn_qk_rope_fwd -> gdn_recurrent, with --graph captured once and replayed.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_fwd_amd as G  # noqa: E402


class Layer:
    """Weights of one layer's front-end (conv taps, q/k norm weights, rotation) and its sizes."""

    def __init__(self, h_qk=16, h_v=48, d=128, width=4, rotary=64, device="cuda:0", seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.h_qk, self.h_v, self.d, self.width, self.rotary, self.device = h_qk, h_v, d, width, rotary, device
        self.groups = [h_qk * d, h_qk * d, h_v * d]
        c = sum(self.groups)
        self.taps = torch.randn(c, width, generator=gen, device=device) / width ** 0.5
        self.bias = 0.1 * torch.randn(c, generator=gen, device=device)
        self.w_q = 1 + 0.1 * torch.randn(d, generator=gen, device=device)
        self.w_k = 1 + 0.1 * torch.randn(d, generator=gen, device=device)
        freqs, self.magnitude = G.gdn_rope_frequencies(rotary)
        self.freqs = freqs.to(device)

    def rope(self, tokens):
        return G.QkRopeProblem(tokens, self.h_qk, self.h_qk, self.d, rotary_dim=self.rotary, magnitude=self.magnitude)

    def turn(self, problem, q, k, positions):
        heads = lambda x: x.view(-1, self.h_qk, self.d)  # noqa: E731
        q, k = heads(q), heads(k)
        return G.gdn_qk_rope_fwd(problem, q, k, positions, self.freqs, q_weight=self.w_q, k_weight=self.w_k, q_out=q,
                                 k_out=k)

    def prompts(self, lengths, x, g, beta):
        """Packed prompts through the chunked path: (o [T, h_v, d], last states [N, h_v, d, d])."""
        cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        on_gpu = torch.from_numpy(cu).to(self.device)
        positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths]).to(self.device)
        q, k, v = G.gdn_conv_fwd(G.ConvProblem(cu, self.groups, width=self.width), x, self.taps, self.bias, on_gpu)
        q, k = self.turn(self.rope(int(cu[-1])), q, k, positions)
        p = G.Problem(cu, self.h_qk, self.h_v, self.d, want_ht=True)
        o, ht, _ = G.gdn_fwd(p, q, k, v.view(-1, self.h_v, self.d), g, beta, on_gpu)
        return o, ht


class Cache:
    """States and conv windows of the sequences being served, and the plans of a decoding step."""

    def __init__(self, layer, slots, batch):
        self.layer, dev = layer, layer.device
        self.states = torch.zeros(slots, layer.h_v, layer.d, layer.d, device=dev)
        self.windows = torch.zeros(slots, layer.width - 1, sum(layer.groups), dtype=torch.bfloat16, device=dev)
        self.conv = G.ConvStepProblem(batch, layer.groups, slots, width=layer.width)
        self.rope = layer.rope(batch)
        self.rule = G.RecurrentProblem(batch, layer.h_qk, layer.h_v, layer.d, slots)

    def admit(self, slots, lengths, x, last_states):
        """Keeps the prompts' last states and their last W - 1 inputs (zeros before a short prompt)."""
        self.states[slots.long()] = last_states
        past = self.layer.width - 1
        end = 0
        for slot, n in zip(slots.tolist(), lengths):
            end += n
            rows = min(n, past)
            self.windows[slot] = 0
            self.windows[slot, past - rows:] = x[end - rows:end]

    def step(self, slots, x, g, beta, positions):
        """One token of every sequence: o [batch, h_v, d]; states and windows move on in place."""
        layer = self.layer
        q, k, v = G.gdn_conv_step(self.conv, x, layer.taps, layer.bias, self.windows, slots, slots)
        q, k = layer.turn(self.rope, q, k, positions)
        return G.gdn_recurrent(self.rule, q, k, v.view(-1, layer.h_v, layer.d), g, beta, self.states, slots, slots)


def serve(lengths=(1000, 1, 130, 2), steps=64, h_qk=16, h_v=48, d=128, rotary=64, graph=False, seed=1):
    """Relative error of the decoded outputs and of the last states against the whole sequences."""
    layer = Layer(h_qk, h_v, d, rotary=rotary)
    dev, batch, c = layer.device, len(lengths), sum(layer.groups)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    # every sequence's stream, prompt and decoded tokens: inputs of the conv, log decays, write strengths
    x = [normal(n + steps, c).bfloat16() for n in lengths]
    g = [torch.nn.functional.logsigmoid(normal(n + steps, h_v) + 3) for n in lengths]
    beta = [torch.sigmoid(normal(n + steps, h_v)) for n in lengths]
    first = lambda xs: torch.cat([t[:n] for t, n in zip(xs, lengths)])  # noqa: E731
    at = lambda xs, i: torch.stack([t[n + i] for t, n in zip(xs, lengths)])  # noqa: E731

    cache = Cache(layer, slots=batch + 2, batch=batch)
    slots = torch.randperm(batch + 2, generator=gen, device=dev)[:batch].to(torch.int32)
    _, last = layer.prompts(lengths, first(x), first(g), first(beta))
    cache.admit(slots, lengths, first(x), last)

    now = [at(x, 0), at(g, 0), at(beta, 0), torch.tensor(lengths, dtype=torch.int32, device=dev)]
    replay = None
    if graph:
        kept = cache.states.clone(), cache.windows.clone()
        cache.step(slots, *now)  # once before the capture, then back to the prompts' end
        torch.cuda.synchronize()
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay):
            out = cache.step(slots, *now)
        cache.states.copy_(kept[0])
        cache.windows.copy_(kept[1])
    decoded = []
    for i in range(steps):
        for buf, new in zip(now, (at(x, i), at(g, i), at(beta, i))):
            buf.copy_(new)
        now[3].copy_(torch.tensor([n + i for n in lengths], dtype=torch.int32))
        if graph:
            replay.replay()
            decoded.append(out.clone())
        else:
            decoded.append(cache.step(slots, *now))

    whole, ht = layer.prompts([n + steps for n in lengths], torch.cat(x), torch.cat(g), torch.cat(beta))
    want, end = [], 0
    for n in lengths:
        end += n + steps
        want.append(whole[end - steps:end])
    off = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())  # noqa: E731
    return off(torch.stack(decoded, 1), torch.stack(want)), off(cache.states[slots.long()], ht)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--graph", action="store_true", help="capture the decoding step and replay it")
    a = ap.parse_args()
    o, s = serve(steps=a.steps, graph=a.graph)
    print("%d decoding steps after ragged prompts: outputs off by %.2e, states by %.2e (2-norm, chunked path)" % (
        a.steps, o, s))
