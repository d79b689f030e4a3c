"""GPU test of the serving operators as they are used together, on caches cut into blocks: a step's maps, RMS norm
with the residual, projections, rotation of q and k, linear attention (prompts chunked, then a few tokens a step on
the cached states), norm in 8 bits. Every operator is held to the 64-bit formula on what it read, and the states and
outputs to the whole sequences' from the tokens that the steps saw; steps run eagerly or as one replayed graph."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
from oracle import linear_oracle as lo
from oracle import rope_oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-6
BF16, E4M3 = 2.0 ** -8, 2.0 ** -4  # half a step
C, H, HV, D, BLOCK, WIDTH, ROTARY = 256, 2, 4, 64, 8, 8, 32


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Layer:
    def __init__(self, gen):
        normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
        self.w_norm = 1 + 0.1 * normal(C)
        self.proj = (normal(C, (2 * H + HV) * D) / C ** 0.5).bfloat16()
        self.gate = (normal(C, HV) / C ** 0.5).bfloat16()
        self.w_out = 1 + 0.1 * normal(HV * D)
        self.freqs, self.magnitude = G.gdn_rope_frequencies(ROTARY)
        self.freqs = self.freqs.to(DEV)

    def rows(self, room):
        return (G.RmsNormProblem(room, C, eps=EPS), G.RmsNormProblem(room, HV * D, out="e4m3", group=64, eps=EPS),
                G.QkRopeProblem(room, H, H, D, rotary_dim=ROTARY, magnitude=self.magnitude))

    def front(self, plans, x, residual, positions):
        y, _, total = G.gdn_rms_norm_fwd(plans[0], x, weight=self.w_norm, residual=residual)
        row = y @ self.proj
        q, k = (row[:, i * H * D:(i + 1) * H * D].contiguous().view(-1, H, D) for i in (0, 1))
        v = row[:, 2 * H * D:].view(-1, HV, D)
        g = torch.nn.functional.logsigmoid((y @ self.gate).float() + 2)
        q1, k1 = G.gdn_qk_rope_fwd(plans[2], q, k, positions, self.freqs)
        return dict(x=x, residual=residual, y=y, total=total, q=q, k=k, q1=q1, k1=k1, v=v, g=g)

    def back(self, plans, r, o):
        r["o"] = o
        r["y8"], r["scales"], _ = G.gdn_rms_norm_fwd(plans[1], o.view(-1, HV * D), weight=self.w_out)
        return r


class Server:
    """Three requests' tables, contexts and block states, and room for a fourth."""

    def __init__(self, seed):
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.layer, self.N = Layer(self.gen), 4
        self.table = torch.full((self.N, WIDTH), -1, dtype=torch.int32, device=DEV)
        self.n_blocks = self.N * WIDTH + 3
        self.free = torch.randperm(self.n_blocks, generator=self.gen, device=DEV).to(torch.int32)
        self.count, self.contexts, self.lengths = i32([self.n_blocks]), i32([0] * self.N), i32([0] * self.N)
        self.states = torch.full((self.n_blocks, HV, D, D), float("nan"), device=DEV)
        self.seen = [[] for _ in range(self.N)]

    def maps(self, room):
        p = G.StepMapsProblem(self.N, room, BLOCK, WIDTH, self.n_blocks)
        return G.gdn_step_maps(p, self.lengths, self.contexts, self.table, self.free, self.count)

    def hidden(self, room):
        return [torch.randn(room, C, generator=self.gen, device=DEV).bfloat16() for _ in range(2)]

    def prompt(self, lengths):
        """All requests from nothing, chunked; the last states go to the requests' last blocks."""
        self.lengths.copy_(i32(lengths))
        room, cu = sum(lengths), np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        m = self.maps(room)
        assert m["cu_seqlens"].tolist() == cu.tolist() and m["slot_in"].tolist() == [-1] * self.N
        plans = self.layer.rows(room)
        r = self.layer.front(plans, *self.hidden(room), m["positions"])
        p = G.LinearProblem(cu, H, HV, D, scale=D ** -0.5, want_ht=True)
        o, ht = G.gdn_linear_fwd(p, r["q1"], r["k1"], r["v"], r["g"], m["cu_seqlens"])
        used = m["slot_out"] >= 0
        self.states[m["slot_out"][used].long()] = ht[used]
        self.note(m, self.layer.back(plans, r, o), chunked=True)

    def plan(self, room, most):
        host = np.minimum(np.arange(self.N + 1) * most, room)
        return self.layer.rows(room), G.LinearStepProblem(self.N, H, HV, D, self.n_blocks, cu_seqlens_host=host,
                                                          scale=D ** -0.5)

    def step(self, plan, x, residual):
        """Some tokens of every request, as lengths says: reads only what is on the GPU, so that it can be captured."""
        plans, rule = plan
        m = self.maps(x.shape[0])
        r = self.layer.front(plans, x, residual, m["positions"])
        o = torch.zeros(x.shape[0], HV, D, dtype=torch.bfloat16, device=DEV)
        G.gdn_linear_step(rule, r["q1"], r["k1"], r["v"], r["g"], self.states, m["slot_in"], m["slot_out"],
                          slot_tok=m["slot_tok"], cu_seqlens=m["cu_seqlens"], o=o)
        return m, self.layer.back(plans, r, o)

    def note(self, m, r, chunked=False):
        cu, pos = m["cu_seqlens"].tolist(), m["positions"].tolist()
        rows = {name: f64(t.float()) for name, t in r.items()}
        for n in range(self.N):
            for t in range(cu[n], cu[n + 1]):
                assert pos[t] == len(self.seen[n])
                self.seen[n].append(dict({name: a[t] for name, a in rows.items()}, chunked=chunked))


def norm_rows(x, w):
    return w * x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)


def check(s):
    layer = s.layer
    w, w8, freqs = f64(layer.w_norm), f64(layer.w_out), rope_oracle.frequencies(ROTARY)[0]
    last = f64(s.states)
    for n, seen in enumerate(s.seen):
        if not seen:
            continue
        a = {name: np.stack([r[name] for r in seen]) for name in seen[0] if name != "chunked"}
        T = len(seen)
        # the sum and its norm: FP32 sums of 256 values, one rounding each
        total = a["x"] + a["residual"]
        assert (np.abs(a["total"] - total) <= 1.01 * BF16 * np.abs(total)).all()
        y = norm_rows(total, w)
        assert (np.abs(a["y"] - y) <= 1.01 * BF16 * np.abs(y)).all()
        # row norm and rotation at 0, 1, ..: an FP32 error goes by the row's largest value
        for name in "qk":
            x = a[name]
            want = rope_oracle.fwd(x, np.arange(T), freqs, rotary_dim=ROTARY, m=layer.magnitude)
            bound = 1.01 * BF16 * np.abs(want) + 2.0 ** -18 * np.abs(want).max(-1, keepdims=True)
            assert (np.abs(a[name + "1"] - want) <= bound).all()
        # the whole sequence; a chunk's decayed products and the state it meets are rounded once in chunked rows
        cu = np.array([0, T])
        o, ht = lo.fwd(cu, a["q1"], a["k1"], a["v"], a["g"], None, D ** -0.5)
        oA, htA = lo.fwd(cu, np.abs(a["q1"]), np.abs(a["k1"]), np.abs(a["v"]), a["g"], None, D ** -0.5)
        chunked = np.array([r["chunked"] for r in seen])[:, None, None]
        small = 2.0 ** -24 * (2 * T + 2 * D + 64)  # a rounding a token for the decays and sums, twice over
        assert (np.abs(a["o"] - o) <= 1.01 * BF16 * (np.abs(o) + chunked * oA) + small * oA).all()
        slot = int(s.table[n, (T - 1) // BLOCK])
        assert (np.abs(last[slot] - ht[0]) <= small * htA[0]).all()
        # its norm in 8 bits: half a step of the value, or of the smallest normal magnitude times the scale
        y = norm_rows(a["o"].reshape(T, HV * D), w8).reshape(T, HV, D)
        scale = np.abs(y).max(-1) / 448
        assert (np.abs(a["scales"] - scale) <= 2.0 ** -18 * scale).all()
        got = a["y8"].reshape(T, HV, D) * a["scales"][..., None]
        assert (np.abs(got - y) <= np.maximum(1.01 * E4M3 * np.abs(y), 1.01 * 2.0 ** -10 * scale[..., None])).all()


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_blocks_serve_a_layer(graph):
    s = Server(7)
    s.prompt([37, 0, 5, 0])
    room, most = 7, 3
    plan, (x, residual) = s.plan(room, most), s.hidden(room)
    if graph:
        kept = [t.clone() for t in (s.table, s.count, s.contexts, s.states)]
        s.lengths.copy_(i32([1, 1, 1, 0]))
        s.step(plan, x, residual)  # once before the capture, then back to the prompts' end
        torch.cuda.synchronize()
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay):
            out = s.step(plan, x, residual)
        for t, k in zip((s.table, s.count, s.contexts, s.states), kept):
            t.copy_(k)
    steps = [[1, 3, 1, 0], [1, 3, 1, 0], [3, 3, 1, 0], [0, 1, 0, 0], [1, 0, 2, 3], [2, 3, 2, 0], [1, 1, 1, 3], [0] * 4,
             [1, 2, 2, 1]]
    for i, lengths in enumerate(steps):
        if i == 4:  # a fourth request shares the second's first block: its tokens, and the state after them
            assert len(s.seen[1]) == 10
            s.table[3, 0] = s.table[1, 0]
            s.contexts[3] = BLOCK
            s.seen[3] = list(s.seen[1][:BLOCK])
        for buf, new in zip((x, residual), s.hidden(room)):
            buf.copy_(new)
        s.lengths.copy_(i32(lengths))
        if graph:
            replay.replay()
            m, r = out
        else:
            m, r = s.step(plan, x, residual)
        assert m["granted"].tolist() == lengths and m["cu_seqlens"].tolist()[-1] == sum(lengths)
        assert not f64(r["o"].float())[sum(lengths):].any()  # behind the last sequence: as it was
        s.note(m, r)
        torch.cuda.synchronize()
    assert s.contexts.tolist() == [len(x) for x in s.seen]
    owned = -(-torch.tensor([len(x) for x in s.seen]) // BLOCK)
    assert int(s.count) == s.n_blocks - int(owned.sum()) + 1  # one block has two owners
    check(s)
