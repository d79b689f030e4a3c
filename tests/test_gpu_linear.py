"""Linear attention with decays on MI355X against its FP64 reference: chunked forward and backward, recurrent step.

Bounds, elementwise. With A the sums of magnitudes (the reference on absolute values), an f32 result is off by at most
k roundings of 2^-24 of A, k = 600: products and sums over 128 values, 64 tokens and the chunks before, and the decays'
exponentials. A bf16 result adds its own rounding, 2^-8 of its value at most, and one rounding to bf16 of each decayed product
or state value in its sums, 2^-8 of A at most. dg is a sum of differences of row products: k roundings of the sum of
their magnitudes over the document.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu

DEV, K = "cuda:0", 600
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(name, got, ref, mag):
    x = f64(got)
    assert x.shape == ref.shape, (name, x.shape, ref.shape)
    bound = K * 2.0 ** -24 * mag
    if got.dtype == torch.bfloat16:
        bound = bound + 1.01 * 2.0 ** -8 * (np.abs(ref) + mag)
    bad = ~(np.abs(x - ref) <= bound + 1e-37)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[0], x[bad][0], ref[bad][0], bound[bad][0])


class Case:
    def __init__(self, lengths, H, HV, d, dtype="bf16", decay="token", h0=True, dht=True, seed=0, scale=0.11, strong=1.0):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
        self.cu_host = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        T, N, dt = int(self.cu_host[-1]), len(lengths), TYPES[dtype]
        self.cu = torch.from_numpy(self.cu_host).to(DEV)
        # parts of one row, as a projection leaves them
        row = normal(T, (2 * H + HV) * d + 8).to(dt)
        self.q = row[:, :H * d].view(T, H, d)
        self.k = row[:, H * d:2 * H * d].view(T, H, d)
        self.v = row[:, 2 * H * d:(2 * H + HV) * d].view(T, HV, d)
        self.g = -strong * torch.rand(HV if decay == "head" else (T, HV), generator=gen, device=DEV) if decay == "head" else \
            -strong * torch.rand(T, HV, generator=gen, device=DEV) ** 4
        self.do = normal(T, HV, d).to(dt)
        self.h0 = normal(N, HV, d, d) if h0 else None
        self.dht = normal(N, HV, d, d) if dht else None
        self.scale, self.group = scale, HV // H
        self.p = G.LinearProblem(self.cu_host, H, HV, d, dtype=dt, scale=scale, decay=decay, has_h0=h0, want_ht=True)

    def fwd(self, **kw):
        return G.gdn_linear_fwd(self.p, self.q, self.k, self.v, self.g, self.cu, h0=self.h0, **kw)

    def bwd(self, **kw):
        return G.gdn_linear_bwd(self.p, self.q, self.k, self.v, self.g, self.cu, self.do, h0=self.h0, dht=self.dht, **kw)

    def reference(self, magnitudes=False, spread=False):
        m = np.abs if magnitudes else (lambda x: x)
        opt = lambda x: None if x is None else m(f64(x))  # noqa: E731
        q, k, v, do = (m(f64(x)) for x in (self.q, self.k, self.v, self.do))
        if spread:  # a q/k head for each value head
            q, k = np.repeat(q, self.group, 1), np.repeat(k, self.group, 1)
        a, g = (self.cu_host, q, k, v), f64(self.g)
        return lo.fwd(*a, g, opt(self.h0), self.scale), lo.bwd(*a, g, do, opt(self.h0), opt(self.dht), self.scale)

    def check(self, fwd, bwd):
        (o, ht), ref = self.reference()
        (oA, htA), A = self.reference(True)
        close("o", fwd[0], o, oA)
        close("ht", fwd[1], ht, htA)
        for x in ("dq", "dk", "dv", "dh0"):
            if bwd[x] is not None:
                close(x, bwd[x], ref[x], A[x])
        if bwd["dg"] is None:
            return
        AS = self.reference(True, True)[1]
        q, k = (np.repeat(np.abs(f64(x)), self.group, 1) for x in (self.q, self.k))
        rows = (q * AS["dq"]).sum(-1) + (k * AS["dk"]).sum(-1)
        mag = np.zeros_like(rows)
        for n in range(len(self.cu_host) - 1):
            at = slice(self.cu_host[n], self.cu_host[n + 1])
            mag[at] = rows[at].sum(0)
            if self.dht is not None:
                mag[at] += (htA[n] * np.abs(f64(self.dht[n]))).sum((-1, -2))
        close("dg", bwd["dg"], ref["dg"], mag if self.g.dim() == 2 else mag.sum(0))


SHAPES = [([1], 1, 1), ([2, 63, 64, 65], 2, 6), ([129, 0, 1, 300], 2, 4), ([385], 1, 2), ([700, 17, 0, 256, 512], 2, 2),
          ([2049, 1000], 1, 3)]


@pytest.mark.parametrize("lengths,H,HV", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_and_backward(lengths, H, HV, d, dtype):
    c = Case(lengths, H, HV, d, dtype, seed=len(lengths) + d)
    c.check(c.fwd(), c.bwd())


@pytest.mark.parametrize("lengths", [[130, 1], [900, 64]])
@pytest.mark.parametrize("h0,dht", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_with_and_without_states(lengths, h0, dht, decay):
    c = Case(lengths, 2, 4, 64, "bf16", decay, h0, dht, seed=7)
    c.check(c.fwd(), c.bwd())


@pytest.mark.parametrize("strong", [0.0, 30.0, 3000.0])
def test_decays_from_none_to_strong(strong):
    c = Case([700, 100], 1, 2, 64, "f32", seed=2, strong=strong)
    c.check(c.fwd(), c.bwd())


def test_a_decay_of_minus_infinity_drops_the_state():
    """g = -inf in the middle: as if a document began there, also in the gradients; its own gradient is 0."""
    c = Case([200], 1, 2, 64, "f32", seed=4)
    c.g[90] = float("-inf")
    o, ht = c.fwd()
    b = c.bwd()
    two = Case([200], 1, 2, 64, "f32", seed=4)
    cu = np.array([0, 90, 200], np.int32)
    h0 = torch.cat([c.h0, torch.zeros_like(c.h0)])
    dht = torch.cat([torch.zeros_like(c.h0), c.dht])
    p = G.LinearProblem(cu, 1, 2, 64, dtype=torch.float32, scale=c.scale, has_h0=True, want_ht=True)
    a = (p, two.q, two.k, two.v, two.g, torch.from_numpy(cu).to(DEV))
    o2, ht2 = G.gdn_linear_fwd(*a, h0=h0)
    b2 = G.gdn_linear_bwd(*a, two.do, h0=h0, dht=dht)
    # one and the same sums in another order: within the roundings of the larger
    near = lambda x, y: float((x.double() - y.double()).abs().max()) <= K * 2.0 ** -24 * 40 * float(y.abs().max())  # noqa: E731
    assert near(o, o2) and near(ht, ht2[1:])
    for x in ("dq", "dk", "dv"):
        assert near(b[x], b2[x]), x
    assert torch.isfinite(b["dg"]).all() and near(b["dh0"], b2["dh0"][:1])


def test_dg_only_where_wanted_and_repeatable():
    c = Case([900, 33], 2, 6, 128, seed=5)
    b = c.bwd()
    for x, y in ((c.fwd(), c.fwd()), (list(b.values()), list(c.bwd().values()))):
        assert all(torch.equal(s, t) for s, t in zip(x, y))
    without = c.bwd(want_dg=False)
    assert without["dg"] is None
    c.check(c.fwd(), without)
    assert torch.equal(without["dv"], b["dv"]) and torch.equal(without["dh0"], b["dh0"])


def test_what_is_not_finite_stays_in_its_document():
    """NaN and infinity from a token on: earlier chunks and other documents keep their bits."""
    for bad in (float("nan"), float("inf")):
        for which in "qkvg":
            a, b = Case([200, 300, 70], 1, 2, 64, seed=6), Case([200, 300, 70], 1, 2, 64, seed=6)
            getattr(b, which)[200 + 150].fill_(bad if which != "g" else float("nan"))
            o, ht = a.fwd()
            o2, ht2 = b.fwd()
            keep = list(range(328)) + list(range(500, 570))  # all but the third chunk of the second document and what follows
            assert torch.equal(o[keep], o2[keep]) and torch.equal(ht[[0, 2]], ht2[[0, 2]])
            assert not torch.isfinite(o2[350]).all()
            x, y = a.bwd(), b.bwd()
            for name in ("dq", "dk", "dv"):
                other = list(range(200)) + list(range(500, 570))
                assert torch.equal(x[name][other], y[name][other]), (which, name)


def test_rows_of_no_document_stay():
    """Device lengths that end earlier than the host's (a replayed graph): rows behind them keep what the buffers held."""
    for lengths, cu in (([300, 200], [0, 100, 164]), ([3000, 500], [0, 2000, 2700])):
        c = Case(lengths, 1, 2, 64, seed=8)
        c.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        o = torch.full((sum(lengths), 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        ht = torch.full((2, 2, 64, 64), 7.0, device=DEV)
        grads = dict(dq=o[:, :1].clone(), dk=o[:, :1].clone(), dv=o.clone(), dg=torch.full((sum(lengths), 2), 7.0, device=DEV),
                     dh0=ht.clone())
        f, b = c.fwd(o=o, ht=ht), c.bwd(grads=grads)
        end = cu[-1]
        assert (o[end:] == 7).all()
        for x in ("dv", "dg"):
            assert (b[x][end:] == 7).all(), x
        c.cu_host = np.array(cu, np.int32)
        for x in ("q", "k", "v", "g", "do"):
            setattr(c, x, getattr(c, x)[:end])
        c.check((f[0][:end], f[1]), {x: (y if x == "dh0" else y[:end]) for x, y in b.items()})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [2, 6])
def test_gradients_outside_the_documents_stay(dtype, H):
    """Documents from a later first token to an earlier last one: every row of no document keeps what it held."""
    for lengths, cu in (([100, 90], [7, 20, 100]), ([3000, 500], [64, 2000, 2700])):
        c = Case(lengths, H, 6, 64, dtype, seed=14)
        c.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        o = torch.full_like(c.v.contiguous(), 7.0)
        grads = dict(dq=torch.full_like(c.q.contiguous(), 7.0), dk=torch.full_like(c.q.contiguous(), 7.0), dv=o.clone(),
                     dg=torch.full_like(c.g, 7.0))
        c.fwd(o=o)
        b = c.bwd(grads=grads)
        inside = slice(cu[0], cu[-1])
        for x in (o, b["dq"], b["dk"], b["dv"], b["dg"]):
            assert (x[:cu[0]] == 7).all() and (x[cu[-1]:] == 7).all() and not (x[inside] == 7).all()


def test_lengths_outside_the_tokens_are_cut():
    """cu_seqlens that falls or leaves [0, T] on the device: nothing outside the buffers is touched, later calls are whole."""
    c = Case([300, 200, 600], 1, 2, 64, seed=9)
    fence = torch.full((4, 1100, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    ok = c.fwd()
    good = c.cu
    for cu in ([0, 500, 300, 1100], [-5, 400, 2000, 1 << 30], [0, -1, -2, -3], [1100, 0, 1100, 0]):
        c.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        c.fwd(o=fence[1])
        c.bwd(grads=dict(dv=fence[2]))
        torch.cuda.synchronize()
        assert (fence[0] == 3).all() and (fence[3] == 3).all()
    c.cu = good
    assert all(torch.equal(x, y) for x, y in zip(ok, c.fwd()))


def test_streams_and_graph():
    """Another stream, given buffers, and a captured forward and backward replayed on new inputs beside eager work."""
    c = Case([700, 100, 31], 2, 4, 64, seed=10)
    f, b = c.fwd(), c.bwd()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    f2, b2 = c.fwd(stream=s), c.bwd(stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(f + tuple(b.values()), f2 + tuple(b2.values())))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f3, b3 = c.fwd(), c.bwd()
    for i in range(3):
        c.do.mul_(-1.5)
        c.v.add_(0.25)
        want, wantb = c.fwd(), c.bwd()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(f3, want)), i
        assert all(torch.equal(b3[x], wantb[x]) for x in wantb), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_document_through_states(dtype):
    """A document in two calls, the second from the first's last state, is the document in one."""
    c = Case([1500], 1, 2, 128, dtype, h0=False, dht=False, seed=11)
    o, ht = c.fwd()
    S, outs = None, []
    for lo_, hi in ((0, 801), (801, 1500)):
        p = G.LinearProblem([0, hi - lo_], 1, 2, 128, dtype=TYPES[dtype], scale=c.scale, has_h0=S is not None, want_ht=True)
        x, S = G.gdn_linear_fwd(p, c.q[lo_:hi], c.k[lo_:hi], c.v[lo_:hi], c.g[lo_:hi],
                                torch.tensor([0, hi - lo_], dtype=torch.int32, device=DEV), h0=S)
        outs.append(x)
    (_, _), _ = (o, ht), None
    ref, A = c.reference()[0], c.reference(True)[0]
    for got in ((o, ht), (torch.cat(outs), S)):
        close("o", got[0], ref[0], A[0])
        close("ht", got[1], ref[1], A[1])


# ------------------------------------------------------------------------------------------ the step


@pytest.mark.parametrize("lengths", [[1], [1] * 9, [3, 0, 1, 8], [40, 2], [1] * 70])
@pytest.mark.parametrize("H,HV,d", [(1, 1, 64), (2, 6, 128), (16, 48, 128)])
@pytest.mark.parametrize("dtype,decay", [("bf16", "token"), ("f32", "head")])
def test_step(lengths, H, HV, d, dtype, decay):
    if sum(lengths) * HV > 700:
        lengths = lengths[:9]
    c = Case(lengths, H, HV, d, dtype, decay, seed=3)
    N, T, one = len(lengths), int(c.cu_host[-1]), max(lengths) == 1
    for keep in (False, True):
        n_slots = 2 * N + T + 2
        order = torch.randperm(n_slots, generator=torch.Generator().manual_seed(N)).to(torch.int32).to(DEV)
        slot_in, slot_out = order[:N].clone(), order[:N].clone()
        slot_in[N // 2] = -1  # a new sequence
        if N > 1:
            slot_out[0] = order[N]
            slot_out[N - 1] = -1
        slot_tok = order[2 * N:2 * N + T].clone() if keep else None
        if keep and T > 2:
            slot_tok[1] = -1
        states = torch.randn(n_slots, HV, d, d, device=DEV)
        before = states.clone()
        p = G.LinearStepProblem(N, H, HV, d, n_slots, cu_seqlens_host=None if one else c.cu_host, dtype=TYPES[dtype],
                                scale=c.scale, decay=decay)
        o = G.gdn_linear_step(p, c.q, c.k, c.v, c.g, states, slot_in, slot_out, slot_tok=slot_tok,
                              cu_seqlens=None if one else c.cu)
        ins = slot_in.tolist()
        h0 = np.stack([f64(before[i]) if i >= 0 else np.zeros((HV, d, d)) for i in ins])
        a = [f64(x) for x in (c.q, c.k, c.v)]
        ref, kept = lo.steps(c.cu_host, *a, f64(c.g), h0, c.scale)
        A, keptA = lo.steps(c.cu_host, *[np.abs(x) for x in a], f64(c.g), np.abs(h0), c.scale)
        close("o", o, ref, A * (2.0 ** -14 if dtype == "bf16" else 1))  # FP32 throughout: bf16 only rounds the output
        touched = set()
        for n in range(N):
            last = c.cu_host[n + 1] - 1
            slot = int(slot_out[n])
            if slot >= 0:
                touched.add(slot)
                empty = lengths[n] == 0
                close("state", states[slot], h0[n] if empty else kept[last], np.abs(h0[n]) if empty else keptA[last])
        if keep:
            for t, slot in enumerate(slot_tok.tolist()):
                if slot >= 0 and slot not in touched:
                    touched.add(slot)
                    close("kept", states[slot], kept[t], keptA[t])
        rest = [s for s in range(n_slots) if s not in touched]
        assert torch.equal(states[rest], before[rest])


def test_step_checks_slots_and_ranges():
    """A slot outside the cache or a range outside the tokens: NaN rows, no state written, neighbours untouched."""
    N, d = 4, 64
    c = Case([1] * N, 1, 2, d, seed=1)
    p = G.LinearStepProblem(N, 1, 2, d, 5, scale=c.scale)
    good = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    base = torch.randn(5, 2, d, d, device=DEV)
    s0 = base.clone()
    want = G.gdn_linear_step(p, c.q, c.k, c.v, c.g, s0, good, good)
    for which in ("slot_in", "slot_out", "slot_tok"):
        for bad in (5, -2, 1 << 30, -(1 << 31)):
            a = dict(slot_in=good.clone(), slot_out=good.clone(), slot_tok=None)
            if which == "slot_tok":
                a["slot_tok"] = torch.full((N,), -1, dtype=torch.int32, device=DEV)
            a[which][2] = bad
            s = base.clone()
            o = G.gdn_linear_step(p, c.q, c.k, c.v, c.g, s, a["slot_in"], a["slot_out"], slot_tok=a["slot_tok"])
            assert torch.isnan(o[2]).all() and torch.equal(o[[0, 1, 3]], want[[0, 1, 3]]), (which, bad)
            if which != "slot_tok":
                assert torch.equal(s[[2, 4]], base[[2, 4]])
            assert torch.equal(s[[0, 1, 3]], s0[[0, 1, 3]])
    p = G.LinearStepProblem(3, 1, 2, d, 5, cu_seqlens_host=[0, 1, 2, 4], scale=c.scale)
    for cu in ([0, 9, 2, 4], [0, 1, -3, 4], [0, 4, 1, 1 << 30]):
        s, slots = base.clone(), good[:3]
        G.gdn_linear_step(p, c.q, c.k, c.v, c.g, s, slots, slots, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        assert torch.equal(s[3:], base[3:])


def test_step_continues_the_chunked_form():
    """A prompt through the chunked form, then tokens one by one, is the whole sequence through it."""
    c = Case([310], 2, 4, 128, "f32", h0=False, dht=False, seed=12)
    o, ht = c.fwd()
    p = G.LinearProblem([0, 300], 2, 4, 128, dtype=torch.float32, scale=c.scale, want_ht=True)
    _, states = G.gdn_linear_fwd(p, c.q[:300], c.k[:300], c.v[:300], c.g[:300], torch.tensor([0, 300], dtype=torch.int32, device=DEV))
    step, slot = G.LinearStepProblem(1, 2, 4, 128, 1, dtype=torch.float32, scale=c.scale), torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = [G.gdn_linear_step(step, c.q[t:t + 1], c.k[t:t + 1], c.v[t:t + 1], c.g[t:t + 1], states, slot, slot) for t in range(300, 310)]
    ref, A = c.reference()[0], c.reference(True)[0]
    close("o", torch.cat(outs), ref[0][300:], A[0][300:])
    close("state", states, ref[1], A[1])


def test_step_graph_and_stream():
    c = Case([1] * 6, 2, 6, 128, seed=2)
    p, slots = G.LinearStepProblem(6, 2, 6, 128, 6, scale=c.scale), torch.arange(6, dtype=torch.int32, device=DEV)
    states = torch.randn(6, 6, 128, 128, device=DEV)
    eager = states.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = G.gdn_linear_step(p, c.q, c.k, c.v, c.g, states, slots, slots)
    s = torch.cuda.Stream()
    for _ in range(3):
        c.v.mul_(-0.5)
        s.wait_stream(torch.cuda.current_stream())
        want = G.gdn_linear_step(p, c.q, c.k, c.v, c.g, eager, slots, slots, stream=s)
        s.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(states, eager)


def test_binding_refusals():
    c = Case([5, 6], 1, 2, 64, seed=1)
    a = [c.p, c.q, c.k, c.v, c.g, c.cu]
    for i, bad in ((1, c.q[:-1]), (1, c.q.float()), (2, c.k.transpose(0, 1)), (3, c.v[:, :1]), (4, c.g[0]), (4, c.g.double()),
                   (5, c.cu.long()), (5, c.cu[:-1]), (5, c.cu.cpu())):
        x = list(a)
        x[i] = bad
        with pytest.raises(G.GdnError):
            G.gdn_linear_fwd(*x, h0=c.h0)
        with pytest.raises(G.GdnError):
            G.gdn_linear_bwd(*x, c.do, h0=c.h0)
    with pytest.raises(G.GdnError):
        G.gdn_linear_fwd(*a)  # has_h0
    with pytest.raises(G.GdnError):
        G.gdn_linear_bwd(*a, c.do[:3], h0=c.h0)
    with pytest.raises(G.GdnError):
        G.gdn_linear_fwd(*a, h0=c.h0, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
