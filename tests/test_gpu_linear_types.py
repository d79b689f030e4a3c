"""Linear attention in the types and forms that test_gpu_linear.py leaves out: one decay a head in f32 and over several
segments, the step with one decay a head in bf16 and with decays a token in f32 (one token, runs, kept states).

Bounds as there."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
from oracle import linear_oracle as lo
from test_gpu_linear import DEV, TYPES, Case, close, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,H,HV", [([1], 1, 1), ([65, 0, 130], 2, 6), ([1500, 40], 1, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h0,dht", [(True, True), (False, False)])
def test_one_decay_a_head(lengths, H, HV, d, dtype, h0, dht):
    c = Case(lengths, H, HV, d, dtype, "head", h0, dht, seed=d + len(lengths))
    c.check(c.fwd(), c.bwd())


@pytest.mark.parametrize("lengths", [[1] * 5, [3, 0, 1, 8], [21]])
@pytest.mark.parametrize("H,HV,d", [(2, 6, 128), (1, 2, 64)])
@pytest.mark.parametrize("dtype,decay", [("bf16", "head"), ("f32", "token")])
@pytest.mark.parametrize("keep", [False, True])
def test_step(lengths, H, HV, d, dtype, decay, keep):
    c = Case(lengths, H, HV, d, dtype, decay, seed=4)
    N, T, one = len(lengths), int(c.cu_host[-1]), max(lengths) == 1
    n_slots = 2 * N + T
    order = torch.randperm(n_slots, generator=torch.Generator().manual_seed(N)).to(torch.int32).to(DEV)
    slot_in, slot_out = order[:N].clone(), order[N:2 * N].clone()
    slot_in[-1] = -1
    slot_tok = order[2 * N:].clone() if keep else None
    states = torch.randn(n_slots, HV, d, d, device=DEV)
    before = states.clone()
    p = G.LinearStepProblem(N, H, HV, d, n_slots, cu_seqlens_host=None if one else c.cu_host, dtype=TYPES[dtype], scale=c.scale,
                            decay=decay)
    o = G.gdn_linear_step(p, c.q, c.k, c.v, c.g, states, slot_in, slot_out, slot_tok=slot_tok, cu_seqlens=None if one else c.cu)
    h0 = np.stack([f64(before[i]) if i >= 0 else np.zeros((HV, d, d)) for i in slot_in.tolist()])
    a = [f64(x) for x in (c.q, c.k, c.v)]
    ref, kept = lo.steps(c.cu_host, *a, f64(c.g), h0, c.scale)
    A, keptA = lo.steps(c.cu_host, *[np.abs(x) for x in a], f64(c.g), np.abs(h0), c.scale)
    close("o", o, ref, A * (2.0 ** -14 if dtype == "bf16" else 1))  # FP32 throughout: bf16 only rounds the output
    untouched = torch.ones(n_slots, dtype=torch.bool)
    for n, slot in enumerate(slot_out.tolist()):
        last = c.cu_host[n + 1] - 1
        want = (h0[n], np.abs(h0[n])) if lengths[n] == 0 else (kept[last], keptA[last])
        close("state", states[slot], *want)
        untouched[slot] = False
    if keep:
        for t, slot in enumerate(slot_tok.tolist()):
            close("kept", states[slot], kept[t], keptA[t])
            untouched[slot] = False
    assert torch.equal(states[untouched], before[untouched])
