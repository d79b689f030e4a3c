"""The decays' gradient of linear attention on documents that are cut into segments (where it is summed from <S, D> at the
borders), in both types and forms of the decays, with and without states, to 20,001 tokens. The root mean square of its errors over
a document is held to the bound that linear_util.py derives: about 2e-5 of dg's for decays a token, 6e-4 for one a head."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
import linear_util as u
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def gpu(x, dtype=torch.float32):
    return None if x is None else torch.from_numpy(x).to(DEV).to(dtype)


def check(lengths, H, HV, d, decay, h0, dht, dtypes, scale=0.11):
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    a = u.dg_inputs(lengths, H, HV, d, decay, h0, dht, len(lengths) + d)
    ref, rows, norms = lo.dg_by_states(cu, *[None if x is None else x.astype(np.float64) for x in a], scale)
    q, k, v, g, do, H0, DT = a
    by_head = decay == "head"
    for dtype in dtypes:
        dt = TYPES[dtype]
        p = G.LinearProblem(cu, H, HV, d, dtype=dt, scale=scale, decay=decay, has_h0=h0)
        assert u.backward_is_cut(p, H, HV, d, dtype)
        b = G.gdn_linear_bwd(p, gpu(q, dt), gpu(k, dt), gpu(v, dt), gpu(g), gpu(cu, torch.int32), gpu(do, dt), h0=gpu(H0), dht=gpu(DT))
        got = b["dg"].double().cpu().numpy()
        bounds = u.dg_bounds(cu, rows, norms, d, by_head, u.most_tokens(dtype, decay))
        for x, y, bound in zip(u.dg_parts(cu, got, by_head), u.dg_parts(cu, ref, by_head), bounds):
            if x.size == 0:
                continue
            off, rms = (float(np.sqrt((z ** 2).mean())) for z in (x - y, y))
            print("%s %s: off by %.2e of %.2e, held to %.2e" % (dtype, x.shape, off, rms, bound), flush=True)
            assert off <= bound


@pytest.mark.parametrize("lengths,H,HV,d", [([900, 64], 2, 4, 64), ([2049, 1000], 1, 3, 128)])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("h0,dht", [(False, False), (True, False), (False, True), (True, True)])
def test_documents_of_several_segments(lengths, H, HV, d, decay, h0, dht):
    check(lengths, H, HV, d, decay, h0, dht, ("bf16", "f32"))


@pytest.mark.parametrize("decay,states", [("token", False), ("token", True), ("head", False)])
def test_long_documents(decay, states):
    check([20001, 1, 0, 65], 1, 1, 64, decay, states, states, ("bf16", "f32"))
