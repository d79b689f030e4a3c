"""On the CPU: the reference of dg by its definition against the one by pairs of tokens, and that the bounds that dg is held to
tell it from mistakes: left out, of the wrong sign, one token off, without a segment's border, without a segment."""
import numpy as np
import pytest

import linear_util as u
from oracle import linear_oracle as lo


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("h0,dht", [(False, False), (True, False), (False, True), (True, True)])
def test_definition_and_pairs(h0, dht, decay):
    cu = np.array([0, 70, 70, 71, 201])
    a = u.dg_inputs([70, 0, 1, 130], 2, 4, 8, decay, h0, dht, 3)
    q, k, v, g, do, H0, DT = (None if x is None else x.astype(np.float64) for x in a)
    dg = lo.dg_by_states(cu, q, k, v, g, do, H0, DT, 0.3)[0]
    np.testing.assert_allclose(dg, lo.bwd(cu, q, k, v, g, do, H0, DT, 0.3)["dg"], rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("lengths,H,HV,d", [([900, 64], 2, 4, 64), ([2049, 1000], 1, 3, 128)])
@pytest.mark.parametrize("dtype,decay", [("bf16", "token"), ("f32", "token"), ("f32", "head")])
@pytest.mark.parametrize("states", [False, True])
def test_bounds_tell_mistakes(lengths, H, HV, d, dtype, decay, states):
    cu = np.concatenate([[0], np.cumsum(lengths)])
    a = u.dg_inputs(lengths, H, HV, d, decay, states, states, 1)
    q, k, v, g, do, h0, dht = (None if x is None else x.astype(np.float64) for x in a)
    dg, rows, norms = lo.dg_by_states(cu, q, k, v, g, do, h0, dht, 0.11)
    by_head = decay == "head"
    per_token = dg
    if by_head:
        per_token = lo.dg_by_states(cu, q, k, v, np.broadcast_to(g, v.shape[:2]), do, h0, dht, 0.11)[0]
    bounds = u.dg_bounds(cu, rows, norms, d, by_head, u.most_tokens(dtype, decay))
    cut = per_token.copy()  # a border's <S, D> left out of the segment before it
    cut[:64] -= per_token[64]
    gone = per_token.copy()  # a segment left out
    gone[64:128] = 0
    late = np.concatenate([per_token[1:], per_token[:1]])
    for name, wrong in (("zero", 0 * per_token), ("sign", -per_token), ("border", cut), ("segment", gone), ("late", late)):
        if name == "late" and by_head:
            continue  # the same sum
        wrong = wrong.sum(0) if by_head else wrong
        off = [float(np.sqrt(((x - y) ** 2).mean())) for x, y in zip(u.dg_parts(cu, wrong, by_head), u.dg_parts(cu, dg, by_head))]
        assert off[0] > 20 * bounds[0], (name, off, bounds)
        rms = float(np.sqrt((dg ** 2).mean()))
        assert max(bounds) < (1e-3 if by_head else 3e-5) * rms, (bounds, rms)
