"""GPU test of the operators as they are used together: prompts through the chunked path, decoding on
cached states and windows, against the whole sequences through the chunked path. The chunked path is
held to 1e-2 of the oracle and the steps to one bf16 rounding, so the two agree to 1e-2."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("kw", [dict(lengths=(70, 1, 3, 200), steps=20, h_qk=2, h_v=6),
                                dict(lengths=(64,), steps=5, h_qk=1, h_v=1, d=64, rotary=16)], ids=["128", "64"])
def test_decoding_continues_the_prompts(kw, graph):
    from serve import serve

    o, s = serve(graph=graph, **kw)
    print("decoded outputs off by %.2e, states by %.2e" % (o, s))
    assert o <= 1e-2 and s <= 1e-2
