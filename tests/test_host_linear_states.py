"""Linear attention refuses states that it writes over states that it reads (no GPU)."""
import ctypes

import pytest

import gated_deltanet_fwd_amd as G

PTR, FAR = 4096, 1 << 40  # never read: every call here is refused first
SIZE = 3 * 4 * 64 * 64 * 4


def problem():
    return G.LinearProblem([0, 5, 5, 75], 2, 4, 64, has_h0=True, want_ht=True)


def refused(text, rc):
    assert rc == 1 and text in G.load_library().gdn_last_error().decode(), (rc, G.load_library().gdn_last_error())


@pytest.mark.parametrize("apart", [0, 16, SIZE - 16])
@pytest.mark.parametrize("sign", [1, -1])
def test_states_over_each_other(apart, sign):
    x = [ctypes.c_void_p(PTR)] * 16
    at = FAR + sign * apart
    lib, h0, end = G.load_library(), ctypes.c_void_p(FAR), ctypes.c_void_p(at)
    refused("ht must not overlap h0", lib.gdn_linear_fwd(problem().ref(), *x[:5], h0, x[0], end, x[0], 1 << 40, None))
    # dh0 over h0, then over dht
    refused("dh0 must not overlap h0", lib.gdn_linear_bwd(problem().ref(), *x[:5], h0, x[0], None, *x[:3], x[0], end, x[0], 1 << 40, None))
    refused("dh0 must not overlap dht", lib.gdn_linear_bwd(problem().ref(), *x[:5], ctypes.c_void_p(1 << 42), x[0], h0, *x[:3], x[0], end,
                                                           x[0], 1 << 40, None))
