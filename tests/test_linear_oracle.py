"""The FP64 reference of linear attention: the masked product against the recurrence, gradients against
differences, on the CPU."""
import numpy as np
import pytest

from oracle import linear_oracle as lo


def make(lengths, H, HV, d, seed=0, by_head=False):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    T, N = cu[-1], len(lengths)
    g = -r.random(HV) if by_head else -r.random((T, HV))
    return cu, [r.standard_normal((T, H, d)), r.standard_normal((T, H, d)), r.standard_normal((T, HV, d)), g], \
        r.standard_normal((N, HV, d, d)), r


@pytest.mark.parametrize("by_head", [False, True])
@pytest.mark.parametrize("lengths", [[1], [5, 0, 9], [70]])
def test_masked_product_is_the_recurrence(lengths, by_head):
    cu, a, h0, _ = make(lengths, 2, 4, 6, by_head=by_head)
    o, ht = lo.fwd(cu, *a, h0, scale=0.3)
    o2, kept = lo.steps(cu, *a, h0, scale=0.3)
    np.testing.assert_allclose(o, o2, rtol=1e-11, atol=1e-11)
    for n, length in enumerate(lengths):
        np.testing.assert_allclose(ht[n], kept[cu[n + 1] - 1] if length else h0[n], rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("by_head", [False, True])
def test_gradients_are_differences(by_head):
    cu, a, h0, r = make([4, 0, 3], 2, 4, 3, seed=3, by_head=by_head)
    do, dht = r.standard_normal(a[2].shape), r.standard_normal(h0.shape)

    def loss():
        o, ht = lo.fwd(cu, *a, h0, scale=0.7)
        return (o * do).sum() + (ht * dht).sum()

    got = lo.bwd(cu, *a, do, h0, dht, scale=0.7)
    for x, dx in zip(a + [h0], [got["dq"], got["dk"], got["dv"], got["dg"], got["dh0"]]):
        assert x.shape == dx.shape
        for at in np.ndindex(x.shape):
            keep, e = x[at], 1e-5
            x[at] = keep + e
            up = loss()
            x[at] = keep - e
            down = loss()
            x[at] = keep
            assert abs((up - down) / (2 * e) - dx[at]) < 1e-7 * (1 + abs(dx[at]))
