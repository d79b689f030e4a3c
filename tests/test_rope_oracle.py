"""The norm + rotation oracle against what fixes it independently (closed forms, torch's float64 norm
and autograd, central differences), the host's frequencies against it, and planted mistakes."""
import importlib.util
import math

import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
from oracle import rope_oracle

SRC = rope_oracle.__file__
T, H, D = 5, 2, 16
POS = np.array([0, 1, 7, -3, 4000])


def _inputs(seed=0):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((T, H, D)), rng.standard_normal((T, H, D)), 1 + 0.2 * rng.standard_normal(D)


def pin_rotation_matrix(mod):
    """Each pair is a 2 x 2 rotation by p f_i; the rest of the head passes."""
    x, _, _ = _inputs(1)
    f, _ = mod.frequencies(8, base=100.0)
    for interleaved in (False, True):
        y = mod.fwd(x, POS, f, norm="none", rotary_dim=8, interleaved=interleaved, m=1.5)
        np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
        for t, p in enumerate(POS):
            for i in range(4):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 4)
                th = p * 100.0 ** (-2 * i / 8)
                R = 1.5 * np.array([[math.cos(th), -math.sin(th)], [math.sin(th), math.cos(th)]])
                np.testing.assert_allclose(y[t][:, [a, b]], x[t][:, [a, b]] @ R.T, rtol=1e-10, atol=1e-10)


def pin_relative_positions(mod):
    """<y_q(p), y_k(p')> depends on p - p' alone."""
    x, z, _ = _inputs(2)
    f, _ = mod.frequencies(D)
    for interleaved in (False, True):
        at = lambda v, shift: mod.fwd(v, POS * 0 + shift, f, norm="l2", interleaved=interleaved)
        one = np.sum(at(x, 9) * at(z, 4), -1)
        two = np.sum(at(x, 1005) * at(z, 1000), -1)
        np.testing.assert_allclose(one, two, rtol=1e-9, atol=1e-9)
        assert np.max(np.abs(one - np.sum(at(x, 9) * at(z, 9), -1))) > 1e-2


def pin_torch_norm_autograd(mod):
    """Position 0 leaves the norm: torch's rms_norm and normalize in float64, gradients by autograd."""
    x, dy, w = _inputs(3)
    f, _ = mod.frequencies(D)
    for norm in ("rms", "l2"):
        xt, wt = (torch.tensor(v, requires_grad=True) for v in (x, w))
        if norm == "rms":
            y = torch.nn.functional.rms_norm(xt, (D,), wt, eps=1e-6)
        else:
            y = xt * torch.rsqrt((xt * xt).sum(-1, keepdim=True) + 1e-6) * wt
        (y * torch.tensor(dy)).sum().backward()
        np.testing.assert_allclose(mod.fwd(x, POS * 0, f, w, norm), y.detach().numpy(), rtol=1e-12)
        dx, dw = mod.bwd(x, dy, POS * 0, f, w, norm)
        np.testing.assert_allclose(dx, xt.grad.numpy(), rtol=1e-10, atol=1e-12)
        np.testing.assert_allclose(dw, wt.grad.numpy(), rtol=1e-10, atol=1e-12)


def pin_differences(mod):
    """Central differences of <dy, y> on x and w."""
    x, dy, w = _inputs(4)
    f, _ = mod.frequencies(8)
    for norm in ("rms", "l2", "none"):
        for interleaved in (False, True):
            kw = dict(norm=norm, rotary_dim=8, interleaved=interleaved, eps=1e-2, m=1.3)
            wt = None if norm == "none" else w
            dx, dw = mod.bwd(x, dy, POS, f, wt, **kw)
            loss = lambda x_, w_: float(np.sum(dy * mod.fwd(x_, POS, f, w_, **kw)))
            h = 1e-5
            for idx in np.ndindex(x.shape):
                e = np.zeros_like(x)
                e[idx] = h
                fd = (loss(x + e, wt) - loss(x - e, wt)) / (2 * h)
                assert abs(fd - dx[idx]) < 1e-7, (norm, idx)
            if wt is not None:
                for i in range(D):
                    e = np.zeros(D)
                    e[i] = h
                    assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def pin_frequencies(mod):
    """Closed forms of the scalings, and the ends of the two blends."""
    plain, m = mod.frequencies(64)
    np.testing.assert_allclose(plain, [10000.0 ** (-i / 32) for i in range(32)], rtol=1e-14)
    assert m == 1.0
    np.testing.assert_allclose(mod.frequencies(64, scaling="linear", factor=8.0)[0], plain / 8, rtol=1e-14)
    ntk = mod.frequencies(64, scaling="ntk", factor=8.0)[0]
    np.testing.assert_allclose(ntk[[0, -1]], [1.0, plain[-1] / 8], rtol=1e-12)  # the slowest pair by the factor
    f, m = mod.frequencies(64, scaling="yarn", factor=8.0, original_length=4096)
    turns = 4096 * plain / (2 * math.pi)
    np.testing.assert_allclose(f[turns > 45], plain[turns > 45], rtol=1e-14)
    np.testing.assert_allclose(f[turns < 0.7], plain[turns < 0.7] / 8, rtol=1e-14)
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-14
    f, m = mod.frequencies(64, scaling="bands", factor=8.0, original_length=4096, fast=4.0)
    np.testing.assert_allclose(f[turns >= 4], plain[turns >= 4], rtol=1e-14)
    np.testing.assert_allclose(f[turns <= 1], plain[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all((f[mid] < plain[mid]) & (f[mid] > plain[mid] / 8)) and m == 1.0


ALL_PINS = [pin_rotation_matrix, pin_relative_positions, pin_torch_norm_autograd, pin_differences, pin_frequencies]


@pytest.mark.parametrize("pin", ALL_PINS, ids=[p.__name__ for p in ALL_PINS])
def test_rope_oracle_pin(pin):
    pin(rope_oracle)


MUTANTS = [
    ("turned_back", "angle = np.asarray(positions, dtype=np.float64)[:, None] * f\n    return", "angle = -np.asarray(positions, dtype=np.float64)[:, None] * f\n    return"),
    ("pairs_of_the_other_layout", "if interleaved else (slice(0, r // 2), slice(r // 2, r))", "if not interleaved else (slice(0, r // 2), slice(r // 2, r))"),
    ("gradient_not_turned_back", "dz = _turn(dy, -angle,", "dz = _turn(dy, angle,"),
    ("projection_dropped", "dx = r * (dn - c * n * np.sum(n * dn, -1, keepdims=True))", "dx = r * dn"),
    ("mean_for_sum", "1 / np.sqrt(np.sum(x * x, -1, keepdims=True) + eps), 1.0", "1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps), 1.0"),
    ("weight_gradient_from_dn", "np.sum(dz * n, axis=(0, 1))", "np.sum(dn * n, axis=(0, 1))"),
    ("magnitude_dropped", "(m * np.exp(1j * angle))", "(np.exp(1j * angle))"),
    ("blend_upside_down", "f * (1 - r) + f / factor * r", "f * r + f / factor * (1 - r)"),
    ("exponent_off", "f = base ** (-2.0 * i / rotary_dim)", "f = base ** (-2.0 * i / (rotary_dim - 2))"),
]


@pytest.mark.parametrize("name,find,repl", MUTANTS, ids=[m[0] for m in MUTANTS])
def test_rope_pins_catch_mutant(name, find, repl, tmp_path):
    src = open(SRC).read()
    assert src.count(find) == 1, "mutation anchor not found: %r" % find
    path = tmp_path / "rope_mutant.py"
    path.write_text(src.replace(find, repl))
    spec = importlib.util.spec_from_file_location("rope_mutant", str(path))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    caught = []
    for pin in ALL_PINS:
        try:
            pin(mod)
        except AssertionError:
            caught.append(pin.__name__)
    assert caught, "no pin catches the planted mistake %s" % name


@pytest.mark.parametrize("kw", [
    {}, dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="yarn", factor=4.0, original_length=32768), dict(scaling="yarn", factor=0.5, original_length=100),
    dict(scaling="bands", factor=8.0, original_length=8192, fast=4.0, slow=1.0)], ids=str)
@pytest.mark.parametrize("rotary", [8, 64, 96, 256])
def test_frequencies_of_the_library(kw, rotary):
    """The 64-bit fractions of a turn give the oracle's frequencies to 1e-13 (the doubles' own
    rounding over a few operations), and the angle at a far position to what 2^-64 turns allow."""
    turns, m = G.gdn_rope_frequencies(rotary, **kw)
    f, m_ref = rope_oracle.frequencies(rotary, **kw)
    got = turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    assert turns.shape == (rotary // 2,)
    np.testing.assert_allclose(got, f, rtol=1e-13)
    assert abs(m - m_ref) < 1e-6


@pytest.mark.parametrize("kw,fragment", [
    (dict(rotary_dim=7), "even"), (dict(rotary_dim=0), "even"), (dict(base=1.0), "base"), (dict(base=float("nan")), "base"),
    (dict(scaling="linear", factor=0.0), "factor"), (dict(scaling="linear", factor=float("inf")), "factor"),
    (dict(scaling="ntk", rotary_dim=2, factor=2.0), "rotary_dim"), (dict(scaling="yarn", factor=2.0), "original_length"),
    (dict(scaling="bands", factor=2.0, original_length=10, fast=1.0, slow=1.0), "fast"),
    (dict(scaling="other"), "unknown scaling")], ids=str)
def test_frequencies_refusals(kw, fragment):
    a = dict(rotary_dim=64)
    a.update(kw)
    with pytest.raises(G.GdnError, match=fragment):
        G.gdn_rope_frequencies(**a)


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=1e-320), dict(scaling="ntk", factor=1e-300),
    dict(scaling="yarn", factor=4.0, original_length=1e300, fast=2e-300, slow=1e-300),
    dict(scaling="bands", factor=1e-300, original_length=1e-3)], ids=str)
def test_frequencies_that_are_no_numbers_are_refused(kw):
    """Settings in range one by one whose frequencies are infinite, NaN or without a fraction."""
    with pytest.raises(G.GdnError, match="frequency"):
        G.gdn_rope_frequencies(64, **kw)
