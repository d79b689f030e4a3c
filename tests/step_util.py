"""Bounds for the tests of the serving steps and of the rotation, elementwise against float64.

f32 results: `k` roundings of 2^-24 of the largest value of the reference, k from the operation's
length (a sum of 128 products rounds at most 128 times, a state a few hundred times before its decay
forgets it). bf16 results: one rounding to 8 significant bits is at most 2^-9 of the value; twice
that leaves room for a value that lies at a rounding boundary, plus the f32 bound."""
import numpy as np
import torch


def check(name, got, ref, k):
    got_np = got.detach().double().cpu().numpy()
    ref = np.asarray(ref, dtype=np.float64)
    assert got_np.shape == ref.shape, (name, got_np.shape, ref.shape)
    if not ref.size:
        return
    assert np.all(np.isfinite(got_np)), "%s: non-finite values" % name
    bound = k * 2.0 ** -24 * np.max(np.abs(ref))
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(ref)
    off = np.abs(got_np - ref) - bound
    at = np.unravel_index(np.argmax(off), off.shape)
    assert off[at] <= 0, "%s at %s: %.9g, expected %.9g" % (name, at, got_np[at], ref[at])


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()
