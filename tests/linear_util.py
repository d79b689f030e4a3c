"""Shared by the tests of the decays' gradient of linear attention: inputs, how far dg may be off, whether a call is cut
into segments.

How far. dg is summed over tokens inside a segment of at most n tokens, from row products q.dq - k.dk (d products each) and from
<S, D> at the segment's borders. dq, dk, S and D are FP32 sums of independent roundings, some 40 on the way to one (a
chunk's products over d and 64 values in steps of 32, in up to three terms, P's before them and the states' after), each
of 2^-24 at most and 0.4 2^-24 in the root mean square: 2.5 2^-24, with a margin KAPPA = 4. An error of that size in each of a
row's values leaves KAPPA 2^-24 |q| |dq| / sqrt(d) in its product, n tokens sqrt(n) times as much, and <S, D> is off by
KAPPA 2^-24 |S| |D| / d. So the root mean square of dg's errors over a document is held to twice (few segments: few
independent errors) KAPPA 2^-24 (sqrt(n) rms(|q||dq| + |k||dk|) / sqrt(d) + rms(|S||D|) / d). One decay a head adds up dg over the
document: n times the error of each segment, and segments independently, so sqrt(T / n) n of the same."""
import numpy as np

import gated_deltanet_fwd_amd as G

KAPPA = 4


def dg_inputs(lengths, H, HV, d, decay, h0, dht, seed):
    """numpy float32: q, k, v, g, do, h0, dht. Values that bf16 holds, so that one reference serves both types."""
    r = np.random.default_rng(seed)
    T, N = int(sum(lengths)), len(lengths)
    short = lambda x: (x.astype(np.float32).view(np.uint32) & 0xffff0000).view(np.float32)  # noqa: E731
    q, k = (short(r.standard_normal((T, H, d))) for _ in range(2))
    v, do = (short(r.standard_normal((T, HV, d))) for _ in range(2))
    g = (-r.random(HV) if decay == "head" else -r.random((T, HV)) ** 4).astype(np.float32)
    state = lambda want: r.standard_normal((N, HV, d, d)).astype(np.float32) if want else None  # noqa: E731
    return q, k, v, g, do, state(h0), state(dht)


def most_tokens(dtype, decay):
    """Of a segment of the backward."""
    return 1024 if dtype == "bf16" and decay == "token" else 512


def dg_bounds(cu, rows, states, d, by_head, n):
    """Of the root mean square of dg's errors, for each document (by_head: one for the vector over the heads)."""
    rms = lambda x: float(np.sqrt((x * x).mean())) if x.size else 0.0  # noqa: E731
    one = []
    for b, e in zip(cu[:-1], cu[1:]):
        m = min(n, max(int(e - b), 1))
        x = 2 * KAPPA * 2.0 ** -24 * (np.sqrt(m) * rms(rows[b:e]) / np.sqrt(d) + rms(states[b:e]) / d)
        one.append(x * m * np.sqrt(max((e - b) / m, 1)) if by_head else x)
    return [float(np.sqrt((np.array(one) ** 2).sum()))] if by_head else one


def dg_parts(cu, dg, by_head):
    """What each bound is for."""
    return [dg] if by_head else [dg[b:e] for b, e in zip(cu[:-1], cu[1:])]


def backward_is_cut(p, H, HV, d, dtype):
    """Whether the plan has segments: its workspace holds more than an uncut call's."""
    size = 2 if dtype == "bf16" else 4
    T, N = p.st.n_tokens, p.st.n_seqs
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    uncut = 2 * up(T * HV * 4) + up(N * HV * 8)
    if H != HV:
        uncut += 2 * (up(T * HV * d * size) + (up(T * HV * 16) if size == 2 else 0))
    have = G.gdn_linear_workspace_bytes(p, G.OP_BWD)
    assert have >= uncut
    return have > uncut
