"""FP64 reference of linear attention with decays (test infrastructure only), each document and head as one
masked product of all its tokens with all:

    o_t = scale (sum_{s <= t} e^{G_t - G_s} (q_t.k_s) v_s + e^{G_t} q_t h0),   G_t = g_1 + .. + g_t
    ht  = sum_s e^{G_T - G_s} k_s v_s^T + e^{G_T} h0

and `steps` the same token by token. Arrays are numpy float64; q, k [T, H, d], v [T, HV, d], g [T, HV] or [HV].
With absolute values for every input but g the results are the sums of the magnitudes of what is added up, which
bound what rounding any term of them can change.
"""
import numpy as np


def _log_decays(g, t, hv):
    return np.broadcast_to(g, (t, hv)) if g.ndim == 1 else g


def _fade(G):
    with np.errstate(over="ignore", invalid="ignore"):
        return np.tril(np.exp(np.tril(G[:, None] - G[None, :])))


def fwd(cu, q, k, v, g, h0=None, scale=1.0):
    (T, HV, d), N, group = v.shape, len(cu) - 1, v.shape[1] // q.shape[1]
    g = _log_decays(g, T, HV)
    o, ht = np.zeros_like(v), np.zeros((N, HV, d, d))
    for n in range(N):
        at = slice(cu[n], cu[n + 1])
        for h in range(HV):
            S0 = np.zeros((d, d)) if h0 is None else h0[n, h]
            if cu[n] == cu[n + 1]:
                ht[n, h] = S0
                continue
            Q, K, V, G = q[at, h // group], k[at, h // group], v[at, h], np.cumsum(g[at, h])
            o[at, h] = scale * (((Q @ K.T) * _fade(G)) @ V + np.exp(G)[:, None] * (Q @ S0))
            ht[n, h] = (K * np.exp(G[-1] - G)[:, None]).T @ V + np.exp(G[-1]) * S0
    return o, ht


def steps(cu, q, k, v, g, h0=None, scale=1.0):
    """(o, the state after every token [T, HV, d, d])"""
    (T, HV, d), group = v.shape, v.shape[1] // q.shape[1]
    g, head = _log_decays(g, T, HV), np.arange(HV) // group
    o, kept = np.zeros_like(v), np.zeros((T, HV, d, d))
    for n in range(len(cu) - 1):
        S = np.zeros((HV, d, d)) if h0 is None else h0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            S = np.exp(g[t])[:, None, None] * S + k[t, head][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hkv,hk->hv", S, q[t, head])
            kept[t] = S
    return o, kept


def bwd(cu, q, k, v, g, do, h0=None, dht=None, scale=1.0):
    (T, HV, d), N, group = v.shape, len(cu) - 1, v.shape[1] // q.shape[1]
    by_head, g = g.ndim == 1, _log_decays(g, T, HV)
    r = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), dg=np.zeros((T, HV)),
             dh0=np.zeros((N, HV, d, d)))
    for n in range(N):
        at = slice(cu[n], cu[n + 1])
        for h in range(HV):
            S0 = np.zeros((d, d)) if h0 is None else h0[n, h]
            D = np.zeros((d, d)) if dht is None else dht[n, h]
            if cu[n] == cu[n + 1]:
                r["dh0"][n, h] = D
                continue
            Q, K, V, dO, G = scale * q[at, h // group], k[at, h // group], v[at, h], do[at, h], np.cumsum(g[at, h])
            fade, up, down = _fade(G), np.exp(G)[:, None], np.exp(G[-1] - G)[:, None]
            A, P = (Q @ K.T) * fade, (dO @ V.T) * fade
            r["dq"][at, h // group] += scale * (P @ K + up * (dO @ S0.T))
            r["dk"][at, h // group] += P.T @ Q + down * (V @ D.T)
            r["dv"][at, h] = A.T @ dO + down * (K @ D)
            r["dh0"][n, h] = (Q * up).T @ dO + np.exp(G[-1]) * D
            M = A * (dO @ V.T)
            into = M.sum(1) + ((up * (Q @ S0)) * dO).sum(1)
            out = M.sum(0) + ((down * (K @ D)) * V).sum(1)
            dG = into - out
            dG[-1] += (((K * down).T @ V + np.exp(G[-1]) * S0) * D).sum()
            r["dg"][at, h] = np.cumsum(dG[::-1])[::-1]
    if by_head:
        r["dg"] = r["dg"].sum(0)
    return r


def dg_by_states(cu, q, k, v, g, do, h0=None, dht=None, scale=1.0):
    """The decays' gradient by its definition, dg_t = e^{g_t} <S_{t-1}, D_t>, with the states S token by token and their
    gradients D_t = e^{g_{t+1}} D_{t+1} + scale q_t do_t^T (D_T takes dht): for documents too long for a product of
    all tokens with all. Also [T, HV] |q_t| |dq_t| + |k_t| |dk_t|, of the row products that dg can be summed from, and
    |S_{t-1}| |D_t| e^{g_t}."""
    (T, HV, d), group = v.shape, v.shape[1] // q.shape[1]
    a, head = np.exp(_log_decays(g, T, HV))[..., None, None], np.arange(HV) // group
    q, k = q[:, head], k[:, head]
    dot = lambda x, y: np.einsum("hi,hi->h", x.reshape(HV, -1), y.reshape(HV, -1))  # noqa: E731 (no BLAS, no temporaries)
    norm = lambda x: np.sqrt(dot(x, x))  # noqa: E731
    dg, rows, states = np.zeros((T, HV)), np.zeros((T, HV)), np.zeros((T, HV))
    for n in range(len(cu) - 1):
        b, e = cu[n], cu[n + 1]
        S = np.zeros((e - b + 1, HV, d, d))
        if h0 is not None:
            S[0] = h0[n]
        for t in range(b, e):
            S[t - b + 1] = a[t] * S[t - b] + k[t][:, :, None] * v[t][:, None, :]
        D = np.zeros((HV, d, d)) if dht is None else dht[n].copy()
        for t in range(e - 1, b - 1, -1):
            D += scale * q[t][:, :, None] * do[t][:, None, :]
            dq, dk = scale * np.einsum("hkv,hv->hk", S[t - b + 1], do[t]), np.einsum("hkv,hv->hk", D, v[t])
            rows[t] = norm(q[t]) * norm(dq) + norm(k[t]) * norm(dk)
            D *= a[t]
            dg[t], states[t] = dot(S[t - b], D), norm(S[t - b]) * norm(D)
    return (dg.sum(0) if g.ndim == 1 else dg), rows, states
