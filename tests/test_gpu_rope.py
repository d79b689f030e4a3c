"""GPU tests of the norms of the q and k heads with the position rotation, forward and backward,
against the FP64 oracle."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
from oracle import rope_oracle
from step_util import check, f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
K = 64  # a row's sum of squares (8 in a lane, 5 levels across), root, divide, angle polynomials, products


def make(T, hq, hk, d, dtype=torch.bfloat16, norm="rms", rotary=None, interleaved=False, packed=False, longest=4096,
         weights=True, seed=5, eps=1e-6, **scaling):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    rotary = d if rotary is None else rotary

    def pair():
        if not packed:
            return normal(T, hq, d).to(dtype), normal(T, hk, d).to(dtype) if hk else None
        x = normal(T, (hq + hk) * d + 24).to(dtype)
        return x[:, :hq * d].view(T, hq, d), x[:, hq * d:(hq + hk) * d].view(T, hk, d) if hk else None

    s = dict(T=T, hq=hq, hk=hk, d=d, norm=norm, rotary=rotary, interleaved=interleaved, eps=eps)
    s["q"], s["k"] = pair()
    s["dyq"], s["dyk"] = pair()
    use = weights and norm != "none"
    s["wq"] = 1 + 0.1 * normal(d) if use else None
    s["wk"] = 1 + 0.1 * normal(d) if use and hk else None
    s["pos"] = torch.randint(0, longest, (T,), generator=gen, device=DEV, dtype=torch.int32)
    s["f"], s["m"] = rope_oracle.frequencies(rotary, **scaling) if rotary else (np.zeros(0), 1.0)
    s["freqs"] = G.gdn_rope_frequencies(rotary, **scaling)[0].to(DEV) if rotary else None
    s["p"] = G.QkRopeProblem(T, hq, hk, d, dtype=dtype, norm=norm, rotary_dim=rotary, interleaved=interleaved, eps=eps,
                             magnitude=s["m"])
    return s


def args(s):
    return s["p"], s["q"], s["k"], s["pos"] if s["rotary"] else None, s["freqs"]


def oracle_kw(s):
    return dict(norm=s["norm"], rotary_dim=s["rotary"], interleaved=s["interleaved"], eps=s["eps"], m=s["m"])


CASES = {
    "one_token": dict(T=1, hq=1, hk=1, d=128),
    "odd_tokens": dict(T=33, hq=5, hk=3, d=128, rotary=64),
    "interleaved": dict(T=70, hq=4, hk=2, d=64, interleaved=True, norm="l2"),
    "rotate_alone": dict(T=19, hq=3, hk=1, d=128, norm="none", interleaved=True, packed=True),
    "rotate_alone_half": dict(T=19, hq=3, hk=1, d=64, norm="none", rotary=16, dtype=torch.float32),
    "norm_alone": dict(T=20, hq=2, hk=2, d=128, rotary=0),
    "wide_256": dict(T=21, hq=2, hk=1, d=256, rotary=128, packed=True),
    "width_96_f32": dict(T=130, hq=3, hk=2, d=96, rotary=24, interleaved=True, dtype=torch.float32),
    "width_80": dict(T=9, hq=2, hk=2, d=80, rotary=40),
    "width_8": dict(T=65, hq=2, hk=1, d=8, dtype=torch.float32),
    "width_200_f32": dict(T=17, hq=1, hk=1, d=200, rotary=72, dtype=torch.float32, packed=True, interleaved=True),
    "no_k": dict(T=12, hq=4, hk=0, d=128, weights=False),
    "l2_weighted_f32": dict(T=40, hq=2, hk=2, d=64, norm="l2", dtype=torch.float32),
    "scaled_far": dict(T=50, hq=2, hk=1, d=128, longest=1 << 20, scaling="yarn", factor=4.0, original_length=32768,
                       dtype=torch.float32),
    "bands_far": dict(T=50, hq=2, hk=1, d=64, longest=1 << 20, scaling="bands", factor=8.0, original_length=8192,
                      fast=4.0, interleaved=True),
    "many_tokens": dict(T=6001, hq=3, hk=2, d=64, rotary=32),
    "many_rows_f32": dict(T=2500, hq=16, hk=4, d=128, dtype=torch.float32),
}


@pytest.mark.parametrize("name", CASES)
def test_qk_rope(name):
    s = make(**CASES[name])
    print("qk_rope", name, flush=True)
    q, k = G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"], k_weight=s["wk"])
    g = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    torch.cuda.synchronize()
    pos = s["pos"].cpu().numpy()
    for name, x, dy, w, y, dx, dw in (("q", s["q"], s["dyq"], s["wq"], q, g["dq"], g["dq_weight"]),
                                      ("k", s["k"], s["dyk"], s["wk"], k, g["dk"], g["dk_weight"])):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        check(name, y, rope_oracle.fwd(f64(x), pos, s["f"], f64(w), **oracle_kw(s)), K)
        dx_ref, dw_ref = rope_oracle.bwd(f64(x), f64(dy), pos, s["f"], f64(w), **oracle_kw(s))
        check("d" + name, dx, dx_ref, K)
        if w is None:
            assert dw is None
        else:  # sums over T * h rows of size sqrt(T h): a row's roundings, then those of the partial sums
            rows = s["T"] * x.shape[1]
            size = np.sqrt(rows) * np.max(np.abs(f64(dy))) * 4 / max(np.max(np.abs(dw_ref)), 1e-30)
            check("dw_" + name, dw, dw_ref, K * max(1.0, size))


def test_positions_at_the_ends_of_int32():
    """The angle is exact at any position of either sign: the oracle's angle by whole-number
    arithmetic on the frequencies' 64-bit fractions."""
    s = make(8, 1, 1, 64, dtype=torch.float32, norm="none")
    pos = [0, -1, 1, 2 ** 31 - 1, -2 ** 31, 1 << 24, (1 << 24) + 1, -123456789]
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
    q, k = G.gdn_qk_rope_fwd(*args(s))
    torch.cuda.synchronize()
    turns = [int(x) % 2 ** 64 for x in s["freqs"].tolist()]
    angle = np.array([[(p * f % 2 ** 64) / 2.0 ** 64 * 2 * np.pi for f in turns] for p in pos])
    for got, x in ((q, f64(s["q"])), (k, f64(s["k"]))):
        z = (x[..., :32] + 1j * x[..., 32:]) * np.exp(1j * angle)[:, None]
        check("y", got, np.concatenate([z.real, z.imag], -1), K)


def test_gradient_against_differences():
    """<gradient, direction> against central differences of the FP64 forward: step 1e-4 leaves a
    relative error of about 1e-8, the f32 gradient about 1e-6 of the summed sizes."""
    s = make(11, 3, 2, 64, dtype=torch.float32, rotary=32, eps=1e-3)
    g = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    torch.cuda.synchronize()
    rng = np.random.default_rng(1)
    pos = s["pos"].cpu().numpy()
    for x, w, dy, dx, dw in ((s["q"], s["wq"], s["dyq"], g["dq"], g["dq_weight"]),
                             (s["k"], s["wk"], s["dyk"], g["dk"], g["dk_weight"])):
        x, w, dy = f64(x), f64(w), f64(dy)
        loss = lambda x_, w_: float(np.sum(dy * rope_oracle.fwd(x_, pos, s["f"], w_, **oracle_kw(s))))
        e, ew, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-4
        fd = (loss(x + h * e, w) - loss(x - h * e, w)) / (2 * h)
        assert abs(fd - np.sum(f64(dx) * e)) < 1e-5 * np.sum(np.abs(f64(dx) * e))
        fd = (loss(x, w + h * ew) - loss(x, w - h * ew)) / (2 * h)
        assert abs(fd - np.sum(f64(dw) * ew)) < 1e-5 * np.sum(np.abs(f64(dw) * ew))


def test_in_place_and_into_parts_of_a_row():
    s = make(37, 4, 2, 128, rotary=64)
    q, k = G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"], k_weight=s["wk"])
    g = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    row = torch.full((37, 7 * 128), 3.0, dtype=torch.bfloat16, device=DEV)
    parts = row[:, :512].view(37, 4, 128), row[:, 512:768].view(37, 2, 128)
    G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"], k_weight=s["wk"], q_out=parts[0], k_out=parts[1])
    assert torch.equal(parts[0], q) and torch.equal(parts[1], k) and (row[:, 768:] == 3).all()
    row.fill_(3.0)
    g2 = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"],
                           grads=dict(dq=parts[0], dk=parts[1]))
    assert torch.equal(parts[0], g["dq"]) and torch.equal(parts[1], g["dk"]) and (row[:, 768:] == 3).all()
    assert torch.equal(g2["dq_weight"], g["dq_weight"])
    g3 = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"],
                           grads=dict(dq=s["dyq"], dk=s["dyk"]))
    assert torch.equal(g3["dq"], g["dq"]) and torch.equal(g3["dk"], g["dk"])
    G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"], k_weight=s["wk"], q_out=s["q"], k_out=s["k"])
    assert torch.equal(s["q"], q) and torch.equal(s["k"], k)


def test_weight_gradients_are_reproducible():
    s = make(5000, 4, 4, 128)
    a = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    b = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_one_weight_only_and_no_tokens():
    s = make(30, 2, 2, 64, dtype=torch.float32)
    q, k = G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"])
    g = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], k_weight=s["wk"])
    pos = s["pos"].cpu().numpy()
    check("k", k, rope_oracle.fwd(f64(s["k"]), pos, s["f"], None, **oracle_kw(s)), K)
    dx, dw = rope_oracle.bwd(f64(s["k"]), f64(s["dyk"]), pos, s["f"], f64(s["wk"]), **oracle_kw(s))
    check("dk", g["dk"], dx, K)
    check("dk_weight", g["dk_weight"], dw, K * 60)
    assert g["dq_weight"] is None
    s = make(0, 2, 2, 64)
    q, k = G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"], k_weight=s["wk"])
    g = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    assert q.shape == (0, 2, 64) and not g["dq_weight"].any() and not g["dk_weight"].any()


def test_rows_of_zeros_infinities_and_nan():
    """A zero row stays zero under the norm's eps, gradients finite; NaN and infinities stay in their row."""
    s = make(6, 2, 2, 64, dtype=torch.float32)
    s["q"][1], s["q"][2, 0, 5], s["k"][3, 1, 7] = 0, float("nan"), float("inf")
    q, k = G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"], k_weight=s["wk"])
    g = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    assert not q[1].any() and torch.isfinite(g["dq"][1]).all()
    keep_q = [(t, h) for t in range(6) for h in range(2) if (t, h) != (2, 0)]
    keep_k = [(t, h) for t in range(6) for h in range(2) if (t, h) != (3, 1)]
    assert all(torch.isfinite(q[x]).all() and torch.isfinite(g["dq"][x]).all() for x in keep_q)
    assert all(torch.isfinite(k[x]).all() and torch.isfinite(g["dk"][x]).all() for x in keep_k)
    assert torch.isnan(q[2, 0]).all() and torch.isnan(k[3, 1]).any()


def test_rows_past_32_bit_offsets():
    T, hq, hk, d = (1 << 15) + 3, 520, 1, 128  # 2^31 values of q pass before the last tokens
    s = make(64, hq, hk, d, norm="l2")
    q = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(T, hk, d, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    q[-64:], k[-64:], pos[-64:] = s["q"], s["k"], s["pos"]
    p = G.QkRopeProblem(T, hq, hk, d, norm="l2")
    a, b = G.gdn_qk_rope_fwd(p, q, k, pos, s["freqs"])
    want = G.gdn_qk_rope_fwd(*args(s))
    assert torch.equal(a[-64:], want[0]) and torch.equal(b[-64:], want[1]) and not a[:-64].any()
    g = G.gdn_qk_rope_bwd(p, q, k, pos, s["freqs"], q, k)
    want = G.gdn_qk_rope_bwd(*args(s), s["q"], s["k"])
    assert torch.equal(g["dq"][-64:], want["dq"]) and torch.equal(g["dk"][-64:], want["dk"])


def test_on_a_stream_of_its_own():
    s = make(300, 4, 2, 128)
    want = G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"], k_weight=s["wk"])
    grads = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"], k_weight=s["wk"], stream=side)
    g2 = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"], stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert all(torch.equal(grads[n], g2[n]) for n in grads)


def test_binding_refuses_wrong_tensors():
    s = make(4, 2, 2, 64)
    p, q, k, pos, f = args(s)
    for a, kw, fragment in (
            ((p, q[:3], k, pos, f), {}, "shape"), ((p, q, k.float(), pos, f), {}, "type"),
            ((p, q, k, pos.long(), f), {}, "type"), ((p, q, k, pos, f[:-1]), {}, "shape"),
            ((p, q, k, None, f), {}, "positions is NULL"), ((p, q, k, pos, None), {}, "freqs is NULL"),
            ((p, q, None, pos, f), {}, "k is NULL"),
            ((p, q.transpose(0, 1).contiguous().transpose(0, 1), k, pos, f), {}, "contiguous"),
            ((p, q, k, pos, f), dict(q_weight=s["wq"].bfloat16()), "type"),
            ((p, q, k, pos, f), dict(q_weight=s["wq"].cpu()), "is on")):
        with pytest.raises(G.GdnError, match=fragment):
            G.gdn_qk_rope_fwd(*a, **kw)
    x = torch.zeros(4, 2 * 64 + 4, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(G.GdnError, match="aligned"):
        G.gdn_qk_rope_fwd(p, x[:, :128].view(4, 2, 64), k, pos, f)
    with pytest.raises(G.GdnError, match="workspace"):
        G.gdn_qk_rope_bwd(p, q, k, pos, f, s["dyq"], s["dyk"], q_weight=s["wq"],
                          workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(G.GdnError, match="needs a norm"):
        G.gdn_qk_rope_fwd(G.QkRopeProblem(4, 2, 2, 64, norm="none"), q, k, pos, f, q_weight=s["wq"])


def test_bad_problems_are_refused_before_anything_is_allocated():
    s = make(4, 2, 1, 64)
    s["p"].st.h_k = -1
    with pytest.raises(G.GdnError):
        G.gdn_qk_rope_fwd(*args(s))


def test_no_tokens_give_empty_gradients_of_both():
    s = make(0, 2, 1, 64)
    g = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    assert g["dq"].shape == (0, 2, 64) and g["dk"].shape == (0, 1, 64)
    assert not g["dq_weight"].any() and not g["dk_weight"].any()


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("size", [1e-20, 1e-16, 1e-6, 1e15])
def test_rows_of_any_size_without_eps(norm, size):
    """eps = 0: the norm does not depend on a row's size, also where the mean square is subnormal (each
    product then is off by up to 2^-150 of 1e-40, the root by 4e-6) or the root's cube overflows."""
    s = make(20, 2, 1, 64, dtype=torch.float32, norm=norm, eps=0.0)
    for x in ("q", "k"):
        s[x].mul_(size).add_(torch.sign(s[x]) * size)  # no value far below the others
    q, k = G.gdn_qk_rope_fwd(*args(s), q_weight=s["wq"], k_weight=s["wk"])
    g = G.gdn_qk_rope_bwd(*args(s), s["dyq"], s["dyk"], q_weight=s["wq"], k_weight=s["wk"])
    pos = s["pos"].cpu().numpy()
    for x, y, w, dy, dx, dw in (("q", q, "wq", "dyq", g["dq"], g["dq_weight"]), ("k", k, "wk", "dyk", g["dk"], g["dk_weight"])):
        more = 64 if size < 1e-19 else 0  # 64 2^-24 = 3.8e-6
        check("y", y, rope_oracle.fwd(f64(s[x]), pos, s["f"], f64(s[w]), **oracle_kw(s)), K + more)
        dx_ref, dw_ref = rope_oracle.bwd(f64(s[x]), f64(s[dy]), pos, s["f"], f64(s[w]), **oracle_kw(s))
        check("dx", dx, dx_ref, K + 2 * more)
        check("dw", dw, dw_ref, 40 * (K + more))
