"""GPU tests of the conv front-end's serving step on cached windows against the FP64 oracle of the
whole convolution: a sequence's window and tokens are one document of it."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
from oracle import conv_oracle
from step_util import check, f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
K = 40  # 4 products, a bias, the sigmoid's exponential, reciprocal and product


def make(lengths, groups, width=4, dtype=torch.bfloat16, bias=True, silu=True, keep=False, fresh=(), packed=False,
         seed=9):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    N, T, C = len(lengths), sum(lengths), sum(groups)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    slots = N + (T if keep else 0) + 2
    order = torch.randperm(slots, generator=gen, device=DEV).to(torch.int32)
    x = normal(T, C + (16 if packed else 0)).to(dtype)[:, :C]
    s = dict(cu_host=cu, cu=torch.from_numpy(cu).to(DEV), x=x, weight=normal(C, width) / width ** 0.5,
             bias=0.1 * normal(C) if bias else None, windows=normal(slots, width - 1, C).to(dtype),
             slot_in=order[:N].clone(), slot_out=order[:N].clone(), slot_tok=order[N:N + T].clone() if keep else None,
             groups=groups, width=width, silu=silu, slots=slots)
    for n in fresh:
        s["slot_in"][n] = -1
    return s


def reference(s):
    w1 = s["width"] - 1
    x, win, weight, bias = f64(s["x"]), f64(s["windows"]), f64(s["weight"]), f64(s["bias"])
    y, out = np.zeros_like(x), win.copy()
    si, so = s["slot_in"].tolist(), s["slot_out"].tolist()
    st = s["slot_tok"].tolist() if s["slot_tok"] is not None else None
    for n in range(len(si)):
        a, e = int(s["cu_host"][n]), int(s["cu_host"][n + 1])
        line = np.concatenate([win[si[n]] if si[n] >= 0 else np.zeros_like(win[0]), x[a:e]])
        cu = np.array([0, line.shape[0]])
        y[a:e] = conv_oracle.conv_fwd(cu, line, weight, bias, silu=s["silu"])[0][w1:]
        for t in range(a, e):
            if st is not None and st[t] >= 0:
                out[st[t]] = line[t - a + 1:t - a + 1 + w1]
        if so[n] >= 0:
            out[so[n]] = line[line.shape[0] - w1:]
    return y, out


def run(s, **kw):
    one = bool(np.all(np.diff(s["cu_host"]) == 1))
    p = G.ConvStepProblem(len(s["cu_host"]) - 1, s["groups"], s["slots"], cu_seqlens_host=None if one else s["cu_host"],
                          width=s["width"], dtype=s["x"].dtype, silu=s["silu"])
    print("conv_step N=%d T=%d C=%d W=%d" % (len(s["cu_host"]) - 1, s["x"].shape[0], s["x"].shape[1], s["width"]), flush=True)
    win = s["windows"].clone()
    y = G.gdn_conv_step(p, s["x"], s["weight"], s["bias"], win if s["width"] > 1 else None, s["slot_in"], s["slot_out"],
                        slot_tok=s["slot_tok"], cu_seqlens=None if one else s["cu"], **kw)
    torch.cuda.synchronize()
    return torch.cat(y, 1), win


CASES = {
    "one": dict(lengths=[1], groups=[2048, 2048, 6144]),
    "decode_300": dict(lengths=[1] * 300, groups=[64, 64, 192], fresh=(7,)),
    "decode_packed_f32": dict(lengths=[1] * 5, groups=[8, 16, 8, 24], packed=True, dtype=torch.float32),
    "ragged": dict(lengths=[0, 1, 2, 3, 4, 9, 0], groups=[520, 24], fresh=(0, 1, 4)),
    "drafts": dict(lengths=[8, 1, 0, 5], groups=[256, 8, 1032], keep=True, bias=False),
    "drafts_w3_f32": dict(lengths=[2, 6], groups=[1032], width=3, keep=True, dtype=torch.float32, silu=False),
    "w2": dict(lengths=[1, 1, 1], groups=[40], width=2),
    "w1": dict(lengths=[2, 1, 0], groups=[40], width=1, dtype=torch.float32),
    "long_run": dict(lengths=[100, 1], groups=[2064]),
}


@pytest.mark.parametrize("name", CASES)
def test_conv_step(name):
    s = make(**CASES[name])
    y, win = run(s)
    y_ref, win_ref = reference(s)
    check("y", y, y_ref, K)
    assert np.array_equal(f64(win), win_ref)  # windows hold inputs as they came


def test_steps_equal_the_whole_convolution():
    """A document in one call of the front-end and token by token on its window: the same taps in the
    same order, and a sigmoid that may differ in its last bits."""
    s = make([9], [64, 64], dtype=torch.float32, fresh=(0,))
    cp = G.ConvProblem(s["cu_host"], s["groups"], dtype=torch.float32)
    want = torch.cat(G.gdn_conv_fwd(cp, s["x"], s["weight"], s["bias"], s["cu"]), 1)
    p = G.ConvStepProblem(1, s["groups"], s["slots"], dtype=torch.float32)
    win, rows = s["windows"], []
    for t in range(9):
        y = G.gdn_conv_step(p, s["x"][t:t + 1], s["weight"], s["bias"], win, s["slot_in"] if t == 0 else s["slot_out"],
                            s["slot_out"])
        rows.append(torch.cat(y, 1))
    torch.cuda.synchronize()
    check("y", torch.cat(rows), f64(want), K)
    assert torch.equal(win[s["slot_out"].long()][0], s["x"][-3:])


@pytest.mark.parametrize("what", ["slot_in", "slot_out", "slot_tok", "cu"])
def test_device_arrays_out_of_range_are_refused_on_the_device(what):
    s = make([2, 3, 4], [16, 8], keep=True)
    y_ref, win_ref = reference(s)
    rows, lost = range(2, 5), s["slot_tok"][2:5].tolist() + [s["slot_out"][1].item()]
    if what == "slot_tok":
        rows, lost = [3], [s["slot_tok"][3].item()]
        s["slot_tok"][3] = -7
    elif what == "cu":
        s["cu"] = torch.tensor([0, 2, 5, 10], dtype=torch.int32, device=DEV)
        rows, lost = range(5, 9), s["slot_tok"][5:9].tolist() + [s["slot_out"][2].item()]
    else:
        s[what][1] = s["slots"] if what == "slot_in" else -2
    before = f64(s["windows"])
    y, win = run(s)
    rows = list(rows)
    assert torch.isnan(y[rows].float()).all()
    good = [t for t in range(9) if t not in rows]
    check("y", y[good], y_ref[good], K)
    win_ref[lost] = before[lost]
    assert np.array_equal(f64(win), win_ref)


def test_values_at_the_ends_of_the_sigmoid():
    """Large pre-activations of either sign, infinities and NaN stay in their channel."""
    s = make([1, 1], [16], dtype=torch.float32, bias=False)
    s["weight"][:] = 0
    s["weight"][:, 3] = 1
    s["x"][0] = torch.tensor([-1e4, -200, -88, -20, 0, 20, 88, 200, 1e4, float("nan"), float("inf"), 1, 2, 3, 4, 5])
    s["windows"][:] = 0
    y, _ = run(s)
    x = f64(s["x"][0])
    with np.errstate(over="ignore", invalid="ignore"):
        ref = x / (1 + np.exp(-x))
    got = f64(y[0])
    assert np.isnan(got[9]) and got[10] == np.inf
    fine = [i for i in range(16) if i not in (9, 10)]
    np.testing.assert_allclose(got[fine], ref[fine], rtol=1e-5, atol=1e-30)


def test_on_a_stream_of_its_own():
    s = make([1] * 6, [64, 32])
    want = run(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(s, stream=side)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("T", [3, 4000], ids=["short", "long"])
def test_outputs_made_by_the_call_do_not_meet(T):
    """A short call's outputs are parts of one allocation, a long one's are not."""
    s = make([1] * T, [24, 8, 136])
    p = G.ConvStepProblem(T, s["groups"], s["slots"])
    call = lambda **kw: G.gdn_conv_step(p, s["x"], s["weight"], s["bias"], s["windows"].clone(), s["slot_in"], s["slot_out"], **kw)
    given = [torch.empty(T, c, dtype=torch.bfloat16, device=DEV) for c in s["groups"]]
    call(outs=given)
    made = call()
    for y, z in zip(made, given):
        assert y.shape == z.shape and y.dtype == z.dtype and y.is_contiguous() and y.data_ptr() % 512 == 0
        assert torch.equal(y, z)
    for i, y in enumerate(made):
        y.fill_(float("nan"))
        for x, z in list(zip(made, given))[i + 1:]:
            assert torch.equal(x, z)
    assert all(torch.isnan(y).all() for y in made)
    assert len({y.untyped_storage().data_ptr() for y in made}) == (1 if T == 3 else 3)
    kept = call()[1]  # the others are released: the part keeps its memory
    fill = [torch.full((1 << 16,), 7.0, device=DEV) for _ in range(4)]
    assert torch.equal(kept, given[1]) and len(fill) == 4


def test_binding_refuses_wrong_tensors():
    s = make([1, 1], [16, 8])
    p = G.ConvStepProblem(2, s["groups"], s["slots"])
    good = dict(x=s["x"], weight=s["weight"], bias=s["bias"], windows=s["windows"], slot_in=s["slot_in"],
                slot_out=s["slot_out"])
    for name, bad, fragment in (
            ("x", s["x"].float(), "type"), ("weight", s["weight"].t(), "shape"), ("windows", None, "windows is NULL"),
            ("windows", s["windows"][:, :2].contiguous(), "shape"), ("bias", s["bias"][:8], "shape"),
            ("slot_in", s["slot_in"].long(), "type"), ("x", s["x"].t().contiguous().t(), "contiguous")):
        with pytest.raises(G.GdnError, match=fragment):
            G.gdn_conv_step(p, **{**good, name: bad})
    with pytest.raises(G.GdnError, match="outs has"):
        G.gdn_conv_step(p, **good, outs=[s["x"]])
    with pytest.raises(G.GdnError, match="n_groups"):
        G.ConvStepProblem(2, [8] * 5, 4)


def test_negative_groups_are_refused_before_anything_is_allocated():
    s = make([1, 1], [16, 8])
    p = G.ConvStepProblem(2, [32, -8], s["slots"])
    with pytest.raises(G.GdnError, match="channels"):
        G.gdn_conv_step(p, s["x"], s["weight"], s["bias"], s["windows"], s["slot_in"], s["slot_out"])


# a call for each kernel and each way through it: one or two sequences a lane, runs
KERNELS = {
    "one_sequence_a_lane": dict(lengths=[1] * 3, groups=[16, 8]),
    "two_sequences_a_lane": dict(lengths=[1] * 1025, groups=[16, 8]),
    "runs": dict(lengths=[2, 9, 3, 5], groups=[16, 8], dtype=torch.float32),
}


@pytest.mark.parametrize("name,what", [(x, y) for x in KERNELS for y in ("slot_in", "slot_out", "start", "end")
                                       if y.startswith("slot") or max(KERNELS[x]["lengths"]) > 1])
def test_every_kernel_refuses_what_is_out_of_range_on_the_device(name, what):
    s = make(**KERNELS[name])
    N = len(s["slot_in"])
    n = dict(slot_in=N - 1, slot_out=1, start=0, end=N - 1)[what]
    rows = slice(int(s["cu_host"][n]), int(s["cu_host"][n + 1]))
    y_ref, win_ref = reference(s)
    slot = s["slot_out"][n].item()
    win_ref[slot] = f64(s["windows"][slot])
    if what == "slot_in":
        s["slot_in"][n] = s["slots"]
    elif what == "slot_out":
        s["slot_out"][n] = -2
    else:
        s["cu"][n if what == "start" else N] += -1 if what == "start" else 1
    y, win = run(s)
    assert torch.isnan(y[rows].float()).all()
    good = torch.ones(y.shape[0], dtype=torch.bool)
    good[rows] = False
    check("y", y[good.to(DEV)], y_ref[good.numpy()], K)
    assert np.array_equal(f64(win), win_ref)


@pytest.mark.parametrize("name", KERNELS)
def test_every_kernel_leaves_windows_nowhere_and_shares_starts(name):
    s = make(**KERNELS[name])
    free = [x for x in range(s["slots"]) if x not in s["slot_in"].tolist()]
    s["slot_in"][1::2] = free[0]
    s["slot_out"][::3] = -1
    y, win = run(s)
    y_ref, win_ref = reference(s)
    check("y", y, y_ref, K)
    assert np.array_equal(f64(win), win_ref)


def test_rows_of_no_sequence_keep_their_values():
    s = make([2, 9, 3, 5], [16, 8])
    s["cu"][-1] = 14
    outs = [torch.full((19, c), 7.0, dtype=torch.bfloat16, device=DEV) for c in s["groups"]]
    y, _ = run(s, outs=outs)
    s["cu_host"][-1] = 14
    y_ref, _ = reference(s)
    assert (y[14:] == 7).all()
    check("y", y[:14], y_ref[:14], K)
