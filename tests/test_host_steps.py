"""Host-side refusals of the serving steps and of the rotation (no GPU: a rejected call launches
nothing, and pointers stand for tensors without being read)."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G

PTR = [0x100000 * (i + 1) for i in range(16)]


def _cu(*lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def _refused(rc, fragment, code=G.GDN_EINVAL):
    msg = G.load_library().gdn_last_error().decode()
    assert rc == code and fragment in msg, (rc, msg)


def _recurrent(p, **over):
    names = ("q", "k", "v", "g", "beta", "cu", "slot_in", "slot_out", "slot_tok", "states", "o")
    a = dict(zip(names, PTR))
    if not p.st.cu_seqlens_host:
        a["cu"] = None
    a["slot_tok"] = None
    a.update(over)
    return G.load_library().gdn_recurrent(p.ref(), *[a[n] for n in names], None)


@pytest.mark.parametrize("field,value,fragment,code", [
    ("n_seqs", 0, "n_seqs", 1), ("h_qk", 0, "head counts", 1), ("h_v", 5, "multiple", 1), ("d", 96, "64 or 128", 2),
    ("dtype", 7, "dtype", 2), ("n_slots", 0, "n_slots", 1), ("reserved0", 1, "reserved0", 1),
    ("n_tokens", 5, "n_tokens", 1), ("q_stride", 8, "q_stride", 1), ("k_stride", 2 * 64 + 4, "aligned", 1),
    ("v_stride", -512, "v_stride", 1), ("v_stride", 1 << 25, "2^24", 1), ("h_v", 65538, "65536", 1)])
def test_recurrent_refuses_bad_problems(field, value, fragment, code):
    p = G.RecurrentProblem(3, 2, 4, 64, 8)
    setattr(p.st, field, value)
    _refused(_recurrent(p), fragment, code)


def test_recurrent_refuses_bad_lengths_and_pointers():
    _refused(_recurrent(G.RecurrentProblem(2, 2, 4, 64, 8, cu_seqlens_host=[0, 4, 3])), "decreases")
    _refused(_recurrent(G.RecurrentProblem(2, 2, 4, 64, 8, cu_seqlens_host=[1, 4, 5])), "must be 0")
    with pytest.raises(G.GdnError, match="cu_seqlens_host"):
        G.RecurrentProblem(3, 2, 4, 64, 8, cu_seqlens_host=[0, 4, 5])
    p, r = G.RecurrentProblem(3, 2, 4, 64, 8), G.RecurrentProblem(2, 2, 4, 64, 8, cu_seqlens_host=_cu(3, 2))
    for name in ("q", "k", "v", "g", "beta", "slot_in", "slot_out", "states", "o"):
        _refused(_recurrent(p, **{name: None}), name + " is NULL")
        _refused(_recurrent(r, **{name: PTR[0] + 4}), name + " is not 16-byte aligned")
    _refused(_recurrent(r, slot_tok=PTR[0] + 4), "slot_tok")
    _refused(_recurrent(p, cu=PTR[0]), "together")
    _refused(_recurrent(r, cu=None), "together")
    _refused(G.load_library().gdn_recurrent(None, *([None] * 12)), "NULL")


def _conv(p, **over):
    names = ("x", "weight", "bias", "cu", "slot_in", "slot_out", "slot_tok", "windows")
    a = dict(zip(names, PTR))
    a["cu"], a["slot_tok"] = None, None
    a["y"] = (ctypes.c_void_p * 4)(*PTR[8:12])
    a.update(over)
    return G.load_library().gdn_conv_step(p.ref(), *[a[n] for n in names], a["y"], None)


@pytest.mark.parametrize("field,value,fragment,code", [
    ("n_seqs", 0, "n_seqs", 1), ("width", 5, "width", 2), ("width", 0, "width", 2), ("channels", 32, "sum", 1),
    ("dtype", 3, "dtype", 2), ("n_groups", 5, "n_groups", 1), ("n_slots", 0, "n_slots", 1), ("n_tokens", 4, "n_tokens", 1),
    ("reserved0", 2, "reserved0", 1), ("x_stride", 16, "x_stride", 1), ("x_stride", 28, "aligned", 1)])
def test_conv_step_refuses_bad_problems(field, value, fragment, code):
    p = G.ConvStepProblem(3, [16, 8], 8)
    setattr(p.st, field, value)
    _refused(_conv(p), fragment, code)


def test_conv_step_refuses_bad_pointers():
    p = G.ConvStepProblem(3, [16, 8], 8)
    for name in ("x", "weight", "slot_in", "slot_out", "windows"):
        _refused(_conv(p, **{name: None}), name + " is NULL")
        _refused(_conv(p, **{name: PTR[0] + 2}), name + " is not 16-byte aligned")
    _refused(_conv(p, bias=PTR[0] + 4), "bias")
    _refused(_conv(p, cu=PTR[0]), "together")
    _refused(_conv(p, y=None), "NULL")
    _refused(_conv(p, y=(ctypes.c_void_p * 4)(PTR[0], None)), "y[g] is NULL")
    _refused(_conv(G.ConvStepProblem(3, [16, 12], 8)), "multiple of 8")
    _refused(G.load_library().gdn_conv_step(None, *([None] * 10)), "NULL")


def _rope(p, back=False, **over):
    names = ("q", "k", "positions", "freqs", "q_weight", "k_weight") + (
        ("dq_out", "dk_out", "dq", "dk", "dq_weight", "dk_weight", "workspace", "bytes") if back else ("q_out", "k_out"))
    a = dict(zip(names, PTR))
    if back:
        a["bytes"] = 1 << 30
    a.update(over)
    f = G.load_library().gdn_qk_rope_bwd if back else G.load_library().gdn_qk_rope_fwd
    return f(p.ref(), *[a[n] for n in names], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("field,value,fragment,code", [
    ("n_tokens", -1, "n_tokens", 1), ("n_tokens", 1 << 31, "tokens", 1), ("h_q", 0, "h_q", 1), ("h_k", -1, "h_k", 1),
    ("h_q", 1 << 15, "h_q", 1), ("d", 0, "multiple of 8", 2), ("d", 264, "multiple of 8", 2), ("d", 100, "multiple of 8", 2),
    ("dtype", 2, "dtype", 2), ("norm", 3, "norm", 1), ("norm", 0, "needs a norm", 1), ("rotary_dim", 72, "rotary_dim", 1),
    ("rotary_dim", 12, "rotary_dim", 1), ("rotary_dim", -8, "rotary_dim", 1), ("eps", -1.0, "eps", 1),
    ("eps", float("nan"), "eps", 1), ("magnitude", float("inf"), "magnitude", 1), ("reserved0", 1, "reserved0", 1),
    ("q_stride", 64, "q_stride", 1), ("k_stride", 132, "aligned", 1), ("qo_stride", -8, "qo_stride", 1),
    ("ko_stride", 130, "aligned", 1), ("q_stride", 1 << 28, "2^27", 1)])
def test_rope_refuses_bad_problems(field, value, fragment, code, back):
    p = G.QkRopeProblem(10, 2, 2, 64)
    setattr(p.st, field, value)
    _refused(_rope(p, back), fragment, code)


def test_rope_refuses_bad_pointers():
    p = G.QkRopeProblem(10, 2, 2, 64)
    for back, names in ((False, ("q", "k", "positions", "freqs", "q_out", "k_out")),
                        (True, ("q", "k", "positions", "freqs", "dq_out", "dk_out", "dq", "dk", "workspace"))):
        for name in names:
            _refused(_rope(p, back, **{name: None}), name + " is NULL")
            _refused(_rope(p, back, **{name: PTR[0] + 8}), name + " is not 16-byte aligned")
    _refused(_rope(p, True, dq_weight=None), "together")
    _refused(_rope(p, True, k_weight=None), "together")
    _refused(_rope(p, True, bytes=G.gdn_qk_rope_workspace_bytes(p) - 1), "workspace", G.GDN_EWORKSPACE)
    _refused(_rope(G.QkRopeProblem(10, 2, 0, 64)), "h_k = 0")
    _refused(G.load_library().gdn_qk_rope_fwd(None, *([None] * 9)), "NULL")
    with pytest.raises(G.GdnError, match="unknown norm"):
        G.QkRopeProblem(10, 2, 2, 64, norm="layer")
    bad = G.QkRopeProblem(10, 2, 2, 65)
    with pytest.raises(G.GdnError, match="multiple of 8"):
        G.gdn_qk_rope_workspace_bytes(bad)


def test_problems_of_no_tokens_need_no_tensors():
    """Zero tokens: nothing is launched, and pointers may be NULL."""
    lib = G.load_library()
    p = G.QkRopeProblem(0, 2, 2, 64)
    assert lib.gdn_qk_rope_fwd(p.ref(), None, None, None, PTR[0], None, None, None, None, None) == G.GDN_OK
    assert G.gdn_qk_rope_workspace_bytes(p) > 0


@pytest.mark.parametrize("make", [lambda t: G.RecurrentProblem(3, 2, 4, 64, 8, dtype=t),
                                  lambda t: G.ConvStepProblem(3, [16], 8, dtype=t),
                                  lambda t: G.QkRopeProblem(3, 2, 2, 64, dtype=t)])
def test_other_types_are_refused(make):
    with pytest.raises(G.GdnError, match="unsupported dtype"):
        make(torch.float16)


def test_native_binding_checks_tensors():
    """The native marshalling is built, and refuses what is not a GPU tensor before anything else."""
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(G.GdnError, match="expected a GPU"):
        G.gdn_recurrent(G.RecurrentProblem(3, 2, 2, 64, 8), x, x, x, x, x, x, x, x)
    with pytest.raises(G.GdnError, match="not a tensor"):
        G.gdn_qk_rope_fwd(G.QkRopeProblem(3, 2, 2, 64), None, x, x, x)
    with pytest.raises(G.GdnError, match="expected a GPU"):
        G.gdn_conv_step(G.ConvStepProblem(3, [128], 8), x, x, None, x, x, x)


@pytest.mark.parametrize("tokens", [0x7ff00001, 2 ** 31 - 1])
def test_counts_near_the_end_of_32_bits_are_refused(tokens):
    """The kernels step over tokens and sequences in 32 bits, some beyond the last one: the steps' limit is
    the rotation's."""
    _refused(_conv(G.ConvStepProblem(1, [8], 8, cu_seqlens_host=[0, tokens]), cu=PTR[0]), "too many")
    _refused(_conv(G.ConvStepProblem(tokens, [8], 8)), "too many")
    _refused(_recurrent(G.RecurrentProblem(1, 1, 1, 64, 8, cu_seqlens_host=[0, tokens])), "too many")
    _refused(_recurrent(G.RecurrentProblem(tokens, 1, 1, 64, 8)), "too many")
