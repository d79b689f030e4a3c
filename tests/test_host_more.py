"""Host checks of linear attention, the RMS norm and a step's maps: sizes, refusals before any launch (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G

PTR = ctypes.c_void_p(4096)  # never read: every call here is refused first


def refused(code, text, rc):
    assert rc == code, rc
    assert text in G.load_library().gdn_last_error().decode()


def linear(lengths=(5, 0, 70), H=2, HV=4, d=64, **kw):
    return G.LinearProblem(np.concatenate([[0], np.cumsum(lengths)]), H, HV, d, **kw)


def lin_fwd(p, q=PTR, g=PTR, h0=None, ht=None, ws=PTR, nbytes=1 << 40):
    return G.load_library().gdn_linear_fwd(p.ref() if p else None, q, PTR, PTR, g, PTR, h0, PTR, ht, ws, nbytes, None)


def lin_bwd(p, dO=PTR, dg=PTR, h0=None, dh0=None, ws=PTR, nbytes=1 << 40):
    return G.load_library().gdn_linear_bwd(p.ref(), PTR, PTR, PTR, PTR, PTR, h0, dO, None, PTR, PTR, PTR, dg, dh0, ws, nbytes, None)


@pytest.mark.parametrize("field,value,code,text", [
    ("n_seqs", 0, 1, "n_seqs"), ("n_seqs", 65536, 1, "n_seqs"), ("h_v", 3, 1, "multiple"), ("h_qk", 0, 1, "head counts"),
    ("d", 96, 2, "64 or 128"), ("dtype", 2, 2, "dtype"), ("decay", 2, 1, "decay"), ("scale", float("nan"), 1, "scale"),
    ("scale", float("inf"), 1, "scale"), ("reserved0", 1, 1, "reserved0"), ("n_tokens", 74, 1, "n_tokens"),
    ("h_v", 2 * 65536, 1, "2^22"), ("h_v", 65536, 1, "65535"), ("q_stride", 120, 1, "q_stride"), ("k_stride", 129, 1, "k_stride"),
    ("v_stride", 255, 1, "v_stride"), ("q_stride", (1 << 22) + 8, 1, "2^22"),
])
def test_linear_problem_refusals(field, value, code, text):
    p = linear()
    setattr(p.st, field, value)
    refused(code, text, lin_fwd(p))
    if "stride" not in field:
        assert G.load_library().gdn_linear_workspace_bytes(p.ref(), G.OP_BWD) == 0


def test_linear_refusals():
    refused(1, "NULL", lin_fwd(None))
    refused(1, "q is NULL", lin_fwd(linear(), q=None))
    refused(1, "not 16-byte", lin_fwd(linear(), q=ctypes.c_void_p(4100)))
    refused(1, "not 4-byte", lin_fwd(linear(), g=ctypes.c_void_p(4098)))
    refused(1, "g is NULL", lin_fwd(linear(), g=None))
    refused(1, "h0", lin_fwd(linear(), h0=PTR))
    refused(1, "h0", lin_fwd(linear(has_h0=True)))
    refused(1, "ht", lin_fwd(linear(), ht=PTR))
    refused(1, "ht", lin_fwd(linear(want_ht=True)))
    refused(1, "workspace", lin_fwd(linear(), ws=None))
    refused(4, "workspace", lin_fwd(linear(), nbytes=0))
    refused(1, "dO", lin_bwd(linear(), dO=None))
    refused(1, "dh0", lin_bwd(linear(), dh0=PTR))
    refused(1, "dh0", lin_bwd(linear(has_h0=True), h0=PTR))
    refused(4, "workspace", lin_bwd(linear(), nbytes=256))
    p = linear()
    p.cu[1] = 80
    refused(1, "decreases", lin_fwd(p))
    p = linear()
    p.cu[0] = 1
    refused(1, "cu_seqlens[0]", lin_fwd(p))
    assert G.load_library().gdn_linear_workspace_bytes(linear().ref(), G.OP_RECOMPUTE) == 0
    with pytest.raises(G.GdnError):
        linear(decay="channel")
    with pytest.raises(G.GdnError):
        linear(dtype=torch.float16)
    with pytest.raises(G.GdnError):
        G.LinearProblem([0], 1, 1, 64)


def test_linear_workspace():
    """Short documents need no states in the workspace; long ones do; the backward more than the forward, shared
    heads more again."""
    short, long = linear([64, 5]), linear([5000])
    assert G.gdn_linear_workspace_bytes(short, G.OP_FWD) == 256
    f, b = (G.gdn_linear_workspace_bytes(long, op) for op in (G.OP_FWD, G.OP_BWD))
    assert f >= 2 * 4 * 64 * 64 * 4 and b >= 2 * f
    assert b - G.gdn_linear_workspace_bytes(linear([5000], H=4), G.OP_BWD) == 2 * 5000 * 4 * (64 * 2 + 16)  # dq and dk: 16 bits each, units


@pytest.mark.parametrize("field,value,code,text", [
    ("n_seqs", 0, 1, "n_seqs"), ("n_slots", 0, 1, "n_slots"), ("n_tokens", 4, 1, "n_tokens"), ("h_v", 3, 1, "multiple"),
    ("d", 32, 2, "64 or 128"), ("dtype", -1, 2, "dtype"), ("decay", 5, 1, "decay"), ("scale", float("nan"), 1, "scale"),
    ("reserved0", 7, 1, "reserved0"), ("v_stride", 8, 1, "v_stride"), ("q_stride", (1 << 24) + 8, 1, "2^24"),
])
def test_linear_step_refusals(field, value, code, text):
    p = G.LinearStepProblem(3, 2, 4, 64, 8)
    setattr(p.st, field, value)
    refused(code, text, G.load_library().gdn_linear_step(p.ref(), *[PTR] * 4, None, PTR, PTR, None, PTR, PTR, None))


def test_linear_step_arrays():
    f, p = G.load_library().gdn_linear_step, G.LinearStepProblem(3, 2, 4, 64, 8)
    refused(1, "NULL", f(None, *[PTR] * 4, None, PTR, PTR, None, PTR, PTR, None))
    refused(1, "together", f(p.ref(), *[PTR] * 4, PTR, PTR, PTR, None, PTR, PTR, None))
    refused(1, "slot_in", f(p.ref(), *[PTR] * 4, None, None, PTR, None, PTR, PTR, None))
    refused(1, "states", f(p.ref(), *[PTR] * 4, None, PTR, PTR, None, None, PTR, None))
    with pytest.raises(G.GdnError):
        G.LinearStepProblem(3, 2, 4, 64, 8, cu_seqlens_host=[0, 1])


@pytest.mark.parametrize("field,value,code,text", [
    ("n_rows", -1, 1, "n_rows"), ("n_rows", 1 << 31, 1, "n_rows"), ("d", 100, 2, "multiple of 8"), ("d", 16392, 2, "16384"),
    ("d", 0, 2, "multiple of 8"), ("dtype", 9, 2, "dtype"), ("out", 2, 1, "out"), ("group", 16, 1, "group"),
    ("group", 64, 1, "e4m3"), ("eps", -1.0, 1, "eps"), ("eps", float("nan"), 1, "eps"), ("reserved0", 1, 1, "reserved0"),
    ("x_stride", 120, 1, "x_stride"), ("residual_stride", 132, 1, "residual_stride"),
])
def test_norm_refusals(field, value, code, text):
    p = G.RmsNormProblem(4, 128)
    setattr(p.st, field, value)
    refused(code, text, G.load_library().gdn_rms_norm_fwd(p.ref(), PTR, PTR, PTR, PTR, None, PTR, None))
    assert G.load_library().gdn_rms_norm_workspace_bytes(p.ref()) == 0


def test_norm_arrays():
    lib, p = G.load_library(), G.RmsNormProblem(4, 128)
    refused(1, "NULL", lib.gdn_rms_norm_fwd(None, PTR, PTR, None, PTR, None, None, None))
    refused(1, "x is NULL", lib.gdn_rms_norm_fwd(p.ref(), None, PTR, None, PTR, None, None, None))
    refused(1, "scales", lib.gdn_rms_norm_fwd(p.ref(), PTR, PTR, None, PTR, PTR, None, None))
    refused(1, "together", lib.gdn_rms_norm_fwd(p.ref(), PTR, PTR, PTR, PTR, None, None, None))
    refused(1, "together", lib.gdn_rms_norm_fwd(p.ref(), PTR, PTR, None, PTR, None, PTR, None))
    e = G.RmsNormProblem(4, 160, out="e4m3", group=32)
    refused(1, "scales", lib.gdn_rms_norm_fwd(e.ref(), PTR, PTR, None, PTR, None, None, None))
    refused(2, "backward", lib.gdn_rms_norm_bwd(e.ref(), PTR, PTR, PTR, None, PTR, PTR, PTR, 1 << 30, None))
    refused(1, "weight", lib.gdn_rms_norm_bwd(p.ref(), PTR, None, PTR, None, PTR, PTR, PTR, 1 << 30, None))
    refused(4, "workspace", lib.gdn_rms_norm_bwd(p.ref(), PTR, PTR, PTR, None, PTR, PTR, PTR, 0, None))
    e.st.group = 64
    refused(1, "multiple of group", lib.gdn_rms_norm_fwd(e.ref(), PTR, PTR, None, PTR, PTR, None, None))
    for kw in (dict(out="e5m2"), dict(dtype=torch.float16)):
        with pytest.raises(G.GdnError):
            G.RmsNormProblem(4, 128, **kw)
    assert G.gdn_rms_norm_workspace_bytes(p) == 4 * 128 * 4 // 4  # one workgroup of four rows


@pytest.mark.parametrize("field,value,text", [
    ("n_seqs", 0, "n_seqs"), ("n_seqs", 4097, "n_seqs"), ("n_tokens", -1, "n_tokens"), ("n_tokens", 1 << 31, "n_tokens"),
    ("block", 0, "block"), ("max_blocks", 0, "max_blocks"), ("n_free", -1, "n_free"), ("reserved0", 1, "reserved0"),
])
def test_maps_refusals(field, value, text):
    p = G.StepMapsProblem(4, 8, 16, 10, 5)
    setattr(p.st, field, value)
    outs = (ctypes.c_void_p * 9)()
    refused(1, text, G.load_library().gdn_step_maps(p.ref(), *[PTR] * 5, outs, None))


def test_maps_arrays():
    f, p, outs = G.load_library().gdn_step_maps, G.StepMapsProblem(4, 8, 16, 10, 5), (ctypes.c_void_p * 9)()
    refused(1, "NULL", f(None, *[PTR] * 5, outs, None))
    refused(1, "NULL", f(p.ref(), *[PTR] * 5, None, None))
    for i, name in enumerate(("lengths", "contexts", "block_table", "free_list", "free_count")):
        a = [PTR] * 5
        a[i] = None
        refused(1, name, f(p.ref(), *a, outs, None))
    outs[3] = 4100
    refused(1, "16-byte", f(p.ref(), *[PTR] * 5, outs, None))


def test_binding_refuses_tensors_on_the_cpu():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    q = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: G.gdn_rms_norm_fwd(G.RmsNormProblem(4, 128), x),
                 lambda: G.gdn_rms_norm_bwd(G.RmsNormProblem(4, 128), x, x),
                 lambda: G.gdn_linear_fwd(linear([5], 2, 2), q, q, q, q, i),
                 lambda: G.gdn_linear_bwd(linear([5], 2, 2), q, q, q, q, i, q),
                 lambda: G.gdn_linear_step(G.LinearStepProblem(5, 2, 2, 64, 8), q, q, q, q, q, i, i),
                 lambda: G.gdn_step_maps(G.StepMapsProblem(4, 8, 16, 10, 5), i, i, i, i, i)):
        with pytest.raises(G.GdnError) as e:
            call()
        assert "expected a GPU" in str(e.value)
