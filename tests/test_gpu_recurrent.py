"""GPU tests of the recurrent gated delta rule on cached states against the FP64 token recurrence:
every output row and every state, at the sizes and slots where it can go wrong."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
import oracle
from step_util import check, f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
# sums of 128 products, and a state's roundings over the tokens it remembers
K = 400


def make(lengths, H, HV, d, dtype=torch.bfloat16, keep=False, fresh=(), spare=3, packed=False, seed=3, **kw):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    N, T = len(lengths), sum(lengths)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    slots = N + (T if keep else 0) + spare
    order = torch.randperm(slots, generator=gen, device=DEV).to(torch.int32)
    s = dict(cu_host=cu, cu=torch.from_numpy(cu).to(DEV), slots=slots)
    if packed:
        x = normal(T, (2 * H + HV) * d + 8).to(dtype)
        s["q"] = x[:, :H * d].view(T, H, d)
        s["k"] = x[:, H * d:2 * H * d].view(T, H, d)
        s["v"] = x[:, 2 * H * d:(2 * H + HV) * d].view(T, HV, d)
    else:
        s["q"], s["k"], s["v"] = normal(T, H, d).to(dtype), normal(T, H, d).to(dtype), normal(T, HV, d).to(dtype)
    s["beta"] = torch.sigmoid(normal(T, HV))
    s["g"] = torch.nn.functional.logsigmoid(normal(T, HV) + 3)
    s["states"] = 0.1 * normal(slots, HV, d, d)
    s["slot_in"] = order[:N].clone()
    for n in fresh:
        s["slot_in"][n] = -1
    s["slot_out"] = order[:N].clone()
    s["slot_tok"] = order[N:N + T].clone() if keep else None
    s.update(kw)
    return s


def reference(s, l2norm=True):
    """(o, states) by the token recurrence, a call per sequence, or per token where states are kept."""
    q, k, v = (x.float().cpu().numpy() for x in (s["q"], s["k"], s["v"]))
    g, beta = s["g"].cpu().numpy(), s["beta"].cpu().numpy()
    start = s["states"].cpu().numpy()
    o, states = np.zeros(v.shape), start.astype(np.float64)
    si, so = s["slot_in"].tolist(), s["slot_out"].tolist()
    st = s["slot_tok"].tolist() if s["slot_tok"] is not None else None
    for n in range(len(si)):
        a, e = int(s["cu_host"][n]), int(s["cu_host"][n + 1])
        h0 = start[si[n]][None] if si[n] >= 0 else np.zeros_like(start[:1])
        part = lambda x, b: np.ascontiguousarray(x[a:b])
        for b in ([e] if st is None else range(a + 1, e + 1)) if e > a else []:
            oo, ht = oracle.fwd(np.array([0, b - a], np.int32), part(q, b), part(k, b), part(v, b), part(g, b),
                                part(beta, b), np.ascontiguousarray(h0), l2norm=l2norm)
            o[a:b] = oo
            if st is not None and st[b - 1] >= 0:
                states[st[b - 1]] = ht[0]
        if so[n] >= 0:
            states[so[n]] = ht[0] if e > a else h0[0]
    return o, states


def run(s, l2norm=True, one=None, **kw):
    H, d, HV = s["q"].shape[1], s["q"].shape[2], s["v"].shape[1]
    one = bool(np.all(np.diff(s["cu_host"]) == 1)) if one is None else one
    p = G.RecurrentProblem(len(s["cu_host"]) - 1, H, HV, d, s["slots"], cu_seqlens_host=None if one else s["cu_host"],
                           dtype=s["v"].dtype, l2norm=l2norm)
    print("recurrent N=%d T=%d (H,HV)=(%d,%d) d=%d" % (len(s["cu_host"]) - 1, s["v"].shape[0], H, HV, d), flush=True)
    states = s["states"].clone()
    o = G.gdn_recurrent(p, s["q"], s["k"], s["v"], s["g"], s["beta"], states, s["slot_in"], s["slot_out"],
                        slot_tok=s["slot_tok"], cu_seqlens=None if one else s["cu"], **kw)
    torch.cuda.synchronize()
    return o, states


CASES = {
    "one_sequence": dict(lengths=[1], H=16, HV=48, d=128),
    "decode_33": dict(lengths=[1] * 33, H=2, HV=6, d=128, fresh=(4, 32)),
    "decode_300_d64": dict(lengths=[1] * 300, H=1, HV=3, d=64),
    "decode_f32": dict(lengths=[1] * 7, H=3, HV=3, d=128, dtype=torch.float32),
    "decode_packed": dict(lengths=[1] * 9, H=2, HV=4, d=64, packed=True),
    "ragged": dict(lengths=[3, 0, 1, 17, 64, 2, 0], H=2, HV=6, d=128, fresh=(1, 3)),
    "ragged_f32_d64": dict(lengths=[5, 130, 0, 63], H=4, HV=8, d=64, dtype=torch.float32, fresh=(0,)),
    "drafts": dict(lengths=[8, 1, 5, 0, 3], H=2, HV=4, d=128, keep=True),
    "drafts_packed_f32": dict(lengths=[2, 4, 7], H=1, HV=2, d=64, keep=True, packed=True, dtype=torch.float32),
    "long": dict(lengths=[1000, 37], H=1, HV=2, d=128, fresh=(0,)),
    "long_f32_many_heads": dict(lengths=[300], H=16, HV=48, d=128, dtype=torch.float32),
}


@pytest.mark.parametrize("l2norm", [True, False], ids=["l2norm", "given"])
@pytest.mark.parametrize("name", CASES)
def test_recurrent(name, l2norm):
    s = make(**CASES[name])
    if not l2norm:  # rows of about unit length
        s["q"], s["k"] = ((x.float() * x.shape[-1] ** -0.5).to(x.dtype) for x in (s["q"], s["k"]))
    o, states = run(s, l2norm)
    o_ref, st_ref = reference(s, l2norm)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)


@pytest.mark.parametrize("keep", [True, False], ids=["keep", "last"])
@pytest.mark.parametrize("N", [1, 3, 8], ids=["16_columns", "one_wave_groups", "four_wave_groups"])
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float32)], ids=["bf16_128", "f32_64"])
def test_few_tokens_by_the_number_of_waves(d, dtype, N, keep):
    s = make([3, 0, 2, 4, 1, 3, 2, 4, 2][:N + (N > 1)], H=16, HV=48 * (128 // d), d=d, dtype=dtype, keep=keep, fresh=(0,))
    o, states = run(s)
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)


# runs go 16 tokens at a time, 64 a turn: lengths at and beside both, and sequences that end in a block
RUNS = {
    "bf16_128": dict(lengths=[16, 17, 15, 64, 65, 63, 129, 1, 0, 128], H=2, HV=4, d=128, fresh=(3, 8)),
    "f32_64_packed": dict(lengths=[80, 7, 33, 0, 192, 97], H=1, HV=3, d=64, dtype=torch.float32, packed=True, fresh=(1,)),
    "f32_128": dict(lengths=[31, 48], H=2, HV=2, d=128, dtype=torch.float32),
    "bf16_64_many": dict(lengths=[13] * 40 + [70], H=2, HV=8, d=64),
    "keep_long": dict(lengths=[40, 3], H=1, HV=2, d=128, keep=True),
}


@pytest.mark.parametrize("gates", ["drawn", "strong", "rising", "none"])
@pytest.mark.parametrize("name", RUNS)
def test_runs(name, gates):
    """Decays as the layer draws them; down to e^-80 and to nothing in places; log decays above 0; no
    decay, full writes and nearly equal keys, where the block's inverse has the largest entries."""
    s = make(**RUNS[name])
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    if gates == "strong":
        pick = torch.rand(s["g"].shape, generator=gen, device=DEV)
        s["g"][pick < 0.2], s["g"][pick > 0.9] = -80.0, -1e30
    elif gates == "rising":
        s["g"] = 0.05 * torch.rand(s["g"].shape, generator=gen, device=DEV)
    elif gates == "none":
        s["g"][:], s["beta"][:] = 0.0, 1.0
        s["k"].copy_((s["k"][:1].float() + 0.05 * s["k"].float()).to(s["k"].dtype))
    o, states = run(s)
    o_ref, st_ref = reference(s)
    # with no decay a state remembers every token: its roundings add up over the run
    k = K * (4 if gates in ("rising", "none") else 1)
    check("o", o, o_ref, k)
    check("states", states, st_ref, k)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_runs_of_many_columns(dtype, d):
    """More columns of 32 than the card has CUs: workgroups of 64 columns and 64 tokens a turn."""
    s = make([80, 7, 33, 0, 129, 64, 65, 63, 16, 1], H=4, HV=32, d=d, dtype=dtype, fresh=(2, 3))
    o, states = run(s)
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)


@pytest.mark.parametrize("l2norm", [True, False], ids=["l2norm", "given"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_long_runs_of_few_columns(dtype, d, l2norm):
    """Two waves share a column: odd and even numbers of blocks and turns, short sequences beside long."""
    s = make([65, 16, 0, 33, 128, 1, 112, 200, 17], H=1, HV=2, d=d, dtype=dtype, fresh=(0, 4), packed=d == 64)
    if not l2norm:
        s["q"].copy_((s["q"].float() * d ** -0.5).to(dtype))
        s["k"].copy_((s["k"].float() * d ** -0.5).to(dtype))
    o, states = run(s, l2norm)
    again = run(s, l2norm)
    assert torch.equal(o, again[0]) and torch.equal(states, again[1])
    o_ref, st_ref = reference(s, l2norm)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)


@pytest.mark.parametrize("N", [15, 16, 17])
def test_sequences_of_any_length_in_any_order(N):
    """Up to 16 sequences run longest first: each still gets its own rows and slots."""
    s = make([(7 * n * n) % 41 for n in range(N)], 1, 2, 64, fresh=(3, N - 1))
    o, states = run(s)
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)


@pytest.mark.parametrize("HV", [2, 48])
def test_runs_in_a_graph(HV):
    s = make([40, 70, 5], H=2, HV=HV, d=128)
    p = G.RecurrentProblem(3, 2, HV, 128, s["slots"], cu_seqlens_host=s["cu_host"])
    out = torch.tensor([i for i in range(s["slots"]) if i not in s["slot_in"].tolist()], dtype=torch.int32, device=DEV)
    call = lambda st: G.gdn_recurrent(p, *(s[x] for x in ("q", "k", "v", "g", "beta")), st, s["slot_in"], out, cu_seqlens=s["cu"])
    eager_states = s["states"].clone()
    eager = call(eager_states)
    states = s["states"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call(states)
    for _ in range(3):
        states.copy_(s["states"])
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager) and torch.equal(states, eager_states)


def test_a_run_does_not_see_its_neighbours():
    """Rows before and after a sequence hold NaN (another sequence's): blocks that end inside the turn
    and loads past the end must not let them in."""
    s = make([20, 37, 70], 1, 2, 64)
    clean = run(s)
    for x in ("q", "k", "v", "g", "beta"):
        s[x][:20], s[x][57:] = float("nan"), float("nan")
    o, states = run(s)
    assert torch.equal(o[20:57], clean[0][20:57])
    slot = s["slot_out"][1].long()
    assert torch.equal(states[slot], clean[1][slot])
    assert torch.isnan(o[:20].float()).all() and torch.isnan(o[57:].float()).all()


def test_a_run_then_steps_equal_the_whole_run():
    s = make([50, 23], 2, 4, 128, dtype=torch.float32)
    o, states = run(s)
    cut = make([50, 23], 2, 4, 128, dtype=torch.float32)
    rows = [slice(0, 41), slice(50, 64)]
    part = {x: torch.cat([cut[x][r] for r in rows]) for x in ("q", "k", "v", "g", "beta")}
    p = G.RecurrentProblem(2, 2, 4, 128, cut["slots"], cu_seqlens_host=[0, 41, 55], dtype=torch.float32)
    st = cut["states"]
    G.gdn_recurrent(p, *part.values(), st, cut["slot_in"], cut["slot_out"],
                    cu_seqlens=torch.tensor([0, 41, 55], dtype=torch.int32, device=DEV))
    one = G.RecurrentProblem(2, 2, 4, 128, cut["slots"], dtype=torch.float32)
    for i in range(9):
        at = torch.tensor([41 + i, 64 + i], device=DEV)
        got = G.gdn_recurrent(one, *(cut[x][at] for x in ("q", "k", "v", "g", "beta")), st, cut["slot_out"], cut["slot_out"])
        check("o", got, f64(o[at]), 2 * K)
    torch.cuda.synchronize()
    check("states", st, f64(states), 2 * K)


def test_slots_not_named_are_untouched_and_sequences_may_share_a_start():
    s = make([1, 2, 3], 2, 4, 64)
    s["slot_in"][:] = s["slot_in"][0]  # one prompt's state, three continuations
    s["slot_out"] = torch.tensor([-1, 4, 5], dtype=torch.int32, device=DEV)
    s["slot_in"][:] = 2
    o, states = run(s)
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)
    for slot in range(s["slots"]):
        if slot not in (4, 5):
            assert torch.equal(states[slot], s["states"][slot])


def test_one_token_with_and_without_lengths_is_the_same():
    s = make([1] * 13, 2, 6, 128)
    a, b = run(s, one=True), run(s, one=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_runs_and_single_tokens_agree_to_rounding():
    """The same tokens in one call and one by one (a new call per token), in place."""
    s = make([6, 6, 6], 2, 4, 128, dtype=torch.float32)
    o, states = run(s)
    p = G.RecurrentProblem(3, 2, 4, 128, s["slots"], dtype=torch.float32)
    st, rows = s["states"].clone(), []
    for i in range(6):
        at = torch.tensor([i, 6 + i, 12 + i], device=DEV)
        rows.append(G.gdn_recurrent(p, *(s[x][at] for x in ("q", "k", "v", "g", "beta")), st, s["slot_in"], s["slot_out"]))
    torch.cuda.synchronize()
    o1 = torch.stack(rows, 1).flatten(0, 1)
    check("o", o1, f64(o), K)
    check("states", st, f64(states), K)


def test_gates_at_their_ends():
    """g = -inf forgets the state, g = 0 keeps it, beta = 0 writes nothing, a zero key row is harmless
    under the norm."""
    s = make([2, 2, 2, 2], 1, 2, 128)
    s["g"][0:2] = float("-inf")
    s["g"][2:4], s["beta"][2:4] = 0.0, 0.0
    s["k"][4:6] = 0
    s["g"][6:8], s["beta"][6:8] = -80.0, 1.0
    o, states = run(s)
    assert torch.equal(states[s["slot_out"][1].long()], s["states"][s["slot_in"][1].long()])
    s["g"][0:2] = -1e30  # the oracle takes finite logs; exp is 0 either way
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)


def test_nan_in_one_state_stays_in_its_sequence_and_head():
    s = make([1, 1, 1], 2, 4, 128)
    s["states"][s["slot_in"][1].long(), 3] = float("nan")
    o, states = run(s)
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[1, 3] = True
    assert torch.equal(torch.isnan(o), bad)
    bad = torch.zeros_like(states, dtype=torch.bool)
    bad[s["slot_out"][1].long(), 3] = True
    assert torch.equal(torch.isnan(states), bad)


@pytest.mark.parametrize("what", ["slot_in", "slot_out", "slot_tok", "cu"])
def test_device_arrays_out_of_range_are_refused_on_the_device(what):
    """NaN rows for the sequence (or token) with the bad entry, no state of it written, the rest right."""
    s = make([2, 3, 4], 2, 4, 64, keep=True)
    s["slot_out"][:] = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    used = set(s["slot_tok"].tolist())
    s["slot_in"][:] = -1
    free = [x for x in range(s["slots"]) if x not in used]
    s["slot_out"][:] = torch.tensor(free[:3], dtype=torch.int32, device=DEV)
    o_ref, st_ref = reference(s)
    rows = range(2, 5)
    if what == "slot_tok":
        lost = [s["slot_tok"][3].item()]
        s["slot_tok"][3] = s["slots"]
        rows = [3]
    else:
        lost = s["slot_tok"][2:5].tolist() + [free[1]]
        if what == "cu":
            s["cu"] = torch.tensor([0, 2, 5, 10], dtype=torch.int32, device=DEV)  # past the last token
            rows, lost = range(5, 9), s["slot_tok"][5:9].tolist() + [free[2]]
        else:
            s[what][1] = s["slots"] if what == "slot_in" else -2
    o, states = run(s)
    rows = list(rows)
    assert torch.isnan(o[rows].float()).all()
    good = [t for t in range(9) if t not in rows]
    check("o", o[good], o_ref[good], K)
    st_ref[lost] = s["states"][lost].double().cpu().numpy()
    check("states", states, st_ref, K)


def test_states_past_32_bit_offsets():
    """Slots whose first element lies past 2^31 and past 2^32 elements."""
    HV, d = 48, 128
    slots = 2 ** 32 // (HV * d * d) + 3
    s = make([1, 1, 2], 16, HV, d, spare=0)
    pool = torch.empty(slots, HV, d, d, device=DEV)
    where = torch.tensor([0, 2 ** 31 // (HV * d * d) + 1, slots - 1], dtype=torch.int32, device=DEV)
    small = s["states"][s["slot_in"].long()].clone()
    pool[where.long()] = small
    p = G.RecurrentProblem(3, 16, HV, d, slots, cu_seqlens_host=s["cu_host"])
    o = G.gdn_recurrent(p, s["q"], s["k"], s["v"], s["g"], s["beta"], pool, where, where, cu_seqlens=s["cu"])
    got = pool[where.long()].clone()
    torch.cuda.synchronize()
    s["states"], s["slot_in"] = small, torch.arange(3, dtype=torch.int32, device=DEV)
    s["slot_out"] = s["slot_in"]
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", got, st_ref, K)


def test_on_a_stream_of_its_own():
    s = make([1] * 20, 2, 4, 128)
    ref = run(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(s, stream=side)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


def test_graph_replays_equal_eager_steps():
    """A captured decoding step, replayed with other eager work between, against eager steps."""
    s = make([1] * 5, 2, 4, 128)
    p = G.RecurrentProblem(5, 2, 4, 128, s["slots"])
    a = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    eager, graphed = s["states"].clone(), s["states"].clone()
    o = torch.empty_like(s["v"])
    G.gdn_recurrent(p, *a, graphed, s["slot_in"], s["slot_out"], o=o)
    graphed.copy_(s["states"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.gdn_recurrent(p, *a, graphed, s["slot_in"], s["slot_out"], o=o)
    for i in range(4):
        s["v"].copy_(torch.roll(s["v"], 1, 0))
        want = G.gdn_recurrent(p, *a, eager, s["slot_in"], s["slot_out"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(graphed, eager), i


def test_binding_refuses_wrong_tensors():
    s = make([1, 1], 2, 4, 64)
    p = G.RecurrentProblem(2, 2, 4, 64, s["slots"])
    good = dict(q=s["q"], k=s["k"], v=s["v"], g=s["g"], beta=s["beta"], states=s["states"], slot_in=s["slot_in"],
                slot_out=s["slot_out"])
    before = s["states"].clone()
    for name, bad, fragment in (
            ("q", s["q"].float(), "type"), ("k", s["k"][:1], "shape"), ("g", s["g"].double(), "type"),
            ("v", s["v"].transpose(0, 1).contiguous().transpose(0, 1), "contiguous"),
            ("states", s["states"][:-1], "shape"), ("slot_in", s["slot_in"].long(), "type"),
            ("slot_out", s["slot_out"].cpu(), "is on"), ("beta", s["beta"].t().contiguous().t(), "contiguous")):
        with pytest.raises(G.GdnError, match=fragment):
            G.gdn_recurrent(p, **{**good, name: bad})
    with pytest.raises(G.GdnError, match="given together"):
        G.gdn_recurrent(p, **good, cu_seqlens=s["cu"])
    torch.cuda.synchronize()
    assert torch.equal(before, s["states"])


def test_an_allocation_that_fails_is_torchs_own_error():
    """Servers catch torch.OutOfMemoryError to shrink a batch: an output that does not fit raises it, as
    it does from the calls that allocate in Python."""
    T, HV, d = 4096, 32, 128
    p = G.RecurrentProblem(1, 1, HV, d, 1, cu_seqlens_host=[0, T])
    s = make([T], 1, HV, d, spare=0)
    a = (s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["slot_in"], s["slot_out"])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction(torch.cuda.memory_reserved() / total)  # nothing more
    try:
        with pytest.raises(torch.OutOfMemoryError):
            G.gdn_recurrent(p, *a, cu_seqlens=s["cu"])
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert G.gdn_recurrent(p, *a, cu_seqlens=s["cu"]).shape == (T, HV, d)
    torch.cuda.synchronize()


def test_bad_problems_are_refused_before_anything_is_allocated():
    """A descriptor that no tensor fits (here a negative width) is a GdnError, not the allocator's."""
    s = make([1, 1], 2, 4, 64)
    a = (s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["slot_in"], s["slot_out"])
    for field, value in (("d", -64), ("h_v", -4), ("n_tokens", -2)):
        p = G.RecurrentProblem(2, 2, 4, 64, s["slots"])
        setattr(p.st, field, value)
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        with pytest.raises(G.GdnError):
            G.gdn_recurrent(p, *a)
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


# the run kernel's forms: 32 columns a workgroup, two waves a column, 64 columns a workgroup
FORMS = {
    "32_columns": dict(lengths=[40, 17, 0, 64, 3], H=2, HV=4),
    "two_waves": dict(lengths=[100, 17, 0, 65, 3], H=1, HV=2),
    "64_columns": dict(lengths=[80, 17, 0, 129, 3, 64, 65], H=4, HV=32),
}


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float32)], ids=["bf16_128", "f32_64"])
@pytest.mark.parametrize("form", FORMS)
def test_runs_whose_decay_products_leave_the_range(form, d, dtype):
    """Log decays of 12 on a state that is empty until just before it is read: the products of a block's
    decays overflow, the recurrence does not, and its outputs are ordinary numbers."""
    s = make(**FORMS[form], d=d, dtype=dtype)
    s["slot_in"][:] = -1
    for a, e in zip(s["cu_host"][:-1], s["cu_host"][1:]):
        at = torch.arange(int(e) - int(a), device=DEV)
        s["g"][a:e] = torch.where(at % 11 == 0, -1e30, 12.0)[:, None]  # the state is forgotten, then multiplied up
        s["beta"][a:e] *= (at % 11 >= 9)[:, None]  # and written only shortly before it is forgotten
    o, states = run(s)
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)


def finite_where_the_recurrence_is(s):
    """Masks (o, last states) of what a float64 token recurrence in torch makes finite."""
    H, HV, d = s["q"].shape[1], s["v"].shape[1], s["q"].shape[2]
    head = torch.arange(HV) // (HV // H)
    q, k, v, g, beta, states = (s[x].double().cpu() for x in ("q", "k", "v", "g", "beta", "states"))
    q, k = (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
    o, last = torch.zeros_like(v), states.clone()
    for n, (a, e) in enumerate(zip(s["cu_host"][:-1], s["cu_host"][1:])):
        S = states[s["slot_in"][n]].clone()
        for t in range(int(a), int(e)):
            S = S * g[t].exp()[:, None, None]
            kt = k[t, head][:, :, None]
            u = beta[t][:, None] * (v[t] - (S * kt).sum(1))
            S = S + kt * u[:, None]
            o[t] = (S * q[t, head][:, :, None]).sum(1)
        last[s["slot_out"][n]] = S
    return torch.isfinite(o), torch.isfinite(last)


@pytest.mark.parametrize("bad", ["v_nan", "v_inf", "k_nan", "q_inf", "g_nan", "beta_inf"])
@pytest.mark.parametrize("form", FORMS)
def test_a_bad_row_reaches_no_earlier_token_of_a_run(form, bad):
    """One value that is not finite, inside a block of 16 tokens: the tokens before it keep their outputs
    to rounding, other sequences and heads theirs bit for bit, as without it."""
    s = make(**FORMS[form], d=64, dtype=torch.float32)
    clean = run(s)
    name, value = bad.split("_")
    t = 21  # of the first sequence, in its second block
    at = (t, 0, 5) if name in "qkv" else (t, 0)
    s[name][at] = float(value)
    o, states = run(s)
    good_o, good_states = (x.to(DEV) for x in finite_where_the_recurrence_is(s))
    assert torch.equal(torch.isfinite(o), good_o) and torch.equal(torch.isfinite(states), good_states)
    assert not good_o[t, 0].all() and good_o[:t].all()
    check("o before it", o[:t], f64(clean[0][:t]), K)
    end = int(s["cu_host"][1])
    assert torch.equal(o[end:], clean[0][end:])
    heads = s["v"].shape[1] // s["q"].shape[1] if name in "qk" else 1
    assert torch.equal(o[:, heads:], clean[0][:, heads:])
    others = [x for x in range(s["slots"]) if x != s["slot_out"][0].item()]
    assert torch.equal(states[others], clean[1][others])


MIXED = {  # (sequences of at most 8 tokens fill the card with run workgroups several times; the others are longer)
    "bf16_128": dict(lengths=[1, 8, 13, 0, 2, 9] * 9 + [90], H=8, HV=48, d=128, fresh=(2, 3)),
    "f32_64": dict(lengths=[3, 1, 0, 8, 1] * 20 + [16, 9, 200], H=4, HV=32, d=64, dtype=torch.float32, fresh=(1, 101)),
}


@pytest.mark.parametrize("name", MIXED)
def test_short_sequences_beside_long_ones(name):
    s = make(**MIXED[name])
    o, states = run(s)
    again = run(s)
    assert torch.equal(o, again[0]) and torch.equal(states, again[1])
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)


def test_lengths_on_the_device_may_differ_from_the_hosts():
    """A captured mixed call replayed with other lengths, the short sequences long and the long short:
    each sequence is taken by one of the call's kernels."""
    d = dict(MIXED["bf16_128"], fresh=())
    s, order = make(**d), list(reversed(d["lengths"]))
    p = G.RecurrentProblem(len(order), d["H"], d["HV"], d["d"], s["slots"], cu_seqlens_host=s["cu_host"])
    states, cu = s["states"].clone(), s["cu"].clone()
    call = lambda: G.gdn_recurrent(p, *(s[x] for x in ("q", "k", "v", "g", "beta")), states, s["slot_in"],
                                   s["slot_out"], cu_seqlens=cu)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call()
    s["cu_host"] = np.concatenate([[0], np.cumsum(order)]).astype(np.int32)
    cu.copy_(torch.from_numpy(s["cu_host"]))
    states.copy_(s["states"])
    o.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)


def test_a_long_sequence_does_not_slow_the_short_ones_down():
    """128 decoding sequences with one of 13 tokens among them: no more than half again over the 128 alone
    (one kernel for all by the longest took twice as long)."""
    def took(lengths):
        s = make(lengths, H=16, HV=48, d=128, spare=0)
        p = G.RecurrentProblem(len(lengths), 16, 48, 128, s["slots"], cu_seqlens_host=s["cu_host"])
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        best = float("inf")
        for _ in range(6):
            a.record()
            for _ in range(10):
                G.gdn_recurrent(p, *(s[x] for x in ("q", "k", "v", "g", "beta")), s["states"], s["slot_in"],
                                s["slot_out"], cu_seqlens=s["cu"])
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) / 10)
        return best

    alone, mixed = took([1] * 128), took([1] * 127 + [13])
    print("128 sequences of one token %.3f ms, with one of 13 %.3f ms" % (alone, mixed), flush=True)
    assert mixed < 1.5 * alone


# a call for each kernel and each way through it
KERNELS = {
    "one_token": dict(lengths=[1] * 5, H=2, HV=4, d=128),
    "one_token_many": dict(lengths=[1] * 60, H=8, HV=48, d=64),
    "few_tokens_16_columns": dict(lengths=[2, 4, 3, 1, 2], H=2, HV=4, d=128),
    "few_tokens_32_columns": dict(lengths=[2, 4, 3, 1, 2] * 6, H=4, HV=48, d=64),
    "run_two_waves": dict(lengths=[70, 33, 90, 16, 5], H=1, HV=2, d=64),
    "run_two_waves_128": dict(lengths=[70, 33, 90, 16, 5], H=1, HV=2, d=128, dtype=torch.float32),
    "run_32_columns": dict(lengths=[17, 33, 20, 16, 5], H=2, HV=4, d=128),
    "run_64_columns": dict(lengths=[17, 33, 80, 16, 5], H=4, HV=48, d=128),
    "mixed": MIXED["bf16_128"],
}


@pytest.mark.parametrize("name,what", [(x, y) for x in KERNELS for y in ("slot_in", "slot_out", "start", "end")
                                       if y.startswith("slot") or max(KERNELS[x]["lengths"]) > 1])
def test_every_kernel_refuses_what_is_out_of_range_on_the_device(name, what):
    """A slot past the cache or a token range that leaves [0, T]: NaN rows for that sequence, no state of
    it, the others right."""
    s = make(**KERNELS[name])
    N = len(s["slot_in"])
    n = dict(slot_in=2, slot_out=1, start=0, end=N - 1)[what]
    rows = slice(int(s["cu_host"][n]), int(s["cu_host"][n + 1]))
    o_ref, st_ref = reference(s)
    slot = s["slot_out"][n].item()
    st_ref[slot] = f64(s["states"][slot])
    if what == "slot_in":
        s["slot_in"][n] = s["slots"]
    elif what == "slot_out":
        s["slot_out"][n] = -2
    else:
        s["cu"][n if what == "start" else N] += -1 if what == "start" else 1
    o, states = run(s)
    assert torch.isnan(o[rows].float()).all() and rows.stop > rows.start
    good = torch.ones(o.shape[0], dtype=torch.bool)
    good[rows] = False
    check("o", o[good.to(DEV)], o_ref[good.numpy()], K)
    check("states", states, st_ref, K)


@pytest.mark.parametrize("name", KERNELS)
def test_every_kernel_leaves_states_nowhere_and_shares_starts(name):
    """slot_out = -1 keeps no state; sequences may start from one slot that none of them writes."""
    s = make(**KERNELS[name])
    free = [x for x in range(s["slots"]) if x not in s["slot_in"].tolist()]
    s["slot_in"][1::2] = free[0]
    s["slot_out"][::3] = -1
    o, states = run(s)
    o_ref, st_ref = reference(s)
    check("o", o, o_ref, K)
    check("states", states, st_ref, K)
    named = set(s["slot_out"].tolist())
    for slot in (x for x in range(s["slots"]) if x not in named):
        assert torch.equal(states[slot], s["states"][slot])


@pytest.mark.parametrize("name", ["few_tokens_16_columns", "run_two_waves", "run_32_columns", "run_64_columns", "mixed"])
def test_rows_of_no_sequence_keep_their_values(name):
    """The device's lengths end before T (a shorter batch): the rows behind them are not written."""
    s = make(**KERNELS[name])
    cut = int(s["cu_host"][-2])
    s["cu"][-1] = cut
    o = torch.full(s["v"].shape, 7.0, dtype=s["v"].dtype, device=DEV)
    run(s, o=o)
    s["cu_host"] = s["cu_host"].copy()
    s["cu_host"][-1] = cut
    o_ref, _ = reference(s)
    assert (o[cut:] == 7).all() and cut < o.shape[0]
    check("o", o[:cut], o_ref[:cut], K)


@pytest.mark.parametrize("end", [0, -1, -2 ** 31])
@pytest.mark.parametrize("name", [x for x in KERNELS if not x.startswith("one")])
def test_a_range_that_falls_is_empty(name, end):
    """The second entry of the device's cu_seqlens below the first, down to the type's lowest value: no rows
    for the first sequence, and for the second NaN from its cut start on if that lies below 0."""
    s = make(**KERNELS[name])
    s["cu"][0], s["cu"][1] = min(end + 1, 0), end
    stop = int(s["cu_host"][2])
    o_ref, st_ref = reference(s)
    if end == 0:  # an empty first sequence, and one that begins too early
        s["cu"][0] = 1
    lost = s["slot_out"][:2].tolist()
    o, states = run(s)
    if end < 0:
        assert torch.isnan(o[:stop].float()).all()
    check("o", o[stop:], o_ref[stop:], K)
    keep = [x for x in range(s["slots"]) if x not in lost]
    check("states", states[keep], st_ref[keep], K)
    assert torch.equal(states[lost[0]], s["states"][lost[0]])
    assert (end == 0) or torch.equal(states[lost[1]], s["states"][lost[1]])
