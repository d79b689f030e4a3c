"""The serving and position operators of the gated delta rule layer: what is timed, at which sizes, and their plain forms.

Three operators, each reached through the package's own entry points:

  recurrent   the gated delta rule token by token on a cache of states (one token a sequence when decoding, a
              few when drafted tokens are checked or a prompt is extended): gdn_recurrent
  qk_rope     norms of the q and k heads with the position rotation in the same pass, forward and backward:
              gdn_qk_rope_fwd, gdn_qk_rope_bwd (norm "none": the rotation alone)
  conv_step   the causal conv1d + SiLU front-end on a cache of windows: gdn_conv_step

A case is a dict of plain values. `prepare` makes a case's inputs on the GPU from a seed, `run` is one pass (the
plain form in elementary torch operations, or the package's calls where `own` is true), `exact` the definition in
64 bits, `work` what a pass cannot do without.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # decoding for one user: a layer's states (16 q/k heads, 48 value heads, 128 wide) move one token on; latency
        dict(name="recurrent decode, 1", op="recurrent", seqs=1, longest=1, h_qk=16, h_v=48, d=128, dtype="bf16",
             l2norm=True, keep=False, fresh=0),
        # decoding for a full batch: one token for each of 256 sequences, states updated in place
        dict(name="recurrent decode, 256", op="recurrent", seqs=256, longest=1, h_qk=16, h_v=48, d=128, dtype="bf16",
             l2norm=True, keep=False, fresh=0),
        # checking drafted tokens: ragged runs of up to 8 tokens, the state after every token kept for the roll-back
        dict(name="recurrent drafts, 24", op="recurrent", seqs=24, longest=8, h_qk=16, h_v=48, d=128, dtype="bf16",
             l2norm=True, keep=True, fresh=0),
        # short prompts and continued ones in one call, f32, 64 wide, some sequences new, one empty
        dict(name="recurrent runs, 700", op="recurrent", seqs=5, longest=700, h_qk=4, h_v=8, d=64, dtype="f32",
             l2norm=True, keep=False, fresh=2),
        # a decoding step's 64 tokens: RMS norm with weights, half of each head rotated, far positions
        dict(name="qk_rope step, 64", op="qk_rope", way="fwd", tokens=64, h_q=16, h_k=16, d=128, rotary=64,
             layout="half", norm="rms", scaling="none", longest=262144, dtype="bf16", packed=True),
        # training: the pack of 4 documents (32,768 tokens) of the layer benchmark, whole heads rotated
        dict(name="qk_rope fwd, 32768", op="qk_rope", way="fwd", tokens=32768, h_q=16, h_k=16, d=128, rotary=128,
             layout="half", norm="rms", scaling="none", longest=12288, dtype="bf16", packed=False),
        # its backward: gradients of q, k and both weights
        dict(name="qk_rope bwd, 32768", op="qk_rope", way="bwd", tokens=32768, h_q=16, h_k=16, d=128, rotary=128,
             layout="half", norm="rms", scaling="none", longest=12288, dtype="bf16", packed=False),
        # rotation alone, interleaved pairs, few k heads, positions scaled for a longer context, odd token count
        dict(name="qk_rope rotate, 8191", op="qk_rope", way="fwd", tokens=8191, h_q=24, h_k=4, d=64, rotary=64,
             layout="interleaved", norm="none", scaling="linear", longest=65536, dtype="bf16", packed=True),
        # backward with L2 norms, f32, a quarter of a 96-wide head rotated with blended frequencies, odd token count
        dict(name="qk_rope bwd l2, 4099", op="qk_rope", way="bwd", tokens=4099, h_q=6, h_k=2, d=96, rotary=24,
             layout="interleaved", norm="l2", scaling="blend", longest=131072, dtype="f32", packed=False),
        # the front-end's step for one user: 10,240 channels, 4 taps; latency
        dict(name="conv_step decode, 1", op="conv_step", seqs=1, longest=1, q=2048, v=6144, width=4, dtype="bf16",
             bias=True, keep=False, fresh=0),
        # a full batch's step
        dict(name="conv_step decode, 256", op="conv_step", seqs=256, longest=1, q=2048, v=6144, width=4, dtype="bf16",
             bias=True, keep=False, fresh=0),
        # ragged runs of drafted tokens and new sequences in f32, the window after every token kept
        dict(name="conv_step drafts, 24", op="conv_step", seqs=24, longest=8, q=256, v=1032, width=3, dtype="f32",
             bias=False, keep=True, fresh=3),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.5 / hi)))))


def draw(rng):
    op = rng.choice(["recurrent", "recurrent", "qk_rope", "qk_rope", "conv_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "recurrent":
        d, kind = rng.choice([64, 128, 128]), rng.choice(["decode", "drafts", "run"])
        h_qk = rng.choice([1, 2, 3, 4, 8, 16])
        h_v = h_qk * rng.choice([1, 2, 3])
        seqs = _log(rng, 1, {"decode": 256, "drafts": 24, "run": 12}[kind])
        longest = {"decode": 1, "drafts": rng.randint(2, 8), "run": _log(rng, 9, 700)}[kind]
        return dict(op=op, seqs=seqs, longest=longest, h_qk=h_qk, h_v=h_v, d=d, dtype=dtype,
                    l2norm=rng.random() < 0.8, keep=kind == "drafts", fresh=rng.choice([0, 0, seqs // 3]))
    if op == "qk_rope":
        d = rng.choice([64, 128, 128, 96, 80, 256])
        norm = rng.choice(["rms", "rms", "l2", "none"])
        h_q, h_k = rng.choice([(16, 16), (24, 4), (8, 1), (5, 5), (32, 8), (3, 1)])
        most = 32768 * 32 * 128 * 2 // ((h_q + h_k) * d * (2 if dtype == "bf16" else 4))
        return dict(op=op, way=rng.choice(["fwd", "bwd"]), tokens=_log(rng, 1, min(most, 65536)), h_q=h_q, h_k=h_k, d=d,
                    rotary=rng.choice([d, d // 2 // 8 * 8, 16]), layout=rng.choice(["half", "interleaved"]), norm=norm,
                    scaling=rng.choice(["none", "linear", "blend"]), longest=_log(rng, 64, 262144), dtype=dtype,
                    packed=rng.random() < 0.5)
    seqs, many = _log(rng, 1, 256), rng.random() < 0.4
    return dict(op=op, seqs=min(seqs, 24) if many else seqs, longest=rng.randint(2, 8) if many else 1,
                q=8 * _log(rng, 1, 256), v=8 * _log(rng, 1, 768), width=rng.choice([2, 3, 4, 4]), dtype=dtype,
                bias=rng.random() < 0.7, keep=many, fresh=rng.choice([0, 0, seqs // 3]))


def _lengths(case):
    """Tokens of each sequence, from the case alone: one sequence has the longest run, the others anything below."""
    n, longest = case["seqs"], case["longest"]
    if longest == 1:
        return [1] * n
    r = random.Random(n * 1000003 + longest)
    lens = [r.randint(0, longest) for _ in range(n)]
    lens[r.randrange(n)] = longest
    return lens


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "recurrent":
        lens = _lengths(case)
        t, d, hv, h = sum(lens), case["d"], case["h_v"], case["h_qk"]
        fresh, live = case["fresh"], sum(x > 0 for x in lens)
        states = sum(x > 0 for x in lens[fresh:]) + (t if case["keep"] else live)
        return {"bytes": states * hv * d * d * 4 + t * (2 * h + 2 * hv) * d * size + t * hv * 8,
                "flops": t * hv * 7 * d * d}
    if case["op"] == "qk_rope":
        rows, d = case["tokens"] * (case["h_q"] + case["h_k"]), case["d"]
        passes = 2 if case["way"] == "fwd" or case["norm"] == "none" else 3
        return {"bytes": passes * rows * d * size + 4 * case["tokens"], "flops": rows * d * (7 if passes == 2 else 14)}
    lens = _lengths(case)
    t, c, w = sum(lens), 2 * case["q"] + case["v"], case["width"]
    rows = sum(x > 0 for x in lens[case["fresh"]:]) + (t if case["keep"] else sum(x > 0 for x in lens))
    return {"bytes": 2 * t * c * size + rows * (w - 1) * c * size + c * (w + 1) * 4, "flops": t * c * (2 * w + 4)}


# ------------------------------------------------------------------------------------------ inputs


def _frequencies(case):
    """Angle per position of each pair (float64, radians) and the magnitude of the rotated part."""
    r, base, factor = case["rotary"], 10000.0, 4.0
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "blend":  # slow pairs interpolated, fast ones kept, a ramp over the pair's index between
        at = lambda turns: r * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    s = dict(case=case)
    if case["op"] == "qk_rope":
        t, hq, hk, d = case["tokens"], case["h_q"], case["h_k"], case["d"]

        def rows():
            if case["packed"]:  # q and k are parts of one projection's output, values behind them
                x = normal(t, (hq + 2 * hk) * d).to(dt)
                return x[:, :hq * d].view(t, hq, d), x[:, hq * d:(hq + hk) * d].view(t, hk, d)
            return normal(t, hq, d).to(dt), normal(t, hk, d).to(dt)

        s["q"], s["k"] = rows()
        if case["way"] == "bwd":
            s["dy_q"], s["dy_k"] = normal(t, hq, d).to(dt), normal(t, hk, d).to(dt)
        s["w_q"] = 1 + 0.1 * normal(d) if case["norm"] == "rms" else None
        s["w_k"] = 1 + 0.1 * normal(d) if case["norm"] == "rms" else None
        longest = case["longest"]
        if t >= 4 * longest or case["way"] == "bwd" or t > 4096:  # documents, each from position 0
            s["positions"] = (torch.arange(t, device=DEV) % longest).to(torch.int32)
        else:  # sequences under way, each at a place of its own
            s["positions"] = torch.randint(0, longest, (t,), generator=gen, device=DEV, dtype=torch.int32)
        f, m = _frequencies(case)
        if own:
            import gated_deltanet_fwd_amd as G

            kw = {"none": {}, "linear": dict(scaling="linear", factor=4.0),
                  "blend": dict(scaling="yarn", factor=4.0, original_length=32768)}[case["scaling"]]
            turns, m = G.gdn_rope_frequencies(case["rotary"], base=10000.0, **kw)
            s["freqs"] = turns.to(DEV)
            s["plan"] = G.QkRopeProblem(t, hq, hk, d, dtype=dt, norm=case["norm"], rotary_dim=case["rotary"],
                                        interleaved=case["layout"] == "interleaved", magnitude=m)
        else:
            angle = torch.arange(longest, dtype=torch.float64, device=DEV)[:, None] * f.to(DEV)
            s["cos"], s["sin"] = (m * angle.cos()).float(), (m * angle.sin()).float()
        return s

    lens = _lengths(case)
    n, t, fresh = case["seqs"], sum(lens), case["fresh"]
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    slots = n + 1 + (t if case["keep"] else 0)
    order = torch.randperm(slots, generator=gen, device=DEV).to(torch.int32)
    s["slot_in"] = order[:n].clone()
    s["slot_in"][:fresh] = -1
    s["slot_out"] = torch.full_like(order[:n], -1) if case["keep"] else order[:n].clone()
    s["slot_tok"] = order[n:n + t].clone() if case["keep"] else None
    s["lens"], s["cu"] = lens, torch.tensor(cu, dtype=torch.int32, device=DEV)
    if case["op"] == "recurrent":
        h, hv, d = case["h_qk"], case["h_v"], case["d"]
        s["q"], s["k"], s["v"] = normal(t, h, d).to(dt), normal(t, h, d).to(dt), normal(t, hv, d).to(dt)
        if not case["l2norm"]:  # rows of about unit length, as the rule needs them
            s["q"], s["k"] = ((x.float() * d ** -0.5).to(dt) for x in (s["q"], s["k"]))
        s["beta"] = torch.sigmoid(normal(t, hv))
        s["g"] = torch.nn.functional.logsigmoid(normal(t, hv) + 3.0)
        s["states"] = 0.1 * normal(slots, hv, d, d)
    else:
        c, w = 2 * case["q"] + case["v"], case["width"]
        s["x"], s["windows"] = normal(t, c).to(dt), normal(slots, w - 1, c).to(dt)
        s["weight"] = normal(c, w) / w ** 0.5
        s["bias"] = 0.1 * normal(c) if case["bias"] else None
    if own:
        import gated_deltanet_fwd_amd as G

        host = None if case["longest"] == 1 else cu
        if case["op"] == "recurrent":
            s["plan"] = G.RecurrentProblem(n, case["h_qk"], case["h_v"], case["d"], slots, cu_seqlens_host=host, dtype=dt,
                                           l2norm=case["l2norm"])
        else:
            s["plan"] = G.ConvStepProblem(n, [case["q"], case["q"], case["v"]], slots, cu_seqlens_host=host,
                                          width=case["width"], dtype=dt)
    else:
        s["rows"] = _rows(case, lens, cu)
    return s


def _rows(case, lens, cu):
    """The plain forms' plan, made once for a batch's lengths: which rows each step reads."""
    if case["op"] == "recurrent":  # sequences longest first; tokens of step i, of the sequences that have them
        order = sorted(range(len(lens)), key=lambda n: -lens[n])
        steps = [[cu[n] + i for n in order if lens[n] > i] for i in range(case["longest"])]
        return dict(order=torch.tensor(order, device=DEV), steps=[torch.tensor(x, device=DEV) for x in steps])
    # conv_step: rows of the windows (first) and of x (after them) under each token's taps
    n, w = len(lens), case["width"]
    at = [[n * (w - 1) + cu[m] + i - j if i >= j else m * (w - 1) + (w - 1) + i - j for j in range(w - 1, -1, -1)]
          for m in range(n) for i in range(lens[m])]
    end = [[m * (w - 1) + lens[m] + j if lens[m] + j < w - 1 else n * (w - 1) + cu[m] + lens[m] + j - (w - 1)
            for j in range(w - 1)] for m in range(n)]
    return dict(taps=torch.tensor(at, dtype=torch.int64, device=DEV).view(-1, w),
                end=torch.tensor(end, dtype=torch.int64, device=DEV).view(-1, w - 1))


# ------------------------------------------------------------------------------------------ passes


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_recurrent(s):
    import gated_deltanet_fwd_amd as G

    o = G.gdn_recurrent(s["plan"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["slot_in"], s["slot_out"],
                        slot_tok=s["slot_tok"], cu_seqlens=None if s["case"]["longest"] == 1 else s["cu"])
    return {"o": o, "states": s["states"]}


def _own_qk_rope(s):
    import gated_deltanet_fwd_amd as G

    a = (s["plan"], s["q"], s["k"], s["positions"], s["freqs"])
    if s["case"]["way"] == "fwd":
        q, k = G.gdn_qk_rope_fwd(*a, q_weight=s["w_q"], k_weight=s["w_k"])
        return {"q": q, "k": k}
    g = G.gdn_qk_rope_bwd(*a, s["dy_q"], s["dy_k"], q_weight=s["w_q"], k_weight=s["w_k"])
    return {"dq": g["dq"], "dk": g["dk"], "dq_weight": g["dq_weight"], "dk_weight": g["dk_weight"]}


def _own_conv_step(s):
    import gated_deltanet_fwd_amd as G

    y = G.gdn_conv_step(s["plan"], s["x"], s["weight"], s["bias"], s["windows"], s["slot_in"], s["slot_out"],
                        slot_tok=s["slot_tok"], cu_seqlens=None if s["case"]["longest"] == 1 else s["cu"])
    return {"q": y[0], "k": y[1], "v": y[2], "windows": s["windows"]}


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _plain_recurrent(s):
    c, plan, states = s["case"], s["rows"], s["states"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["l2norm"]:
        q, k = _unit(q), _unit(k)
    group = c["h_v"] // c["h_qk"]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    a, o = s["g"].exp(), torch.empty_like(v)
    slot = s["slot_in"][plan["order"]].long()
    S = states[slot.clamp(min=0)] * (slot >= 0)[:, None, None, None]
    for rows in plan["steps"]:
        m = rows.numel()
        now, kt = S[:m], k[rows]
        now *= a[rows][:, :, None, None]
        u = s["beta"][rows][:, :, None] * (v[rows] - torch.matmul(kt[:, :, None], now)[:, :, 0])
        now += kt[..., None] * u[:, :, None]
        o[rows] = torch.matmul(q[rows][:, :, None], now)[:, :, 0]
        if c["keep"]:
            states[s["slot_tok"][rows].long()] = now
    if not c["keep"]:
        out = s["slot_out"][plan["order"]].long()
        states[out] = S
    return {"o": o.to(s["v"].dtype), "states": states}


def _turn(x, cos, sin, case):
    """The rotation of the first `rotary` values of each head by the angles whose cosines and sines are given."""
    r = case["rotary"]
    if case["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., r:]], -1)


def _plain_qk_rope(s):
    c, at = s["case"], s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    mean = c["d"] if c["norm"] == "rms" else 1

    def inverse(x):
        return torch.rsqrt((x * x).sum(-1, keepdim=True) / mean + 1e-6)

    def forward(x, w):
        x = x.float()
        if c["norm"] != "none":
            x = x * inverse(x)
        return _turn(x * w if w is not None else x, cos, sin, c).to(s["q"].dtype)

    def backward(x, w, dy):
        x, dz = x.float(), _turn(dy.float(), cos, -sin, c)
        if c["norm"] == "none":
            return dz.to(s["q"].dtype), None
        r = inverse(x)
        n = x * r
        dw = (dz * n).sum((0, 1)) if w is not None else None
        dn = dz * w if w is not None else dz
        return (r * (dn - n * ((n * dn).sum(-1, keepdim=True) / mean))).to(s["q"].dtype), dw

    if c["way"] == "fwd":
        return {"q": forward(s["q"], s["w_q"]), "k": forward(s["k"], s["w_k"])}
    dq, dwq = backward(s["q"], s["w_q"], s["dy_q"])
    dk, dwk = backward(s["k"], s["w_k"], s["dy_k"])
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def _plain_conv_step(s):
    c, plan, windows = s["case"], s["rows"], s["windows"]
    slot = s["slot_in"].long()
    past = windows[slot.clamp(min=0)] * (slot >= 0)[:, None, None]
    every = torch.cat([past.flatten(0, 1), s["x"]])
    rows = every[plan["taps"]]  # [tokens, taps, channels]
    y = (rows.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    y = (y / (1 + torch.exp(-y))).to(s["x"].dtype)
    if c["keep"]:
        windows[s["slot_tok"].long()] = rows[:, 1:]
    else:
        windows[s["slot_out"].long()] = every[plan["end"]]
    q, k, v = y.split([c["q"], c["q"], c["v"]], 1)
    return {"q": q, "k": k, "v": v, "windows": windows}


_OWN = {"recurrent": _own_recurrent, "qk_rope": _own_qk_rope, "conv_step": _own_conv_step}
_PLAIN = {"recurrent": _plain_recurrent, "qk_rope": _plain_qk_rope, "conv_step": _plain_conv_step}


# ------------------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"recurrent": _exact_recurrent, "qk_rope": _exact_qk_rope, "conv_step": _exact_conv_step}[case["op"]](s, case)


def _exact_recurrent(s, case):
    """S_t = a S + beta k (v - a S^T k)^T, o = S_t^T q, each sequence's heads together, by the definition."""
    group = case["h_v"] // case["h_qk"]
    q, k, v, g, beta = (s[x].double() for x in ("q", "k", "v", "g", "beta"))
    if case["l2norm"]:
        q, k = (x / ((x ** 2).sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
    head = torch.arange(case["h_v"], device=DEV) // group
    o, states = torch.empty_like(v), s["states"].double()
    if case["longest"] == 1 and case["fresh"] == 0:  # one token of every sequence
        slot = s["slot_in"].long()
        S = torch.exp(g)[..., None, None] * states[slot]
        kh, qh = k[:, head], q[:, head]
        u = beta[..., None] * (v - torch.einsum("nhkv,nhk->nhv", S, kh))
        S += torch.einsum("nhk,nhv->nhkv", kh, u)
        states[slot] = S
        return {"o": torch.einsum("nhkv,nhk->nhv", S, qh), "states": states}
    given, at = states.clone(), 0
    slot_in, slot_out = s["slot_in"].tolist(), s["slot_out"].tolist()
    slot_tok = s["slot_tok"].tolist() if case["keep"] else None
    for n, length in enumerate(s["lens"]):
        S = given[slot_in[n]].clone() if slot_in[n] >= 0 else torch.zeros_like(given[0])
        for i in range(at, at + length):
            kh = k[i, head]
            S = S * torch.exp(g[i])[:, None, None]
            u = beta[i][:, None] * (v[i] - (S * kh[..., None]).sum(1))
            S = S + kh[..., None] * u[:, None]
            o[i] = (S * q[i, head][..., None]).sum(1)
            if slot_tok:
                states[slot_tok[i]] = S
        at += length
        if slot_out[n] >= 0:
            states[slot_out[n]] = S
    return {"o": o, "states": states}


def _exact_qk_rope(s, case):
    """The norm, then each pair as a complex number times m e^(i angle); gradients by differentiation."""
    f, m = _frequencies(case)
    r = case["rotary"]
    turn = torch.polar(torch.full((), m, dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None, None] * f.to(DEV))

    def y(x, w):
        if case["norm"] == "rms":
            x = x / ((x ** 2).mean(-1, keepdim=True) + 1e-6).sqrt()
        elif case["norm"] == "l2":
            x = x / ((x ** 2).sum(-1, keepdim=True) + 1e-6).sqrt()
        x = x if w is None else x * w
        if case["layout"] == "interleaved":
            z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * turn
            z = torch.stack([z.real, z.imag], -1).flatten(-2)
        else:
            z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, x[..., r:]], -1)

    q, k, wq, wk = (x if x is None else x.double() for x in (s["q"], s["k"], s["w_q"], s["w_k"]))
    if case["way"] == "fwd":
        return {"q": y(q, wq), "k": y(k, wk)}
    got = {}
    for name, x, w, dy in (("dq", q, wq, s["dy_q"]), ("dk", k, wk, s["dy_k"])):
        x = x.detach().requires_grad_()
        w = w if w is None else w.detach().requires_grad_()
        torch.autograd.backward(y(x, w), dy.double())
        got[name], got[name + "_weight"] = x.grad, None if w is None else w.grad
    return got


def _exact_conv_step(s, case):
    """Each sequence's window and tokens in one row of rows, the taps slid along it."""
    w, weight = case["width"], s["weight"].double()
    x, windows = s["x"].double(), s["windows"].double()
    given = windows.clone()
    y, at = torch.empty_like(x), 0
    slot_in, slot_out = s["slot_in"].tolist(), s["slot_out"].tolist()
    slot_tok = s["slot_tok"].tolist() if case["keep"] else None
    for n, length in enumerate(s["lens"]):
        past = given[slot_in[n]] if slot_in[n] >= 0 else torch.zeros_like(given[0])
        line = torch.cat([past, x[at:at + length]])
        for i in range(length):
            pre = torch.einsum("wc,cw->c", line[i:i + w], weight)
            pre = pre if s["bias"] is None else pre + s["bias"].double()
            y[at + i] = pre * torch.sigmoid(pre)
            if slot_tok:
                windows[slot_tok[at + i]] = line[i + 1:i + w]
        at += length
        if slot_out[n] >= 0:
            windows[slot_out[n]] = line[length:]
    q, k, v = y.split([case["q"], case["q"], case["v"]], 1)
    return {"q": q, "k": k, "v": v, "windows": windows}
