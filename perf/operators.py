"""The workloads of the operators beside the gated delta rule, and their plain forms.

Three operators: the gated linear recurrence (forward, training step, one
decode token), rotary positions, and group norm with an activation, channels
last. ``run`` computes them with elementary torch operations in fp32 (fp64
where angles need it) or, with ``own`` set, through ``libgdn.so``; ``exact``
gives the values in fp64, written from the definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
MOST = 131072 * 4096    # token x channel elements of the largest case


# ------------------------------------------------------------------- cases
def listed():
    return [
        # serving: one token for a handful of sequences (latency), and for a full batch
        {"name": "step_8", "op": "step", "B": 8, "D": 4096, "dtype": "bf16"},
        {"name": "step_512", "op": "step", "B": 512, "D": 4096, "dtype": "fp16"},
        # prefill of one layer at batch 2, continuing from a state
        {"name": "recur_layer", "op": "recur", "B": 2, "T": 2048, "D": 1536, "seqs": 0, "dtype": "bf16"},
        # prefill of one long context: 32 heads of 128 channels
        {"name": "recur_long", "op": "recur", "B": 1, "T": 131072, "D": 4096, "seqs": 0, "dtype": "bf16"},
        # training on 16 packed sequences of ragged lengths
        {"name": "recur_train_packed", "op": "recur_train", "B": 1, "T": 65536, "D": 4096, "seqs": 16, "dtype": "bf16"},
        # a small fp32 training step of odd length (6 heads of 64 channels)
        {"name": "recur_train_small", "op": "recur_train", "B": 2, "T": 100, "D": 384, "seqs": 0, "dtype": "fp32"},
        # serving: q and k of one token per sequence at far positions, a quarter of the head rotated
        {"name": "rotary_decode", "op": "rotary", "B": 64, "T": 1, "Hq": 32, "Hk": 16, "d": 128, "rot": 32,
         "layout": "half", "scaling": "by_parts", "inverse": False, "far": 1000000, "dtype": "bf16"},
        # prefill of one long context, the whole head, table scaled for long contexts
        {"name": "rotary_long", "op": "rotary", "B": 1, "T": 131072, "Hq": 16, "Hk": 16, "d": 128, "rot": 128,
         "layout": "half", "scaling": "by_parts", "inverse": False, "far": 0, "dtype": "bf16"},
        # the gradient of q and k (the inverse rotation) in a training step, interleaved pairs
        {"name": "rotary_grad", "op": "rotary", "B": 2, "T": 2048, "Hq": 6, "Hk": 6, "d": 256, "rot": 64,
         "layout": "interleaved", "scaling": "plain", "inverse": True, "far": 0, "dtype": "fp16"},
        # per-token, per-head output norm over a long context
        {"name": "norm_long", "op": "norm", "N": 131072, "L": 1, "C": 4096, "G": 32, "act": "silu", "dtype": "bf16"},
        # the same in a training step over packed tokens
        {"name": "norm_train", "op": "norm_train", "N": 65536, "L": 1, "C": 4096, "G": 32, "act": "silu", "dtype": "fp16"},
        # training with statistics over whole rows of 2048 positions, 6 groups of 256 channels
        {"name": "norm_rows_train", "op": "norm_train", "N": 2, "L": 2048, "C": 1536, "G": 6, "act": "silu", "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "recur", "recur_train", "rotary", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "step":
        return {"op": op, "B": _spread(rng, 1, 2048), "D": _spread(rng, 64, 8192), "dtype": dtype}
    if op in ("recur", "recur_train"):
        most = MOST // (2 if dtype == "fp32" else 1) // (4 if op == "recur_train" else 1)
        d = _spread(rng, 64, 8192)
        d = d // 8 * 8 if rng.random() < 0.7 else d
        b = _spread(rng, 1, 16)
        t = min(_spread(rng, 16, 131072), most // (b * d))
        seqs = rng.randint(2, 64) if b == 1 and t >= 256 else 0
        return {"op": op, "B": b, "T": t, "D": d, "seqs": seqs, "dtype": dtype}
    if op == "rotary":
        d = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([d, d, d // 2, d // 4])
        hq, hk = _spread(rng, 1, 32), rng.choice([0, 1, 2, 4, 8])
        b = _spread(rng, 1, 64)
        most = MOST // (2 if dtype == "fp32" else 1)
        t = max(1, min(_spread(rng, 1, 65536), most // (b * (hq + hk) * d)))
        return {"op": op, "B": b, "T": t, "Hq": hq, "Hk": hk, "d": d, "rot": rot,
                "layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["plain", "linear", "by_parts"]),
                "inverse": rng.random() < 0.5, "far": rng.choice([0, 4000, 1000000]), "dtype": dtype}
    most = MOST // (2 if dtype == "fp32" else 1) // (4 if op == "norm_train" else 1)
    g = _spread(rng, 1, 64)
    c = g * rng.choice([8, 16, 24, 40, 64, 65, 128, 256])
    l = 1 if rng.random() < 0.5 else _spread(rng, 2, 16384)
    l = min(l, max(1, most // c))
    n = min(_spread(rng, 1, 131072) if l == 1 else _spread(rng, 1, 64), max(1, most // (c * l)))
    return {"op": op, "N": n, "L": l, "C": c, "G": g, "act": rng.choice(["silu", "silu", "none"]), "dtype": dtype}


def _lengths(case):
    """The packed sequences' lengths of a case, each at least one token."""
    n, total = case["seqs"], case["T"]
    rng = random.Random(n * 1000003 + total)
    cuts = sorted(rng.sample(range(1, total), n - 1))
    return [hi - lo for lo, hi in zip([0] + cuts, cuts + [total])]


def _inverse_frequencies(case, device):
    """fp64 radians per position of every rotated pair."""
    rot, scaling = case["rot"], case["scaling"]
    f = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=device) / rot)
    if scaling == "linear":
        return f / 4.0
    if scaling == "by_parts":
        # pairs that turn more than 4 times over the original 8192 positions stay, those that turn less than once
        # are interpolated by the factor 16, those between are blended
        keep = ((8192.0 * f / (2.0 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f * keep + f / 16.0 * (1.0 - keep)
    return f


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, act = case["op"], DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=act):
        return torch.randn(shape, generator=gen, dtype=dtype, device=dev).mul_(std).add_(mean)

    s = {"case": dict(case), "op": op}
    if op in ("step", "recur", "recur_train"):
        B, D = case["B"], case["D"]
        T, seqs = case.get("T", 1), case.get("seqs", 0)
        s["x"], s["a"], s["b"] = normal(B, T, D), normal(B, T, D), normal(B, T, D)
        # decay rates 1 to 16, time constants 0.001 to 0.1: from a few tokens to about a thousand of memory
        u = torch.rand((2, D), generator=gen, dtype=torch.float32, device=dev)
        s["A_log"] = torch.log(1.0 + 15.0 * u[0])
        dt = torch.exp(u[1] * math.log(100.0) + math.log(0.001))
        s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))
        N = seqs or B
        s["state"] = normal(N, D, dtype=torch.float32)
        s["cu"] = s["first"] = s["last"] = None
        if seqs:
            ends = torch.tensor(_lengths(case), dtype=torch.int64, device=dev).cumsum(0)
            s["cu"] = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
            s["first"], s["last"] = s["cu"][:-1].long(), ends - 1
        if op == "recur_train":
            s["dout"], s["dfinal"] = normal(B, T, D), normal(N, D, dtype=torch.float32)
        if own:
            from linear_attention_sequence_qkv_gb300 import gdn
            s["gdn"] = gdn
            s["desc"] = gdn.recurrence_desc_for(s["x"], s["a"], s["b"], s["cu"])
            if op == "step":
                s["out"] = torch.empty_like(s["x"])
            else:
                s["bufs"] = gdn.alloc_recurrence(s["desc"], dev, want_chunk_states=op == "recur_train")
            if op == "recur_train":
                s["grads"] = gdn.alloc_recurrence_grads(s["desc"], dev)
    elif op == "rotary":
        B, T, Hq, Hk, d = (case[k] for k in ("B", "T", "Hq", "Hk", "d"))
        # q and k are views into one projection's output
        s["qk"] = normal(B, T, (Hq + Hk) * d)
        s["q"], s["k"] = s["qk"][..., :Hq * d], s["qk"][..., Hq * d:] if Hk else None
        s["inv_freq"] = _inverse_frequencies(case, dev)
        s["offsets"] = None
        if case["far"]:
            s["offsets"] = torch.randint(0, case["far"], (B,), generator=gen, device=dev).to(torch.int32)
        if own:
            from linear_attention_sequence_qkv_gb300 import gdn
            s["gdn"] = gdn
            scaling = {"plain": {}, "linear": {"scaling": "linear", "factor": 4.0},
                       "by_parts": {"scaling": "by_parts", "factor": 16.0, "low": 1.0, "high": 4.0, "original": 8192}}
            s["table"] = gdn.rotary_table(case["rot"], 10000.0, device=dev, **scaling[case["scaling"]])
            s["q_out"] = torch.empty((B, T, Hq * d), dtype=act, device=dev)
            s["k_out"] = torch.empty((B, T, Hk * d), dtype=act, device=dev) if Hk else None
            s["desc"] = gdn.rotary_desc_for(s["q"], s["k"], s["q_out"], s["k_out"], d=d, rot=case["rot"],
                                            layout=case["layout"], inverse=case["inverse"])
            s["ws"] = torch.empty(gdn.gdn_rotary_workspace_bytes(s["desc"]), dtype=torch.uint8, device=dev)
    else:
        N, L, C, G = (case[k] for k in ("N", "L", "C", "G"))
        s["x"] = normal(N, L, C)
        # a recurrent layer's heads differ in level and scale
        s["x"] = s["x"] * normal(C, std=0.3, mean=1.0) + normal(C, std=0.5)
        s["weight"], s["bias"] = normal(C, std=0.1, mean=1.0), normal(C, std=0.1)
        if op == "norm_train":
            s["dout"] = normal(N, L, C)
        if own:
            from linear_attention_sequence_qkv_gb300 import gdn
            s["gdn"] = gdn
            s["desc"] = gdn.group_norm_desc_for(s["x"], s["weight"], groups=G, act=case["act"], eps=1e-5)
            s["bufs"] = gdn.alloc_group_norm(s["desc"], dev)
            if op == "norm_train":
                s["grads"] = gdn.alloc_group_norm_grads(s["desc"], dev)
    return s


# -------------------------------------------------------------- plain forms
def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _gates(s):
    """decay, its logarithm, d(-log decay)/d(a), write scale and write gate of every token, fp32."""
    z = s["a"].float() + s["dt_bias"]
    rate = torch.exp(s["A_log"])
    softplus = z.clamp(min=0.0) + torch.log1p(torch.exp(-z.abs()))
    g = -rate * softplus
    return torch.exp(g), g, rate * _sigmoid(z), torch.sqrt(-torch.expm1(2.0 * g)), _sigmoid(s["b"].float())


def _scan(decay, write):
    """h_t = decay_t h_{t-1} + write_t along dim 1: pairs of tokens are combined, the half-length
    recurrence over the pairs gives every second h, one more step the others."""
    T = decay.shape[1]
    if T == 1:
        return write
    m = T // 2
    a0, a1 = decay[:, 0:2 * m:2], decay[:, 1::2]
    odd = _scan(a0 * a1, a1 * write[:, 0:2 * m:2] + write[:, 1::2])
    h = torch.empty_like(write)
    h[:, 1::2] = odd
    h[:, :1] = write[:, :1]
    h[:, 2::2] = decay[:, 2::2] * odd[:, :(T - 1) // 2] + write[:, 2::2]
    return h


def _recur(s):
    """(h, decay inside sequences, everything _gates gives) with the initial state written at each first token."""
    gates = _gates(s)
    alpha, write = gates[0].clone(), gates[3] * gates[4] * s["x"].float()
    if s["cu"] is None:
        write[:, 0] += alpha[:, 0] * s["state"]
        alpha[:, 0] = 0.0
    else:
        write[0, s["first"]] += alpha[0, s["first"]] * s["state"]
        alpha[0, s["first"]] = 0.0
    return _scan(alpha, write), alpha, gates


def _ends(s, h):
    return h[:, -1] if s["cu"] is None else h[0, s["last"]]


def _plain_recur_train(s):
    h, inside, (alpha, g, rate, scale, beta) = _recur(s)
    act, x = s["x"].dtype, s["x"].float()
    into = s["dout"].float().clone()
    if s["cu"] is None:
        into[:, -1] += s["dfinal"]
    else:
        into[0, s["last"]] += s["dfinal"]
    # delta_t = into_t + decay_{t+1} delta_{t+1}: the same scan from the last token
    after = torch.cat([inside[:, 1:], torch.zeros_like(inside[:, :1])], dim=1)
    delta = _scan(after.flip(1), into.flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], dim=1)
    if s["cu"] is None:
        before[:, 0] = s["state"]
    else:
        before[0, s["first"]] = s["state"]
    dg = delta * (alpha * before - beta * x * alpha * alpha / scale)
    da = -dg * rate
    dstate = alpha[:, 0] * delta[:, 0] if s["cu"] is None else alpha[0, s["first"]] * delta[0, s["first"]]
    return {"out": h.to(act), "final": _ends(s, h), "dx": (delta * scale * beta).to(act), "da": da.to(act),
            "db": (delta * scale * beta * (1.0 - beta) * x).to(act), "dA_log": (dg * g).sum((0, 1)),
            "ddt_bias": da.sum((0, 1)), "dstate": dstate}


def _plain_rotary(s):
    c = s["case"]
    d, rot = c["d"], c["rot"]
    B, T = s["q"].shape[:2]
    at = torch.arange(T, dtype=torch.float64, device=s["q"].device).expand(B, T)
    if s["offsets"] is not None:
        at = at + s["offsets"].double()[:, None]
    angle = (at[..., None] * s["inv_freq"])[:, :, None]          # [B, T, 1, rot / 2]
    co, si = torch.cos(angle).float(), torch.sin(angle).float()
    si = -si if c["inverse"] else si

    def turn(x):
        if x is None:
            return None
        y = x.float().view(B, T, -1, d)
        if c["layout"] == "half":
            x1, x2 = y[..., :rot // 2], y[..., rot // 2:rot]
            turned = torch.cat([x1 * co - x2 * si, x2 * co + x1 * si], dim=-1)
        else:
            x1, x2 = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([x1 * co - x2 * si, x2 * co + x1 * si], dim=-1).flatten(-2)
        return torch.cat([turned, y[..., rot:]], dim=-1).view(B, T, -1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _plain_norm(s):
    c, x = s["case"], s["x"]
    N, L, C = x.shape
    y = x.float().view(N, L, c["G"], -1)
    y = y - y.mean((1, 3), keepdim=True)
    rstd = torch.rsqrt((y * y).mean((1, 3), keepdim=True) + 1e-5)
    xh = (y * rstd).view(N, L, C)
    w = s["weight"].float()
    z = xh * w + s["bias"].float()
    sg = _sigmoid(z) if c["act"] == "silu" else torch.ones_like(z)
    out = (z * sg).to(x.dtype)
    if s["op"] == "norm":
        return {"out": out}
    dz = s["dout"].float() * sg
    if c["act"] == "silu":
        dz = dz * (1.0 + z * (1.0 - sg))
    t, xg = (dz * w).view(N, L, c["G"], -1), xh.view(N, L, c["G"], -1)
    dx = rstd * (t - t.mean((1, 3), keepdim=True) - xg * (t * xg).mean((1, 3), keepdim=True))
    return {"out": out, "dx": dx.view(N, L, C).to(x.dtype), "dweight": (dz * xh).sum((0, 1)), "dbias": dz.sum((0, 1))}


def _plain(s):
    op = s["op"]
    if op == "step":
        alpha, _, _, scale, beta = _gates(s)
        s["state"].copy_(alpha[:, 0] * s["state"] + (scale * beta * s["x"].float())[:, 0])
        return {"out": s["state"].to(s["x"].dtype)[:, None], "state": s["state"]}
    if op == "recur":
        h = _recur(s)[0]
        return {"out": h.to(s["x"].dtype), "final": _ends(s, h)}
    if op == "recur_train":
        return _plain_recur_train(s)
    if op == "rotary":
        return _plain_rotary(s)
    return _plain_norm(s)


def run(state):
    s = state
    if not own:
        return _plain(s)
    gdn, op, d = s["gdn"], s["op"], s["desc"]
    if op == "step":
        gdn.gdn_recurrence_step(d, s["x"], s["a"], s["b"], s["A_log"], s["dt_bias"], s["state"], s["out"])
        return {"out": s["out"], "state": s["state"]}
    if op in ("recur", "recur_train"):
        f = s["bufs"]
        gdn.gdn_recurrence_forward(d, s["x"], s["a"], s["b"], s["A_log"], s["dt_bias"], s["cu"], s["state"], f.out,
                                   f.final_state, f.chunk_states, f.workspace, f.ws_bytes)
        if op == "recur":
            return {"out": f.out, "final": f.final_state}
        r = s["grads"]
        gdn.gdn_recurrence_backward(d, s["x"], s["a"], s["b"], s["A_log"], s["dt_bias"], s["cu"], s["state"],
                                    f.chunk_states, s["dout"], s["dfinal"], r.dx, r.da, r.db, r.dA_log, r.ddt_bias,
                                    r.dinitial_state, r.workspace, r.ws_bytes)
        return {"out": f.out, "final": f.final_state, "dx": r.dx, "da": r.da, "db": r.db, "dA_log": r.dA_log,
                "ddt_bias": r.ddt_bias, "dstate": r.dinitial_state}
    if op == "rotary":
        gdn.gdn_rotary(d, s["q"], s["k"], s["table"], None, None, s["offsets"], s["q_out"], s["k_out"], s["ws"],
                       s["ws"].numel())
        return {"q": s["q_out"], "k": s["k_out"]}
    f = s["bufs"]
    gdn.gdn_group_norm_forward(d, s["x"], s["weight"], s["bias"], f.out, f.mean, f.rstd, f.workspace, f.ws_bytes)
    if op == "norm":
        return {"out": f.out}
    r = s["grads"]
    gdn.gdn_group_norm_backward(d, s["x"], s["weight"], s["bias"], f.mean, f.rstd, s["dout"], r.dx, r.dweight, r.dbias,
                                r.workspace, r.ws_bytes)
    return {"out": f.out, "dx": r.dx, "dweight": r.dweight, "dbias": r.dbias}


# ------------------------------------------------------ work and exact values
def work(case):
    op, es = case["op"], BYTES[case["dtype"]]
    if op == "step":
        n = case["B"] * case["D"]
        return {"bytes": n * (4 * es + 8) + 8 * case["D"], "flops": 15 * n}
    if op in ("recur", "recur_train"):
        D = case["D"]
        n, states = case["B"] * case["T"] * D, (case["seqs"] or case["B"]) * D
        if op == "recur":
            return {"bytes": 4 * es * n + 8 * D + 8 * states, "flops": 15 * n}
        return {"bytes": 8 * es * n + 16 * D + 16 * states, "flops": 45 * n}
    if op == "rotary":
        heads = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * es * heads * case["d"], "flops": 3 * heads * case["rot"]}
    n = case["N"] * case["L"] * case["C"]
    if op == "norm":
        return {"bytes": 2 * es * n + 2 * es * case["C"], "flops": 12 * n}
    return {"bytes": 4 * es * n + (2 * es + 8) * case["C"], "flops": 35 * n}


def _exact_recur(case, s):
    """Token by token in fp64; the gates' derivatives by torch's own differentiation, the state's by the adjoint loop."""
    train = case["op"] == "recur_train"
    leaf = {k: s[k].double().requires_grad_(train) for k in ("x", "a", "b", "A_log", "dt_bias")}
    g = -leaf["A_log"].exp() * torch.nn.functional.softplus(leaf["a"] + leaf["dt_bias"], threshold=700.0)
    alpha, write = g.exp(), (-(2.0 * g).expm1()).sqrt() * torch.sigmoid(leaf["b"]) * leaf["x"]
    B, T, D = s["x"].shape
    first, last = ({0: None}, {T - 1: None}) if s["cu"] is None else (
        {t: n for n, t in enumerate(s["first"].tolist())}, {t: n for n, t in enumerate(s["last"].tolist())})
    of = lambda v, n: v.double() if n is None else v[n:n + 1].double()  # noqa: E731
    al, wr, state = alpha.detach(), write.detach(), s["state"]
    h, ends = torch.empty_like(wr), {}
    for t in range(T):
        before = of(state, first[t]) if t in first else h[:, t - 1]
        torch.addcmul(wr[:, t], al[:, t], before, out=h[:, t])
        if t in last:
            ends[last[t]] = h[:, t].clone()
    final = torch.cat([ends[n] for n in sorted(ends, key=lambda n: n or 0)])
    if not train:
        return {"out": h, "final": final}
    delta, dalpha, dstate = torch.empty_like(h), torch.empty_like(h), {}
    for t in reversed(range(T)):
        d = s["dout"][:, t].double()
        if t in last:
            d = d + of(s["dfinal"], last[t])
        else:
            d = torch.addcmul(d, al[:, t + 1], delta[:, t + 1])
        delta[:, t] = d
        if t in first:
            dstate[first[t]] = al[:, t] * d
            dalpha[:, t] = d * of(state, first[t])
        else:
            torch.mul(d, h[:, t - 1], out=dalpha[:, t])
    grads = torch.autograd.grad([alpha, write], list(leaf.values()), [dalpha, delta])
    return {"out": h, "final": final, "dx": grads[0], "da": grads[1], "db": grads[2], "dA_log": grads[3],
            "ddt_bias": grads[4], "dstate": torch.cat([dstate[n] for n in sorted(dstate, key=lambda n: n or 0)])}


def _exact_rotary(case, s):
    """Each pair as a complex number times e^{i angle}."""
    d, rot, half = case["d"], case["rot"], case["rot"] // 2
    B, T = s["q"].shape[:2]
    at = torch.arange(T, device=s["q"].device)[None] + (0 if s["offsets"] is None else s["offsets"].long()[:, None])
    angle = at.double()[..., None] * s["inv_freq"] * (-1.0 if case["inverse"] else 1.0)
    unit = torch.polar(torch.ones_like(angle), angle)[:, :, None]
    idx = torch.arange(rot, device=s["q"].device)
    pairs = idx.view(2, half).t() if case["layout"] == "half" else idx.view(half, 2)

    def turn(x):
        if x is None:
            return None
        y = x.double().reshape(B, T, -1, d).clone()
        z = torch.view_as_real(torch.complex(y[..., pairs[:, 0]], y[..., pairs[:, 1]]) * unit)
        y[..., pairs[:, 0]], y[..., pairs[:, 1]] = z[..., 0], z[..., 1]
        return y.reshape(B, T, -1)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _exact_norm(case, s):
    train = case["op"] == "norm_train"
    x, w, b = (s[k].double().requires_grad_(train) for k in ("x", "weight", "bias"))
    N, L, C = x.shape
    y = x.view(N, L, case["G"], -1)
    var, mean = torch.var_mean(y, dim=(1, 3), keepdim=True, correction=0)
    z = ((y - mean) / (var + 1e-5).sqrt()).view(N, L, C) * w + b
    out = torch.nn.functional.silu(z) if case["act"] == "silu" else z
    if not train:
        return {"out": out}
    dx, dw, db = torch.autograd.grad(out, [x, w, b], s["dout"].double())
    return {"out": out.detach(), "dx": dx, "dweight": dw, "dbias": db}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "step":
        g = -s["A_log"].double().exp() * torch.nn.functional.softplus(s["a"].double() + s["dt_bias"].double(), threshold=700.0)
        write = (-(2.0 * g).expm1()).sqrt() * torch.sigmoid(s["b"].double()) * s["x"].double()
        h = g.exp() * s["state"].double()[:, None] + write
        return {"out": h, "state": h[:, 0]}
    if op in ("recur", "recur_train"):
        with torch.set_grad_enabled(op == "recur_train"):
            return _exact_recur(case, s)
    return _exact_rotary(case, s) if op == "rotary" else _exact_norm(case, s)
