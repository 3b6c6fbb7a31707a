"""The workloads of the attention layers that stand between delta rule layers, and their plain forms.

Four operators: the norm of every head of q and k with the rotary positions (forward, training step),
causal attention over a window with a few first tokens that stay visible (forward, training step), the
same for one new token per sequence over a cache of fixed size, and the filling of that cache from a
prefill. ``run`` computes them with elementary torch operations in fp32 (fp64 for angles) or, with
``own`` set, through ``libgdn.so``; ``exact`` gives the values in fp64, written from the definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
EPS = 1e-6
MOST_NORM = 131072 * 48 * 128      # elements of q and k of the largest norm
MOST_PAIRS = 131072 * 2048 * 32    # (query, key) pairs over all heads of the largest attention
MOST_CACHE = 256 * 8 * 4100 * 128  # elements of the largest cache of keys
MOST_EXACT = 3.5e12                # operations that exact() spends on a case in fp64 at most
MOST_BLOCKS = 12000                # and blocks of scores that it goes through
BAND = 1024                        # queries whose scores the plain form holds at a time


# ------------------------------------------------------------------- cases
def listed():
    return [
        # serving: q and k of one token per sequence at far positions, a quarter of the head rotated
        {"name": "norm_step", "op": "norm", "B": 64, "T": 1, "Hq": 32, "Hk": 16, "d": 128, "rot": 32,
         "layout": "half", "far": 1000000, "dtype": "bf16"},
        # prefill of one long context: 32 heads of queries, 16 of keys
        {"name": "norm_long", "op": "norm", "B": 1, "T": 131072, "Hq": 32, "Hk": 16, "d": 128, "rot": 128,
         "layout": "half", "far": 0, "dtype": "bf16"},
        # a training step at batch 2 with wide heads, interleaved pairs
        {"name": "norm_train", "op": "norm_train", "B": 2, "T": 2048, "Hq": 6, "Hk": 6, "d": 256, "rot": 64,
         "layout": "interleaved", "far": 0, "dtype": "fp16"},
        # prefill of a small layer at batch 2
        {"name": "attn_layer", "op": "attn", "B": 2, "T": 2048, "past": 0, "seqs": 0, "Hq": 6, "Hk": 6, "d": 128,
         "window": 512, "sinks": 4, "dtype": "bf16"},
        # prefill of one long context
        {"name": "attn_long", "op": "attn", "B": 1, "T": 131072, "past": 0, "seqs": 0, "Hq": 32, "Hk": 16, "d": 128,
         "window": 2048, "sinks": 4, "dtype": "bf16"},
        # serving: the prompts of 64 requests in one pass, of 1 to 8192 tokens
        {"name": "attn_packed", "op": "attn", "B": 1, "T": 65536, "past": 0, "seqs": 64, "Hq": 32, "Hk": 8, "d": 64,
         "window": 1024, "sinks": 4, "dtype": "fp16"},
        # training on 16 packed sequences of ragged lengths
        {"name": "attn_train_packed", "op": "attn_train", "B": 1, "T": 32768, "past": 0, "seqs": 16, "Hq": 32, "Hk": 16,
         "d": 128, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # a small fp32 training step of odd length
        {"name": "attn_train_small", "op": "attn_train", "B": 2, "T": 100, "past": 0, "seqs": 0, "Hq": 6, "Hk": 2, "d": 64,
         "window": 32, "sinks": 4, "dtype": "fp32"},
        # serving: one token for a handful of sequences (latency), and for a full batch
        {"name": "step_8", "op": "step", "B": 8, "Hq": 32, "Hk": 16, "d": 128, "window": 1024, "sinks": 4, "slack": 0,
         "far": 20000, "dtype": "bf16"},
        {"name": "step_256", "op": "step", "B": 256, "Hq": 32, "Hk": 8, "d": 128, "window": 4096, "sinks": 4, "slack": 0,
         "far": 20000, "dtype": "fp16"},
        # one more piece of 128 tokens of a few running prompts into their caches
        {"name": "fill_piece", "op": "fill", "B": 8, "T": 128, "seqs": 0, "Hk": 16, "d": 128, "window": 1024, "sinks": 4,
         "slack": 0, "far": 20000, "dtype": "bf16"},
        # the prompts of 64 requests into fresh caches
        {"name": "fill_packed", "op": "fill", "B": 1, "T": 262144, "seqs": 64, "Hk": 8, "d": 128, "window": 4096, "sinks": 4,
         "slack": 0, "far": 0, "dtype": "fp16"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "attn", "attn", "attn_train", "step", "step", "fill"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    wide = 2 if dtype == "fp32" else 1
    if op in ("norm", "norm_train"):
        d = rng.choice([64, 80, 96, 128, 192, 256])
        hq, hk = _spread(rng, 1, 32), rng.choice([0, 1, 2, 4, 8])
        b = _spread(rng, 1, 64)
        most = MOST_NORM // wide // (4 if op == "norm_train" else 1)
        t = max(1, min(_spread(rng, 1, 65536), most // (b * (hq + hk) * d)))
        return {"op": op, "B": b, "T": t, "Hq": hq, "Hk": hk, "d": d, "rot": rng.choice([d, d, d // 2, d // 4]),
                "layout": rng.choice(["half", "interleaved"]), "far": rng.choice([0, 4000, 1000000]), "dtype": dtype}
    hk, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 3, 4, 8])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128])
    window, sinks = _spread(rng, 16, 8192), rng.choice([0, 1, 4, 4, 64, 130])
    if op in ("step", "fill"):
        slack = rng.choice([0, 0, 1, 100])
        b = max(1, min(_spread(rng, 1, 512), MOST_CACHE // wide // (hk * d * (window + sinks + slack))))
        if op == "step":
            return {"op": op, "B": b, "Hq": hk * group, "Hk": hk, "d": d, "window": window, "sinks": sinks, "slack": slack,
                    "far": rng.choice([10, 4000, 1000000]), "dtype": dtype}
        b = min(b, 64)
        seqs = b if b > 1 and rng.random() < 0.5 else 0
        t = _spread(rng, 1, 16384)
        t = max(b, min(t * b, 262144)) if seqs else min(t, 262144 // b)
        return {"op": op, "B": 1 if seqs else b, "T": t, "seqs": seqs, "Hk": hk, "d": d, "window": window, "sinks": sinks,
                "slack": slack, "far": rng.choice([0, 10, 1000000]), "dtype": dtype}
    # exact fp32 sums have no matrix unit: such cases are smaller; a training step costs 3.5 forwards
    most = MOST_PAIRS * 128 // d // (16 if dtype == "fp32" else 1) // (4 if op == "attn_train" else 1)
    b = _spread(rng, 1, 16)
    t = _spread(rng, 1, 131072)
    seqs = rng.randint(2, 64) if b == 1 and t >= 256 else 0
    past = rng.choice([0, 0, 0, _spread(rng, 1, 4096)])
    t = max(1, min(t, most // (b * hk * group * min(window + sinks, t + past)), 262144 // b))
    return {"op": op, "B": b, "T": t, "past": past, "seqs": seqs if t >= 256 else 0, "Hq": hk * group, "Hk": hk, "d": d,
            "window": window, "sinks": sinks, "dtype": dtype}


def _lengths(case):
    """The packed sequences' lengths of a case, each at least one token."""
    n, total = case["seqs"], case["T"]
    rng = random.Random(n * 1000003 + total)
    cuts = sorted(rng.sample(range(1, total), n - 1))
    return [hi - lo for lo, hi in zip([0] + cuts, cuts + [total])]


def _spans(case):
    """(first query, queries, first key, keys) of every sequence, rows flattened."""
    past, q, k, spans = case.get("past", 0), 0, 0, []
    for n in (_lengths(case) if case["seqs"] else [case["T"]] * case["B"]):
        spans.append((q, n, k, n + past))
        q, k = q + n, k + n + past
    return spans


def _inverse_frequencies(case, device):
    """fp64 radians per position of every rotated pair."""
    return 10000.0 ** (-2.0 * torch.arange(case["rot"] // 2, dtype=torch.float64, device=device) / case["rot"])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, act, d = case["op"], DTYPES[case["dtype"]], case["d"]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, dtype=act, device=dev).mul_(std).add_(mean)

    def offsets(n):
        return torch.randint(0, case["far"], (n,), generator=gen, device=dev).to(torch.int32) if case["far"] else None

    s = {"case": dict(case), "op": op}
    if op in ("norm", "norm_train"):
        B, T, Hq, Hk = (case[k] for k in ("B", "T", "Hq", "Hk"))
        # q and k are views into one projection's output, whose heads differ in scale
        qk = normal(B, T, (Hq + Hk) * d) * normal((Hq + Hk) * d, std=0.3, mean=1.5)
        s["q"], s["k"] = qk[..., :Hq * d], qk[..., Hq * d:] if Hk else None
        s["q_weight"], s["k_weight"] = normal(d, std=0.1, mean=1.0), normal(d, std=0.1, mean=1.0) if Hk else None
        s["inv_freq"], s["offsets"] = _inverse_frequencies(case, dev), offsets(B)
        if op == "norm_train":
            s["dq_out"], s["dk_out"] = normal(B, T, Hq * d), normal(B, T, Hk * d) if Hk else None
        if own:
            from linear_attention_sequence_qkv_gb300 import gdn
            s["gdn"] = gdn
            s["table"] = gdn.rotary_table(case["rot"], 10000.0, device=dev)
            s["q_out"] = torch.empty((B, T, Hq * d), dtype=act, device=dev)
            s["k_out"] = torch.empty((B, T, Hk * d), dtype=act, device=dev) if Hk else None
            s["desc"] = gdn.norm_rotary_desc_for(s["q"], s["k"], s["q_out"], s["k_out"], s["q_weight"], d=d,
                                                 rot=case["rot"], layout=case["layout"], eps=EPS)
            s["ws"] = torch.empty(gdn.gdn_norm_rotary_workspace_bytes(s["desc"]), dtype=torch.uint8, device=dev)
            if op == "norm_train":
                s["grads"] = gdn.alloc_norm_rotary_grads(s["desc"], dev)
        return s
    Hk = case["Hk"]
    if op in ("attn", "attn_train"):
        B, T, Hq, past = (case[k] for k in ("B", "T", "Hq", "past"))
        if past:
            rows = sum(n for _, _, _, n in _spans(case)) // B
            s["q"], s["k"], s["v"] = normal(B, T, Hq * d, std=2.0), normal(B, rows, Hk * d), normal(B, rows, Hk * d)
        else:
            # q, k and v are views into one buffer; scores with a standard deviation of 2
            s["qkv"] = normal(B, T, (Hq + 2 * Hk) * d)
            s["qkv"][..., :Hq * d] *= 2.0
            s["q"], s["k"], s["v"] = s["qkv"].split([Hq * d, Hk * d, Hk * d], dim=-1)
        s["cu"] = s["cu_k"] = None
        if case["seqs"]:
            at = _spans(case)
            s["cu"] = torch.tensor([a[0] for a in at] + [T], dtype=torch.int32, device=dev)
            s["cu_k"] = torch.tensor([a[2] for a in at] + [at[-1][2] + at[-1][3]], dtype=torch.int32, device=dev) if past else None
        if op == "attn_train":
            s["dout"] = normal(B, T, Hq * d)
        if own:
            from linear_attention_sequence_qkv_gb300 import gdn
            s["gdn"] = gdn
            s["desc"] = gdn.window_attention_desc_for(s["q"], s["k"], s["v"], d=d, window=case["window"],
                                                      sinks=case["sinks"], cu_seqlens=s["cu"])
            s["bufs"] = gdn.alloc_window_attention(s["desc"], dev)
            if op == "attn_train":
                s["grads"] = gdn.alloc_window_attention_grads(s["desc"], dev)
        return s
    slots, B = case["sinks"] + case["window"] + case["slack"], case["seqs"] if op == "fill" and case["seqs"] else case["B"]
    s["k_cache"], s["v_cache"] = normal(B, Hk, slots, d), normal(B, Hk, slots, d)
    s["lengths"] = offsets(B)
    if s["lengths"] is None:
        s["lengths"] = torch.zeros(B, dtype=torch.int32, device=dev)
    if op == "step":
        kv = normal(B, 1, 2 * Hk * d)
        s["q"], s["k"], s["v"] = normal(B, 1, case["Hq"] * d, std=2.0), kv[..., :Hk * d], kv[..., Hk * d:]
        if own:
            from linear_attention_sequence_qkv_gb300 import gdn
            s["gdn"] = gdn
            s["desc"] = gdn.window_attention_desc_for(s["q"], s["k"], s["v"], d=d, window=case["window"],
                                                      sinks=case["sinks"], slots=slots)
            s["out"] = torch.empty_like(s["q"])
            s["ws"] = torch.empty(gdn.gdn_window_attention_step_workspace_bytes(s["desc"]), dtype=torch.uint8, device=dev)
        return s
    kv = normal(case["B"], case["T"], 2 * Hk * d)
    s["k"], s["v"] = kv[..., :Hk * d], kv[..., Hk * d:]
    s["cu"] = torch.tensor([a[0] for a in _spans(case)] + [case["T"]], dtype=torch.int32, device=dev) if case["seqs"] else None
    if own:
        from linear_attention_sequence_qkv_gb300 import gdn
        s["gdn"] = gdn
        s["desc"] = gdn.window_attention_desc_for(None, s["k"], s["v"], d=d, window=case["window"], sinks=case["sinks"],
                                                  slots=slots, cu_seqlens=s["cu"])
        s["ws"] = torch.empty(gdn.gdn_window_cache_write_workspace_bytes(s["desc"]), dtype=torch.uint8, device=dev)
    return s


# -------------------------------------------------------------- plain forms
def _turn(x, co, si, case):
    """The first rot channels of [B, T, H, d] rotated by angles whose cosines and sines are [B, T, 1, rot / 2]."""
    rot = case["rot"]
    if case["layout"] == "half":
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([x1 * co - x2 * si, x2 * co + x1 * si], dim=-1)
    else:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([x1 * co - x2 * si, x2 * co + x1 * si], dim=-1).flatten(-2)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_norm(s):
    c = s["case"]
    B, T = s["q"].shape[:2]
    at = torch.arange(T, dtype=torch.float64, device=s["q"].device).expand(B, T)
    if s["offsets"] is not None:
        at = at + s["offsets"].double()[:, None]
    angle = (at[..., None] * s["inv_freq"])[:, :, None]
    co, si = torch.cos(angle).float(), torch.sin(angle).float()

    def norm(x, w):
        y = x.float().view(B, T, -1, c["d"])
        rstd = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        return y * rstd, rstd, w.float()

    def forward(x, w):
        if x is None:
            return None
        xh, _, w = norm(x, w)
        return _turn(xh * w, co, si, c).view(B, T, -1).to(x.dtype)

    def backward(x, w, dout):
        if x is None:
            return None, None
        xh, rstd, w = norm(x, w)
        dz = _turn(dout.float().view(B, T, -1, c["d"]), co, -si, c)
        t = dz * w
        dx = rstd * (t - xh * (t * xh).mean(-1, keepdim=True))
        return dx.view(B, T, -1).to(x.dtype), (dz * xh).double().sum((0, 1, 2)).float()

    out = {"q": forward(s["q"], s["q_weight"]), "k": forward(s["k"], s["k_weight"])}
    if s["op"] == "norm_train":
        out["dq"], out["dq_weight"] = backward(s["q"], s["q_weight"], s["dq_out"])
        out["dk"], out["dk_weight"] = backward(s["k"], s["k_weight"], s["dk_out"])
    return out


def _bands(case):
    """Blocks of queries with the keys that any of them sees, for all scores of a long context do not fit the card:
    (first query, one past the last, key of the query's own position for the first query, the keys' runs)."""
    w, sinks = case["window"], case["sinks"]
    for q0, nq, k0, nk in _spans(case):
        for a in range(0, nq, BAND):
            b = min(a + BAND, nq)
            lo = max(0, nk - nq + a - w + 1)
            runs = ([(k0, k0 + min(sinks, lo))] if lo and sinks else []) + [(k0 + lo, k0 + nk - nq + b)]
            yield q0 + a, q0 + b, k0 + nk - nq + a, k0, runs


def _plain_attention(s):
    c, train = s["case"], s["op"] == "attn_train"
    Hk, d, scale = c["Hk"], c["d"], 1.0 / math.sqrt(c["d"])
    G = c["Hq"] // Hk
    flat = lambda x, *h: x.reshape(-1, *h, d)  # noqa: E731
    q, k, v = flat(s["q"], Hk, G), flat(s["k"], Hk), flat(s["v"], Hk)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    if train:
        dout, dq = flat(s["dout"], Hk, G), torch.empty_like(q)
        dk, dv = (torch.zeros(k.shape, dtype=torch.float32, device=q.device) for _ in range(2))
    for a, b, at, first, runs in _bands(c):
        key = torch.cat([torch.arange(x, y, device=q.device) for x, y in runs])
        pos = torch.arange(at, at + b - a, device=q.device)[:, None]
        seen = (key <= pos) & ((key > pos - c["window"]) | (key < first + c["sinks"]))
        qb = q[a:b].float().permute(1, 2, 0, 3)                                 # [Hk, G, queries, d]
        kb = torch.cat([k[x:y] for x, y in runs]).float().permute(1, 2, 0)[:, None]   # [Hk, 1, d, keys]
        vb = torch.cat([v[x:y] for x, y in runs]).float().transpose(0, 1)[:, None]    # [Hk, 1, keys, d]
        x = torch.where(seen, (qb @ kb) * scale, -math.inf)
        most = x.amax(-1, keepdim=True)
        p = torch.exp(x - most)
        total = p.sum(-1, keepdim=True)
        p = p / total
        o = p @ vb
        out[a:b] = o.permute(2, 0, 1, 3).to(out.dtype)
        lse[a:b] = (most + torch.log(total))[..., 0].permute(2, 0, 1)
        if train:
            g = dout[a:b].float().permute(1, 2, 0, 3)
            dp = g @ vb.transpose(-1, -2)
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
            dq[a:b] = (ds @ kb.transpose(-1, -2)).permute(2, 0, 1, 3).to(dq.dtype)
            dkb = (ds.transpose(-1, -2) @ qb).sum(1).transpose(0, 1)
            dvb = (p.transpose(-1, -2) @ g).sum(1).transpose(0, 1)
            dk.index_add_(0, key, dkb)
            dv.index_add_(0, key, dvb)
    shape = s["q"].shape
    res = {"out": out.view(shape)}
    if not train:
        res["lse"] = lse.flatten(1).t()
        return res
    return {**res, "dq": dq.view(shape), "dk": dk.to(q.dtype).view(s["k"].shape), "dv": dv.to(q.dtype).view(s["v"].shape)}


def _slot(position, case):
    """The cache slot of a position: its own for the first ones, then round and round the others."""
    sinks, ring = case["sinks"], case["window"] + case["slack"]
    return torch.where(position < sinks, position, sinks + (position - sinks) % ring)


def _plain_step(s):
    c = s["case"]
    B, Hk, slots, d = s["k_cache"].shape
    t = s["lengths"].long()
    row, slot = torch.arange(B, device=t.device), _slot(t, c)
    s["k_cache"][row, :, slot] = s["k"].reshape(B, Hk, d)
    s["v_cache"][row, :, slot] = s["v"].reshape(B, Hk, d)
    i = torch.arange(slots, device=t.device)
    # the position that a slot holds: its own, or the last one up to t that falls on it
    held = torch.where(i < c["sinks"], i, t[:, None] - (t[:, None] - i) % (slots - c["sinks"]))
    seen = (held >= torch.clamp(i, max=c["sinks"])) & (held <= t[:, None]) & ((held > t[:, None] - c["window"]) | (i < c["sinks"]))
    q = s["q"].float().view(B, Hk, -1, d)
    x = torch.where(seen[:, None, None], (q @ s["k_cache"].float().transpose(-1, -2)) / math.sqrt(d), -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    return {"out": (p @ s["v_cache"].float()).view(B, 1, -1).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_fill(s):
    c = s["case"]
    n, Hk, slots, d = s["k_cache"].shape
    dev, ring = s["k"].device, slots - c["sinks"]
    tokens = torch.arange(c["B"] * c["T"], device=dev)
    if s["cu"] is None:
        row, at, count = tokens // c["T"], tokens % c["T"], torch.full_like(tokens, c["T"])
    else:
        row = torch.bucketize(tokens, s["cu"][1:].long(), right=True)
        at, count = tokens - s["cu"].long()[row], s["cu"].long().diff()[row]
    pos = s["lengths"].long()[row] + at
    kept = (pos < c["sinks"]) | (at >= count - ring)
    row, slot, kept = row[kept], _slot(pos[kept], c), tokens[kept]
    for name in ("k", "v"):
        s[name + "_cache"][row, :, slot] = s[name].reshape(-1, Hk, d)[kept]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


PLAIN = {"norm": _plain_norm, "norm_train": _plain_norm, "attn": _plain_attention, "attn_train": _plain_attention,
         "step": _plain_step, "fill": _plain_fill}


def run(state):
    s = state
    if not own:
        return PLAIN[s["op"]](s)
    gdn, op, d = s["gdn"], s["op"], s["desc"]
    if op in ("norm", "norm_train"):
        gdn.gdn_norm_rotary_forward(d, s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], None, None, s["offsets"],
                                    s["q_out"], s["k_out"], s["ws"], s["ws"].numel())
        if op == "norm":
            return {"q": s["q_out"], "k": s["k_out"]}
        r = s["grads"]
        gdn.gdn_norm_rotary_backward(d, s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], None, None, s["offsets"],
                                     s["dq_out"], s["dk_out"], r.dq, r.dk, r.dq_weight, r.dk_weight, r.workspace, r.ws_bytes)
        return {"q": s["q_out"], "k": s["k_out"], "dq": r.dq, "dq_weight": r.dq_weight, "dk": r.dk, "dk_weight": r.dk_weight}
    if op in ("attn", "attn_train"):
        f = s["bufs"]
        gdn.gdn_window_attention_forward(d, s["q"], s["k"], s["v"], s["cu"], s["cu_k"], f.out, f.lse, f.workspace, f.ws_bytes)
        if op == "attn":
            return {"out": f.out, "lse": f.lse}
        r = s["grads"]
        gdn.gdn_window_attention_backward(d, s["q"], s["k"], s["v"], f.out, f.lse, s["dout"], s["cu"], s["cu_k"], r.dq, r.dk,
                                          r.dv, r.workspace, r.ws_bytes)
        return {"out": f.out, "dq": r.dq, "dk": r.dk, "dv": r.dv}
    if op == "step":
        gdn.gdn_window_attention_step(d, s["q"], s["k"], s["v"], s["lengths"], s["k_cache"], s["v_cache"], s["out"], s["ws"],
                                      s["ws"].numel())
        return {"out": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    gdn.gdn_window_cache_write(d, s["k"], s["v"], s["cu"], s["lengths"], s["k_cache"], s["v_cache"], s["ws"], s["ws"].numel())
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ------------------------------------------------------ work and exact values
def _pairs(case):
    """(query, key) pairs that the mask leaves, of one head."""
    w, sinks, total = case["window"], case["sinks"], 0
    for _, nq, _, nk in _spans(case):
        lo, hi = nk - nq + 1, nk            # visible positions up to a query's own: lo .. hi of them
        tri = lambda n: n * (n + 1) // 2    # noqa: E731
        reach = w + sinks                   # a query sees at most these
        full = max(0, hi - max(lo - 1, reach))
        low = min(hi, reach)
        total += full * reach + (tri(low) - tri(lo - 1) if low >= lo else 0)
    return total


def work(case):
    op, es, d = case["op"], BYTES[case["dtype"]], case["d"]
    if op in ("norm", "norm_train"):
        heads = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        if op == "norm":
            return {"bytes": 2 * es * heads * d + 2 * es * d, "flops": heads * (4 * d + 3 * case["rot"])}
        return {"bytes": 4 * es * heads * d + (2 * es + 8) * d, "flops": heads * (15 * d + 6 * case["rot"])}
    if op in ("attn", "attn_train"):
        spans = _spans(case)
        nq, nk = sum(a[1] for a in spans), sum(a[3] for a in spans)
        q, k, pairs = nq * case["Hq"] * d, nk * case["Hk"] * d, _pairs(case) * case["Hq"]
        if op == "attn":
            return {"bytes": es * (2 * q + 2 * k) + 4 * nq * case["Hq"], "flops": 4 * d * pairs}
        return {"bytes": es * (4 * q + 4 * k), "flops": 14 * d * pairs}
    Hk, slots = case["Hk"], case["sinks"] + case["window"]
    if op == "step":
        # the mean over lengths from 0 to far of what a query sees: itself and the tokens before it, `slots` at most
        far = case["far"]
        seen = (slots * (far - slots) + slots * (slots + 1) / 2) / far if far > slots else (far + 1) / 2
        new = case["B"] * d * (2 * case["Hq"] + 4 * Hk)
        return {"bytes": es * (2 * case["B"] * Hk * d * seen + new), "flops": 4 * d * seen * case["B"] * case["Hq"]}
    kept = sum(min(a[1], slots + case["slack"]) for a in _spans(case))
    return {"bytes": 4 * es * kept * Hk * d, "flops": kept}


def _exact_norm(case, s):
    """Each pair as a complex number times e^{i angle}; gradients by torch's own differentiation."""
    d, rot, half, train = case["d"], case["rot"], case["rot"] // 2, case["op"] == "norm_train"
    B, T = s["q"].shape[:2]
    dev = s["q"].device
    at = torch.arange(T, device=dev)[None] + (0 if s["offsets"] is None else s["offsets"].long()[:, None])
    angle = (at.double()[..., None] * s["inv_freq"]).expand(B, T, half)
    unit = torch.polar(torch.ones_like(angle), angle)[:, :, None]
    idx = torch.arange(rot, device=dev)
    pairs = idx.view(2, half).t() if case["layout"] == "half" else idx.view(half, 2)
    back = torch.argsort(pairs.reshape(-1))
    res = {}
    for name in ("q", "k"):
        if s[name] is None:
            res[name] = None
            continue
        x, w = (v.double().detach().clone().requires_grad_(train) for v in (s[name], s[name + "_weight"]))
        y = x.view(B, T, -1, d)
        z = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w
        turned = torch.view_as_real(torch.view_as_complex(z[..., pairs.reshape(-1)].unflatten(-1, (half, 2))) * unit)
        out = torch.cat([turned.flatten(-2)[..., back], z[..., rot:]], dim=-1).reshape(B, T, -1)
        res[name] = out.detach()
        if train:
            res["d" + name], res["d" + name + "_weight"] = torch.autograd.grad(out, [x, w], s["d" + name + "_out"].double())
    if not train:
        return res
    order = ("q", "k", "dq", "dq_weight", "dk", "dk_weight")
    return {n: res.get(n) for n in order}


def _exact_attention(case, s):
    """Head by head, a run of queries against the sequence's keys by index; gradients by torch's own differentiation."""
    d, Hq, Hk, train = case["d"], case["Hq"], case["Hk"], case["op"] == "attn_train"
    group, w, sinks = Hq // Hk, case["window"], case["sinks"]
    spans = _spans(case)
    touched = sum(nq * min(nk, w + sinks + 512) for _, nq, _, nk in spans)
    blocks = sum(-(-nq // 512) for _, nq, _, _ in spans) * Hq
    if 4.0 * d * Hq * touched * (3.5 if train else 1.0) > MOST_EXACT or blocks * (3 if train else 1) > MOST_BLOCKS:
        return None
    dev = s["q"].device
    leaf = {n: s[n].double().detach().reshape(-1, s[n].shape[-1] // d, d).transpose(0, 1).contiguous().requires_grad_(train)
            for n in ("q", "k", "v")}
    out = torch.zeros_like(leaf["q"], requires_grad=False)
    lse = torch.zeros(leaf["q"].shape[:2], dtype=torch.float64, device=dev)
    grads = {n: torch.zeros_like(t, requires_grad=False) for n, t in leaf.items()}
    if train:
        dout = s["dout"].double().reshape(-1, Hq, d).transpose(0, 1)
    for q0, nq, k0, nk in spans:
        for a in range(0, nq, 512):
            rows = torch.arange(a, min(a + 512, nq), device=dev)
            pos = rows + (nk - nq)
            keys = torch.arange(nk, device=dev)
            keys = keys[(keys <= pos[-1]) & ((keys > pos[0] - w) | (keys < sinks))]
            hidden = ~((keys[None] <= pos[:, None]) & ((pos[:, None] - keys[None] < w) | (keys[None] < sinks)))
            for h in range(Hq):
                qs, ks, vs = (t.requires_grad_(train) for t in (leaf["q"].detach()[h, q0 + rows], leaf["k"].detach()[h // group, k0 + keys],
                                                               leaf["v"].detach()[h // group, k0 + keys]))
                x = (torch.einsum("qd,kd->qk", qs, ks) * d ** -0.5).masked_fill(hidden, -math.inf)
                o = torch.softmax(x, dim=-1) @ vs
                out[h, q0 + rows] = o.detach()
                lse[h, q0 + rows] = torch.logsumexp(x, dim=-1).detach()
                if train:
                    gq, gk, gv = torch.autograd.grad(o, [qs, ks, vs], dout[h, q0 + rows])
                    grads["q"][h, q0 + rows] = gq
                    grads["k"][h // group, k0 + keys] += gk
                    grads["v"][h // group, k0 + keys] += gv
    of = lambda t, like: t.transpose(0, 1).reshape(like.shape)  # noqa: E731
    if not train:
        return {"out": of(out, s["q"]), "lse": lse}
    return {"out": of(out, s["q"]), "dq": of(grads["q"], s["q"]), "dk": of(grads["k"], s["k"]), "dv": of(grads["v"], s["v"])}


def _exact_step(case, s):
    """The cache as a list of (slot, position), sequence by sequence."""
    B, Hk, slots, d = s["k_cache"].shape
    sinks, ring, w = case["sinks"], slots - case["sinks"], case["window"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    rows = []
    for b, t in enumerate(s["lengths"].tolist()):
        here = t if t < sinks else sinks + (t - sinks) % ring
        kc[b, :, here], vc[b, :, here] = s["k"][b, 0].double().view(Hk, d), s["v"][b, 0].double().view(Hk, d)
        near = torch.arange(max(sinks, t - w + 1), t + 1, device=kc.device)
        idx = torch.cat([torch.arange(min(sinks, t + 1), device=kc.device), sinks + (near - sinks) % ring])
        q = s["q"][b, 0].double().view(Hk, -1, d)
        x = torch.einsum("hgd,hkd->hgk", q, kc[b][:, idx]) * d ** -0.5
        rows.append(torch.einsum("hgk,hkd->hgd", torch.softmax(x, -1), vc[b][:, idx]).reshape(1, -1))
    return {"out": torch.stack(rows), "k_cache": kc, "v_cache": vc}


def _exact_fill(case, s):
    """Copies: the last `ring` tokens and the first `sinks` positions, sequence by sequence."""
    n, Hk, slots, d = s["k_cache"].shape
    sinks, ring = case["sinks"], slots - case["sinks"]
    res = {}
    for name in ("k", "v"):
        cache, new = s[name + "_cache"].double(), s[name].double().reshape(-1, Hk, d)
        for b, ((q0, nq, _, _), t) in enumerate(zip(_spans(case), s["lengths"].tolist())):
            first = max(0, min(nq, sinks - t))
            if first:
                cache[b, :, t:t + first] = new[q0:q0 + first].transpose(0, 1)
            at = torch.arange(max(first, nq - ring), nq, device=cache.device)
            cache[b, :, sinks + (t + at - sinks) % ring] = new[q0 + at].transpose(0, 1)
        res[name + "_cache"] = cache
    return res


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_train"):
        return _exact_norm(case, s)
    if op in ("attn", "attn_train"):
        return _exact_attention(case, s)
    return _exact_step(case, s) if op == "step" else _exact_fill(case, s)
