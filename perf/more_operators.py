"""Workloads of what a mixture-of-experts decoder layer does around the packed products: choosing experts from
the router's logits, the experts' gated feed-forward network over packed weights, and linear attention with a
decay for each head (prompts and single tokens over one kept state).

``run`` computes a workload in its plain form (elementary torch operations in fp32) or, where ``own`` is
true, through the library's calls. ``exact`` states the operators' definitions in fp64.

Experts' weights are uint8 rows [expert][row][row bytes] in the GGUF formats bf16, f16, q4_0, q4_k, q6_k, q8_0
and q5_0.
"""
import math

import torch

own = False

DEVICE = "cuda:0"
# weights and bytes of a block
BLOCK = {"bf16": (1, 2), "f16": (1, 2), "q4_0": (32, 18), "q4_k": (256, 144), "q6_k": (256, 210), "q8_0": (32, 34),
         "q5_0": (32, 22)}


# ------------------------------------------------------------------ cases ----

def _route(name, n_pos, n_experts, top_k, score, normalize, scale, masked=0.0):
    return {"name": name, "kind": "route", "n_pos": n_pos, "n_experts": n_experts, "top_k": top_k, "score": score,
            "normalize": normalize, "scale": scale, "masked": masked}


def _ffn(name, act, fmt, fmt_down, n_pos, d, n_ff, n_experts, top_k):
    return {"name": name, "kind": "ffn", "act": act, "fmt": fmt, "fmt_down": fmt_down, "n_pos": n_pos, "d": d,
            "n_ff": n_ff, "n_experts": n_experts, "top_k": top_k}


def _linear(name, n_seqs, n_new, n_heads, n_qk, dk, dv, max_len, ragged, empty=0, constant=False):
    return {"name": name, "kind": "linear", "n_seqs": n_seqs, "n_new": n_new, "n_heads": n_heads, "n_qk": n_qk,
            "dk": dk, "dv": dv, "max_len": max_len, "ragged": ragged, "empty": empty, "constant": constant}


def listed():
    return [
        # one user's token: the choice of 8 of 64 experts, a call's latency
        _route("route_one", 1, 64, 8, "softmax", True, 1.0),
        # a prompt's chunk over many small experts, a few of them switched off
        _route("route_chunk", 4099, 256, 8, "sigmoid", True, 2.5, masked=0.05),
        # one user's token through 8 small experts
        _ffn("ffn_one", "swiglu", "q4_k", "q6_k", 1, 2048, 768, 64, 8),
        # one user's token through 2 large experts
        _ffn("ffn_one_wide", "swiglu", "q4_0", "q4_0", 1, 4096, 14336, 8, 2),
        # a few users' tokens, hardly any expert shared
        _ffn("ffn_batch", "swiglu", "q8_0", "q8_0", 8, 2048, 768, 64, 8),
        # drafted tokens through odd-sized experts, two formats
        _ffn("ffn_drafts", "geglu", "q5_0", "q8_0", 5, 1376, 352, 24, 4),
        # 16-bit experts, a serving batch
        _ffn("ffn_bf16", "geglu", "bf16", "bf16", 24, 1536, 640, 40, 6),
        # the widest batch: every expert has many rows
        _ffn("ffn_chunk", "swiglu", "q4_k", "q4_k", 256, 2048, 1024, 64, 8),
        # linear attention of one user's token
        _linear("linear_one", 1, 1, 32, 16, 128, 128, 801, 0.0),
        # one decoding step of a batch, a few slots idle
        _linear("linear_step", 64, 1, 32, 16, 128, 128, 4000, 0.9, empty=2),
        # one long prompt
        _linear("linear_prompt", 1, 12001, 16, 16, 128, 128, 12001, 0.0),
        # prompts of different lengths, some of them a later chunk of theirs; one decay for each head
        _linear("linear_ragged", 6, 1777, 12, 4, 64, 96, 2500, 0.6, constant=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("route", "ffn", "ffn", "ffn", "linear", "linear"))
    if kind == "route":
        n_experts = _log(rng, 4, 512)
        got = _route("", _log(rng, 1, 8192 * 256 // max(n_experts, 256)), n_experts, _log(rng, 1, min(16, n_experts)),
                     rng.choice(("softmax", "sigmoid")), rng.random() < 0.7, rng.choice((1.0, 1.0, 2.5)),
                     rng.choice((0.0, 0.0, 0.1, 0.7)))
    elif kind == "ffn":
        # a model's experts: one format, the down matrix often in a wider one
        fmt, fmt_down = rng.choice((("q4_k", "q4_k"), ("q4_k", "q6_k"), ("q6_k", "q6_k"), ("q4_0", "q4_0"), ("q5_0", "q8_0"),
                                    ("q8_0", "q8_0"), ("q4_k", "q8_0"), ("q4_k", "q5_0"), ("f16", "f16"), ("bf16", "bf16")))
        step_d, step_ff = (256 if f in ("q4_k", "q6_k") else 32 if f not in ("f16", "bf16") else 2 for f in (fmt, fmt_down))
        d, n_ff = (max(1, _log(rng, 256, hi) // step) * step for hi, step in ((5000, step_d), (4000, step_ff)))
        n_experts = _log(rng, 2, max(3, min(128, 10 ** 9 // (3 * d * n_ff))))
        top_k = _log(rng, 1, min(10, n_experts))
        n_pos = _log(rng, 1, max(2, min(256, 2048 * 1024 * 2048 // (top_k * d * n_ff))))
        got = _ffn("", rng.choice(("swiglu", "swiglu", "geglu")), fmt, fmt_down, n_pos, d, n_ff, n_experts, top_k)
    else:
        dk, dv = rng.choice((32, 64, 96, 128, 128)), rng.choice((32, 64, 96, 128, 128, 192, 256))
        n_qk = rng.choice((1, 2, 4, 8, 16))
        n_heads = n_qk * rng.choice((1, 1, 2, 3, 4))
        n_seqs = _log(rng, 1, 64)
        n_new = 1
        if rng.random() < 0.65:
            n_new = _log(rng, 2, max(3, min(12001, int((12001 ** 2 * 16 / (n_seqs * n_heads)) ** 0.5))))
        max_len = n_new + (0 if rng.random() < 0.4 else _log(rng, 1, 4000))
        got = _linear("", n_seqs, n_new, n_heads, n_qk, dk, dv, max_len, round(rng.uniform(0.0, 0.98), 3),
                      empty=rng.choice((0, 0, 1)) if n_seqs > 1 else 0, constant=rng.random() < 0.3)
    del got["name"]
    return got


def _lens(c):
    """Positions that the sequences hold, the new ones included: the first max_len, the others up to `ragged` of it
    shorter, the last `empty` none."""
    out = [c["max_len"] - int(c["ragged"] * c["max_len"] * ((0.6180339887 * i) % 1.0)) for i in range(c["n_seqs"])]
    return [0 if i >= c["n_seqs"] - c["empty"] else max(n, 1) for i, n in enumerate(out)]


# ---------------------------------------------------------------- weights ----

def _row_bytes(fmt, k):
    return k // BLOCK[fmt][0] * BLOCK[fmt][1]


def _weights(g, fmt, n_experts, n, k):
    """Packed weights of about unit gain: uniform codes, scales that vary by a factor of two."""
    std = k ** -0.5
    if fmt in ("bf16", "f16"):
        w = torch.randn((n_experts, n, k), generator=g, device=DEVICE) * std
        return w.to(torch.float16 if fmt == "f16" else torch.bfloat16).view(torch.uint8)
    per, size = BLOCK[fmt]
    shape = (n_experts, n, k // per)
    raw = torch.randint(0, 256, (*shape, size), generator=g, device=DEVICE, dtype=torch.uint8)
    # the codes' standard deviation about their middle, times the mean of the sub-blocks' scales where there are some
    spread = {"q4_0": 4.6, "q5_0": 9.2, "q8_0": 73.9, "q4_k": 4.6 * 40, "q6_k": 18.5 * 40}[fmt]
    d = (torch.rand(shape, generator=g, device=DEVICE) + 0.5) * (std / spread)

    def f16(x):
        return x.half().unsqueeze(-1).view(torch.uint8)

    if fmt == "q4_k":
        # mins of about 7.5 scales, as a fit to weights around zero leaves them
        sc = torch.randint(24, 57, (*shape, 8), generator=g, device=DEVICE)
        m = (sc + torch.randint(-4, 5, sc.shape, generator=g, device=DEVICE)).clamp(0, 63)
        raw[..., 0:2], raw[..., 2:4] = f16(d), f16(d * 7.5)
        raw[..., 4:8] = (sc[..., :4] + (sc[..., 4:] // 16) * 64).to(torch.uint8)
        raw[..., 8:12] = (m[..., :4] + (m[..., 4:] // 16) * 64).to(torch.uint8)
        raw[..., 12:16] = (sc[..., 4:] % 16 + (m[..., 4:] % 16) * 16).to(torch.uint8)
    elif fmt == "q6_k":
        sc = torch.randint(24, 57, (*shape, 16), generator=g, device=DEVICE)
        sign = torch.randint(0, 2, sc.shape, generator=g, device=DEVICE) * 2 - 1
        raw[..., 192:208] = (sc * sign).to(torch.int8).view(torch.uint8)
        raw[..., 208:210] = f16(d)
    else:
        raw[..., 0:2] = f16(d)
    return raw.reshape(n_experts, n, -1)


def _f16_at(blocks, at):
    return blocks[..., at:at + 2].contiguous().view(torch.float16).float()


def _values(raw, fmt, k):
    """fp32 weights [.., k] of packed rows [.., row bytes]."""
    if fmt == "f16":
        return raw.view(torch.float16).float()
    if fmt == "bf16":
        return raw.view(torch.bfloat16).float()
    b = raw.unflatten(-1, (-1, BLOCK[fmt][1]))
    if fmt == "q8_0":
        w = b[..., 2:].contiguous().view(torch.int8).float() * _f16_at(b, 0)
    elif fmt == "q4_0":
        w = (torch.cat((b[..., 2:] & 15, b[..., 2:] >> 4), -1).float() - 8.0) * _f16_at(b, 0)
    elif fmt == "q5_0":
        high = (b[..., 2:6].unsqueeze(-1) >> torch.arange(8, device=raw.device, dtype=torch.uint8)) & 1
        code = torch.cat((b[..., 6:] & 15, b[..., 6:] >> 4), -1) | (high.flatten(-2) << 4)
        w = (code.float() - 16.0) * _f16_at(b, 0)
    elif fmt == "q4_k":
        s, m, both = b[..., 4:8], b[..., 8:12], b[..., 12:16]
        sc = torch.cat((s & 63, (both & 15) | ((s >> 6) << 4)), -1).float() * _f16_at(b, 0)
        mn = torch.cat((m & 63, (both >> 4) | ((m >> 6) << 4)), -1).float() * _f16_at(b, 2)
        c = b[..., 16:].unflatten(-1, (4, 32))
        w = torch.stack((c & 15, c >> 4), -2).flatten(-3, -2).float() * sc.unsqueeze(-1) - mn.unsqueeze(-1)
    else:
        ql = b[..., :128].unflatten(-1, (2, 2, 32))                       # [half, which 32, byte]
        qh = b[..., 128:192].unflatten(-1, (2, 32))
        low = torch.cat((ql & 15, ql >> 4), -2)                           # [half, quarter, byte]
        shift = torch.tensor([0, 2, 4, 6], device=raw.device, dtype=torch.uint8).unsqueeze(-1)
        code = low | (((qh.unsqueeze(-2) >> shift) & 3) << 4)
        sc = b[..., 192:208].contiguous().view(torch.int8).float() * _f16_at(b, 208)
        w = (code.float() - 32.0).flatten(-3).unflatten(-1, (16, 16)) * sc.unsqueeze(-1)
    return w.flatten(raw.dim() - 1)


# ---------------------------------------------------------------- prepare ----

def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    st = {"case": c}
    if c["kind"] == "route":
        st["logits"] = normal(c["n_pos"], c["n_experts"]) * 1.5
        if c["masked"]:
            off = torch.rand((c["n_pos"], c["n_experts"]), generator=g, device=DEVICE) < c["masked"]
            st["logits"].masked_fill_(off, -math.inf)
    elif c["kind"] == "ffn":
        st["x"] = normal(c["n_pos"], c["d"])
        chosen = normal(c["n_pos"], c["n_experts"]).topk(c["top_k"], -1)
        st["ids"] = chosen.indices.to(torch.int32)
        st["weights"] = torch.softmax(chosen.values, -1)
        st["gate"] = _weights(g, c["fmt"], c["n_experts"], c["n_ff"], c["d"])
        st["up"] = _weights(g, c["fmt"], c["n_experts"], c["n_ff"], c["d"])
        st["down"] = _weights(g, c["fmt_down"], c["n_experts"], c["d"], c["n_ff"])
    else:
        s, t, h = c["n_seqs"], c["n_new"], c["n_heads"]
        # one product's output row holds q, k and v of a token side by side
        st["qkv"] = normal(s, t, 2 * c["n_qk"] * c["dk"] + h * c["dv"])
        # heads that forget within a few positions beside heads that remember hundreds
        rate = torch.logspace(-2.5, 0.0, h, device=DEVICE)
        st["decay"] = -rate if c["constant"] else -rate * torch.nn.functional.softplus(normal(s, t, h))
        st["state"] = normal(s, h, c["dk"], c["dv"])
        st["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEVICE)
        st["out"] = torch.empty((s, t, h, c["dv"]), device=DEVICE)
        st["state_out"] = torch.empty_like(st["state"])
    return st


def _qkv(st):
    """q, k and v of a product's output rows, as views."""
    c = st["case"]
    w = c["n_qk"] * c["dk"]
    q, k, v = st["qkv"].split((w, w, c["n_heads"] * c["dv"]), -1)
    return q.unflatten(-1, (-1, c["dk"])), k.unflatten(-1, (-1, c["dk"])), v.unflatten(-1, (-1, c["dv"]))


# -------------------------------------------------------------------- run ----

def _plain_route(st):
    c = st["case"]
    order = torch.sort(st["logits"], dim=-1, descending=True, stable=True)
    best = order.values[:, :c["top_k"]]
    on = best > -math.inf
    if c["score"] == "sigmoid":
        # log of the logistic function: its ratios keep their precision far from 0
        s = torch.where(on, torch.clamp(best, max=0.0) - torch.log1p(torch.exp(-torch.abs(best))), -math.inf)
        total = torch.exp(s - s[:, :1]).sum(-1, keepdim=True)
        w = torch.exp(s - s[:, :1]) / total if c["normalize"] else torch.exp(s)
    else:
        over = best if c["normalize"] else order.values
        w = torch.exp(best - best[:, :1]) / torch.exp(over - best[:, :1]).sum(-1, keepdim=True)
    ids = torch.where(on, order.indices[:, :c["top_k"]], -1).to(torch.int32)
    return ids, torch.where(on, w * c["scale"], 0.0)


def _activated(g, act):
    if act == "swiglu":
        return g / (1.0 + torch.exp(-g))
    z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)
    return g / (1.0 + torch.exp(-2.0 * z))


def _plain_ffn(st):
    c = st["case"]
    n, k = c["n_pos"], c["top_k"]
    gather = n * k <= c["n_experts"]
    ids = st["ids"].long().flatten() if gather else slice(None)           # a slice for each pair, or every slice once
    gate, up = _values(st["gate"][ids], c["fmt"], c["d"]), _values(st["up"][ids], c["fmt"], c["d"])
    down = _values(st["down"][ids], c["fmt_down"], c["n_ff"])
    x = st["x"].repeat_interleave(k, 0).unsqueeze(1) if gather else st["x"]
    h = _activated(torch.matmul(x, gate.transpose(1, 2)), c["act"]) * torch.matmul(x, up.transpose(1, 2))
    y = torch.matmul(h, down.transpose(1, 2))                             # [slice, row, d]
    if gather:
        return (y.view(n, k, -1) * st["weights"].unsqueeze(-1)).sum(1)
    share = torch.zeros((n, c["n_experts"]), device=y.device).scatter_add_(1, st["ids"].long(), st["weights"])
    return (y * share.t().unsqueeze(-1)).sum(0)


def _plain_linear(st):
    c = st["case"]
    q, k, v = (x.transpose(1, 2) for x in _qkv(st))                       # [sequence, head, row, dim]
    group, rows = c["n_heads"] // c["n_qk"], c["n_new"]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    lens = st["lens"].long()
    t = torch.arange(rows, device=q.device)
    here = (t >= rows - lens.unsqueeze(1)).view(-1, 1, rows)              # rows that are positions
    g = st["decay"].unsqueeze(-1).expand(-1, rows).unsqueeze(0) if c["constant"] else st["decay"].transpose(1, 2)
    total = torch.where(here, g, 0.0).double().cumsum(-1)                 # in 64 bits: differences of long sums follow
    high = total.float()
    low = (total - high.double()).float()
    s0 = torch.where((lens > rows).view(-1, 1, 1, 1), st["state"], 0.0)   # a sequence that begins here begins at zero
    v = torch.where(here.unsqueeze(-1), v, 0.0)
    k = torch.where(here.unsqueeze(-1), k, 0.0)
    d = (high.unsqueeze(-1) - high.unsqueeze(-2)) + (low.unsqueeze(-1) - low.unsqueeze(-2))
    d.masked_fill_(t.unsqueeze(-1) < t, -math.inf).exp_()
    o = torch.matmul(torch.matmul(q, k.transpose(2, 3)).mul_(d), v)
    o = o + torch.matmul(q, s0) * torch.exp(high).unsqueeze(-1)
    o = torch.where(here.unsqueeze(-1), o * c["dk"] ** -0.5, 0.0)
    state = torch.matmul((k * d[..., -1, :].unsqueeze(-1)).transpose(2, 3), v)
    state = state + s0 * torch.exp(high[..., -1])[..., None, None]
    return o.transpose(1, 2), torch.where((lens > 0).view(-1, 1, 1, 1), state, st["state"])


def run(state):
    st, c = state, state["case"]
    if c["kind"] == "route":
        if not own:
            return _plain_route(st)
        import quantized_weight_gguf_gb300 as lib
        return lib.route_experts(st["logits"], c["top_k"], score=c["score"], normalize=c["normalize"], scale=c["scale"])
    if c["kind"] == "ffn":
        if not own:
            return _plain_ffn(st)
        import quantized_weight_gguf_gb300 as lib
        return lib.experts_ffn(c["act"], c["fmt"], st["gate"], st["up"], c["fmt_down"], st["down"], st["x"], st["ids"],
                               st["weights"], c["d"], c["n_ff"], c["n_experts"])
    if not own:
        return _plain_linear(st)
    import quantized_weight_gguf_gb300 as lib
    q, k, v = _qkv(st)
    lib.linear_attend(q, k, v, st["decay"], st["state"], st["lens"], out=st["out"], state_out=st["state_out"])
    return st["out"], st["state_out"]


# ------------------------------------------------------------------- work ----

def work(case):
    c = case
    if c["kind"] == "route":
        # logits read, ids and weights written
        return {"bytes": 4 * c["n_pos"] * (c["n_experts"] + 2 * c["top_k"]), "flops": 2 * c["n_pos"] * c["n_experts"]}
    if c["kind"] == "ffn":
        # the slices of the experts that are chosen at all (as many as ids drawn at random leave), x, ids and weights
        # read, y written
        share = 1.0 - (1.0 - c["top_k"] / c["n_experts"]) ** c["n_pos"]
        slice_bytes = 2 * c["n_ff"] * _row_bytes(c["fmt"], c["d"]) + c["d"] * _row_bytes(c["fmt_down"], c["n_ff"])
        pairs = c["n_pos"] * c["top_k"]
        return {"bytes": int(c["n_experts"] * share * slice_bytes) + 8 * c["n_pos"] * c["d"] + 8 * pairs,
                "flops": 6 * pairs * c["d"] * c["n_ff"]}
    lens, h, t = _lens(c), c["n_heads"], c["n_new"]
    rows = sum(min(n, t) for n in lens)
    state = 4 * h * c["dk"] * c["dv"]
    # q, k, v and the decays of the rows that are positions, every output row, the states that are not begun here, the
    # states written
    values = rows * (2 * c["n_qk"] * c["dk"] + h * c["dv"]) + c["n_seqs"] * t * h * c["dv"]
    values += h if c["constant"] else rows * h
    return {"bytes": 4 * values + state * (c["n_seqs"] + sum(n > t or n == 0 for n in lens)),
            "flops": 4 * rows * h * c["dk"] * c["dv"]}


# ------------------------------------------------------------------ exact ----

def _exact_route(state):
    c, x = state["case"], state["logits"].double()
    left, ids, got = x.clone(), [], []
    for _ in range(c["top_k"]):
        top = left.amax(-1, keepdim=True)
        first = (left == top).to(torch.int8).argmax(-1, keepdim=True)     # the lowest index among equals
        none = torch.isinf(top)
        ids.append(torch.where(none, -1, first))
        got.append(torch.where(none, -math.inf, top))
        left.scatter_(1, first, -math.inf)
    ids, got = torch.cat(ids, 1), torch.cat(got, 1)
    if c["score"] == "softmax":
        w = torch.softmax(got, -1) if c["normalize"] else torch.exp(got - torch.logsumexp(x, -1, keepdim=True))
    else:
        w = torch.sigmoid(got)
        w = w / w.sum(-1, keepdim=True) if c["normalize"] else w
    return ids.to(torch.int32), torch.where(ids >= 0, w * c["scale"], 0.0)


def _exact_rows(raw, fmt, k):
    """fp64 weights [rows, k] of packed rows, from integer arithmetic on their bytes."""
    rows = raw.shape[0]
    if fmt == "f16":
        return raw.contiguous().view(torch.float16).double()
    if fmt == "bf16":
        bits = raw.contiguous().view(torch.int16).to(torch.int32) << 16
        return bits.view(torch.float32).double()
    b = raw.reshape(rows, -1, BLOCK[fmt][1])
    i = b.to(torch.int64)
    half = lambda at: b[..., at:at + 2].contiguous().view(torch.float16).double()  # noqa: E731
    out = torch.empty((rows, b.shape[1], BLOCK[fmt][0]), dtype=torch.float64, device=raw.device)
    if fmt == "q8_0":
        out[:] = ((i[..., 2:] + 128) % 256 - 128).double() * half(0)
    elif fmt == "q4_0":
        out[..., :16] = (i[..., 2:] % 16 - 8).double() * half(0)
        out[..., 16:] = (i[..., 2:] // 16 - 8).double() * half(0)
    elif fmt == "q5_0":
        for e in range(32):
            bit = i[..., 2 + e // 8] // 2 ** (e % 8) % 2
            low = i[..., 6 + e % 16]
            low = low % 16 if e < 16 else low // 16
            out[..., e] = (low + 16 * bit - 16).double() * half(0)[..., 0]
    elif fmt == "q4_k":
        for s in range(8):
            if s < 4:
                sc, m = i[..., 4 + s] % 64, i[..., 8 + s] % 64
            else:
                sc = i[..., 8 + s] % 16 + i[..., s] // 64 * 16
                m = i[..., 8 + s] // 16 + i[..., 4 + s] // 64 * 16
            code = i[..., 16 + 32 * (s // 2):48 + 32 * (s // 2)]
            code = code // 16 if s % 2 else code % 16
            out[..., 32 * s:32 * s + 32] = code * (sc.double() * half(0)[..., 0]).unsqueeze(-1) \
                - (m.double() * half(2)[..., 0]).unsqueeze(-1)
    else:
        for s in range(16):
            h, r, l = s // 8, s % 8 // 2, 16 * (s % 2)
            low = i[..., 64 * h + 32 * (r % 2) + l:64 * h + 32 * (r % 2) + l + 16]
            low = low // 16 if r >= 2 else low % 16
            top = i[..., 128 + 32 * h + l:128 + 32 * h + l + 16] // 4 ** r % 4
            sc = (i[..., 192 + s] + 128) % 256 - 128
            out[..., 16 * s:16 * s + 16] = (low + 16 * top - 32) * (sc.double() * half(208)[..., 0]).unsqueeze(-1)
    return out.reshape(rows, k)


def _exact_ffn(state):
    c = state["case"]
    x, y = state["x"].double(), torch.zeros((c["n_pos"], c["d"]), dtype=torch.float64, device=DEVICE)
    for e in torch.unique(state["ids"]).tolist():
        pos, slot = torch.nonzero(state["ids"] == e, as_tuple=True)
        gate = x[pos] @ _exact_rows(state["gate"][e], c["fmt"], c["d"]).T
        up = x[pos] @ _exact_rows(state["up"][e], c["fmt"], c["d"]).T
        if c["act"] == "swiglu":
            h = gate * torch.sigmoid(gate) * up
        else:
            # 1 + tanh z = 2 sigmoid(2 z)
            h = gate * torch.sigmoid(math.sqrt(8.0 / math.pi) * (gate + 0.044715 * gate ** 3)) * up
        y.index_add_(0, pos, (h @ _exact_rows(state["down"][e], c["fmt_down"], c["n_ff"]).T)
                     * state["weights"][pos, slot].double().unsqueeze(-1))
    return y


def _exact_linear(state):
    c = state["case"]
    t, h = c["n_new"], c["n_heads"]
    x = state["qkv"].double()
    w = c["n_qk"] * c["dk"]
    kv = torch.arange(h, device=DEVICE) // (h // c["n_qk"])
    q, k = x[..., :w].reshape(*x.shape[:2], c["n_qk"], -1), x[..., w:2 * w].reshape(*x.shape[:2], c["n_qk"], -1)
    v = x[..., 2 * w:].reshape(*x.shape[:2], h, -1)
    keep = torch.exp(state["decay"].double())
    lens = state["lens"].long()
    s = state["state"].double()
    s = torch.where(((lens <= t) & (lens > 0))[:, None, None, None], 0.0, s)
    out = torch.zeros((c["n_seqs"], t, h, c["dv"]), dtype=torch.float64, device=DEVICE)
    for i in range(t):
        on = (i >= t - lens)[:, None, None, None]
        a = keep[None] if c["constant"] else keep[:, i]
        s = torch.where(on, s * a[..., None, None] + k[:, i][:, kv].unsqueeze(-1) * v[:, i].unsqueeze(-2), s)
        o = (q[:, i][:, kv].unsqueeze(-2) @ s).squeeze(-2) / math.sqrt(c["dk"])
        out[:, i] = torch.where(on[..., 0], o, 0.0)
    return out, s


def exact(case, seed):
    state = prepare(case, seed)
    return {"route": _exact_route, "ffn": _exact_ffn, "linear": _exact_linear}[case["kind"]](state)
