"""The operators that complete a transformer layer in 8 bits, as they are measured: the gated pair of products of a feed-forward block (`gated`) and its
gradient (`gated_grad`), norms of queries and keys with the position rotation (`rotate`) and their gradient (`rotate_grad`), and attention of a batch
whose sequences share their first tokens (`shared`).

`run` computes a case in its plain form, or, where `own` is true, through the framework's entry points.  `exact` computes it in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TOP = 448.0          # largest E4M3 value
LEAST = 2.0 ** -100  # the quantizer's least amax
F8 = torch.float8_e4m3fn
CUBE = 0.044715      # of the tanh form of GELU


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token through a small block: latency
        {"name": "gated-one", "op": "gated", "m": 1, "n": 4096, "k": 4096, "act": "silu", "out": "bf16", "keep": False, "rows_k": False},
        # a decoding batch of 16 through the two up-projections, quantized for the down-projection: all of both weights is read
        {"name": "gated-decode", "op": "gated", "m": 16, "n": 28672, "k": 8192, "act": "silu", "out": "e4m3", "keep": False, "rows_k": False},
        # a training step's tokens, with what the gradient needs kept
        {"name": "gated-train", "op": "gated", "m": 4096, "n": 28672, "k": 8192, "act": "silu", "out": "e4m3", "keep": True, "rows_k": False},
        # ragged sizes, the other activation, BF16 out
        {"name": "gated-ragged", "op": "gated", "m": 1741, "n": 7000, "k": 4112, "act": "gelu", "out": "bf16", "keep": False, "rows_k": False},
        # the gradient of the training step's block: every operand of the products that come next
        {"name": "gated-grad-train", "op": "gated_grad", "r": 4096, "c": 28672, "act": "silu", "x": "bf16", "out": "e4m3"},
        # ragged sizes, BF16 gradients
        {"name": "gated-grad-ragged", "op": "gated_grad", "r": 1741, "c": 7000, "act": "gelu", "x": "f32", "out": "bf16"},
        # one new token for each of 64 sequences
        {"name": "rotate-token", "op": "rotate", "tokens": 64, "heads": 64, "kv": 8, "d": 128, "rot": 128, "interleaved": False, "x": "bf16",
         "norm": True, "far": 8192},
        # long prompts, pairs side by side, half of the head rotated, far positions
        {"name": "rotate-prompt", "op": "rotate", "tokens": 8192, "heads": 32, "kv": 8, "d": 128, "rot": 64, "interleaved": True, "x": "bf16",
         "norm": True, "far": 1000000},
        # the gradient on a training step's tokens
        {"name": "rotate-grad-train", "op": "rotate_grad", "tokens": 8192, "heads": 32, "kv": 8, "d": 128, "rot": 128, "interleaved": False,
         "x": "bf16", "norm": True, "far": 8192},
        # few tokens, small heads, FP32
        {"name": "rotate-grad-small", "op": "rotate_grad", "tokens": 333, "heads": 16, "kv": 4, "d": 64, "rot": 32, "interleaved": True, "x": "f32",
         "norm": True, "far": 131071},
        # a decoding batch behind one prompt of 8192 tokens
        {"name": "shared-token", "op": "shared", "batch": 64, "new": 1, "shared": 8192, "longest": 1000, "spread": 0.9, "heads": 64, "kv": 8,
         "d": 128, "page": 64},
        # four drafted tokens for each of 16 sequences behind a long document
        {"name": "shared-draft", "op": "shared", "batch": 16, "new": 4, "shared": 65536, "longest": 2047, "spread": 0.5, "heads": 32, "kv": 4,
         "d": 128, "page": 16},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "rotate", "rotate_grad", "shared", "shared"])
    if op == "gated":
        while True:
            m, n, k = _spread(rng, 1, 8192), _spread(rng, 16, 28672), _spread(rng, 1, 1024) * 16
            out, rows_k = rng.choice(["e4m3", "e4m3", "bf16", "f32"]), rng.random() < 0.25
            n = -(-n // 16) * 16 if rows_k or out == "e4m3" else n
            if 2e6 <= m * n * k <= 5e11 and m * n <= 4096 * 28672:
                return {"op": op, "m": m, "n": n, "k": k, "act": rng.choice(["silu", "gelu"]), "out": out, "keep": rng.random() < 0.4, "rows_k": rows_k}
    if op == "gated_grad":
        while True:
            out = rng.choice(["e4m3", "bf16"])
            r, c = _spread(rng, 1, 16384), _spread(rng, 16, 28672)
            c = -(-c // 16) * 16 if out == "e4m3" else c
            if 1e4 <= r * c <= 4096 * 28672:
                return {"op": op, "r": r, "c": c, "act": rng.choice(["silu", "gelu"]), "x": rng.choice(["bf16", "f32"]), "out": out}
    d, kv, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8, 16])
    if op != "shared":
        while True:
            tokens = _spread(rng, 1, 16384)
            if tokens * kv * (group + 1) * d <= 8192 * 40 * 128:
                return {"op": op, "tokens": tokens, "heads": kv * group, "kv": kv, "d": d, "rot": rng.choice([d, d, d // 2, d // 4]),
                        "interleaved": rng.random() < 0.5, "x": rng.choice(["bf16", "bf16", "f32"]), "norm": rng.random() < 0.7,
                        "far": _spread(rng, 100, 2000000)}
    page = rng.choice([16, 32, 64, 128])
    while True:
        batch, shared, longest = _spread(rng, 2, 128), _spread(rng, 100, 65536) // page * page, _spread(rng, 30, 8000)
        new = 1 if rng.random() < 0.6 else _spread(rng, 2, 64)
        if shared and new <= longest and batch * longest * kv * d <= 64 * 1000 * 8 * 128 * 2 and batch * new * kv * group * (shared + longest) <= 16 * 4 * 32 * 67000:
            return {"op": op, "batch": batch, "new": new, "shared": shared, "longest": longest, "spread": round(rng.random(), 2), "heads": kv * group,
                    "kv": kv, "d": d, "page": page}


def _lengths(case):
    """Tokens that each sequence holds behind the shared ones, and how many of them are new: the longest first."""
    b = case["batch"]
    after = [max(1, round(case["longest"] * (1 - case["spread"] * i / max(1, b - 1)))) for i in range(b)]
    return after, [min(t, case["new"]) for t in after]


def _blocks128(n):
    return -(-n // 128)


def work(case):
    op = case["op"]
    if op == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        out = m * n * {"e4m3": 1, "bf16": 2, "f32": 4}[case["out"]] + (4 * m * _blocks128(n) if case["out"] == "e4m3" else 0)
        return {"bytes": m * k + 2 * n * k + 4 * _blocks128(k) * (m + 2 * _blocks128(n)) + out + (4 * m * n if case["keep"] else 0), "flops": 4 * m * n * k}
    if op == "gated_grad":
        r, c = case["r"], case["c"]
        read = r * c * (4 + (2 if case["x"] == "bf16" else 4))
        if case["out"] == "bf16":
            return {"bytes": read + 4 * r * c, "flops": 12 * r * c}
        down = c * (-(-r // 16) * 16)
        return {"bytes": read + 2 * r * c + 3 * down + 4 * (2 * r * _blocks128(c) + 3 * c * _blocks128(r)), "flops": 12 * r * c}
    if op in ("rotate", "rotate_grad"):
        t, h, d, size = case["tokens"], case["heads"] + case["kv"], case["d"], 2 if case["x"] == "bf16" else 4
        passes = 2 if op == "rotate" else 3 if case["norm"] else 2
        return {"bytes": passes * t * h * d * size + 4 * t + 8 * (case["rot"] // 2) + (8 * d * (1 if op == "rotate" else 2) if case["norm"] else 0),
                "flops": t * h * (3 * case["rot"] + (4 * d if op == "rotate" else 9 * d) * case["norm"])}
    after, new = _lengths(case)
    kv, d, h, page, p = case["kv"], case["d"], case["heads"], case["page"], case["shared"]
    pairs = sum(n * (p + a - n) + n * (n + 1) // 2 for a, n in zip(after, new))
    return {"bytes": 2 * kv * d * (p + sum(after)) + 8 * kv * (-(-p // page) + sum(-(-a // page) for a in after)) + sum(new) * h * (4 * d + 4),
            "flops": 4 * h * d * pairs}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _empty8(rows, cols):
    """Codes of a rows x cols matrix with a scale for each 128 of a row."""
    return (torch.empty(rows, cols, device=DEV, dtype=torch.uint8), torch.empty(rows, _blocks128(cols), device=DEV))


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = _blocks128(k), _blocks128(n)
        # normal values, each block's largest near 448; scales that differ from block to block and give gates of a few units
        s["A"] = torch.randn(m, k, generator=g, device=DEV).mul_(100.0).clamp_(-TOP, TOP).to(F8).view(torch.uint8)
        s["sA"] = torch.exp(0.5 * torch.randn(m, kb, generator=g, device=DEV)) * 0.01
        for name in ("gate", "up"):
            w = torch.randn(n, k, generator=g, device=DEV).mul_(100.0).clamp_(-TOP, TOP).to(F8).view(torch.uint8)
            scale = torch.exp(0.3 * torch.randn(nb, kb, generator=g, device=DEV)) * (0.015 / math.sqrt(k))
            s["w_" + name], s["s_" + name] = (w.t().contiguous(), scale.t().contiguous()) if case["rows_k"] else (w, scale)
        if case["out"] == "e4m3":
            s["H"], s["sH"] = _empty8(m, n)
        else:
            s["H"], s["sH"] = torch.empty(m, n, device=DEV, dtype=_type(case["out"])), None
        for name in ("gate", "up"):
            s[name] = torch.empty(m, n, device=DEV, dtype=torch.bfloat16) if case["keep"] else None
        return s
    if op == "gated_grad":
        r, c = case["r"], case["c"]
        for name in ("gate", "up"):
            s[name] = (1.5 * torch.randn(r, c, generator=g, device=DEV)).to(torch.bfloat16)
        # gradients differ from token to token by orders of magnitude
        dh = torch.randn(r, c, generator=g, device=DEV) * torch.exp(torch.randn(r, 1, generator=g, device=DEV)) * 1e-4
        s["dH"] = dh.to(_type(case["x"]))
        if case["out"] == "bf16":
            s["out"] = {name: torch.empty(r, c, device=DEV, dtype=torch.bfloat16) for name in ("dgate", "dup")}
        else:
            s["out"] = {name: _empty8(r, c) for name in ("dgate_rows", "dup_rows")}
            tall = -(-r // 16) * 16
            for name in ("dgate_cols", "dup_cols", "hidden_cols"):
                s["out"][name] = (torch.empty(c, tall, device=DEV, dtype=torch.uint8), torch.empty(c, _blocks128(r), device=DEV))
        return s
    if op in ("rotate", "rotate_grad"):
        t, h, kv, d, rot = case["tokens"], case["heads"], case["kv"], case["d"], case["rot"]
        dt = _type(case["x"])
        # one buffer of a layer's queries, keys and values, as its projection writes it
        rows = torch.randn(t, (h + 2 * kv) * d, generator=g, device=DEV)
        rows *= torch.exp(0.5 * torch.randn(t, 1, generator=g, device=DEV))
        rows = rows.to(dt)
        s["q"], s["k"] = rows[:, :h * d].view(t, h, d), rows[:, h * d:(h + kv) * d].view(t, kv, d)
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV, dtype=torch.int32)
        base = 10000.0 if case["far"] <= 10000 else 500000.0  # long contexts turn more slowly
        s["freqs"] = base ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        s["factor"] = 1.0 if case["far"] <= 200000 else 1.2
        for name in ("q", "k"):
            s["w" + name] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV) if case["norm"] else None
            s[name + "_out"] = torch.empty(s[name].shape, device=DEV, dtype=dt)
            if op == "rotate_grad":
                s["d" + name] = (0.01 * torch.randn(s[name].shape, generator=g, device=DEV)).to(dt)
                s["dw" + name] = torch.empty(d, device=DEV) if case["norm"] else None
        return s
    after, new = _lengths(case)
    kv, d, page, h, p = case["kv"], case["d"], case["page"], case["heads"], case["shared"]
    total = [p + a for a in after]
    first = p // page
    need = [-(-t // page) - first for t in total]
    pages = first + sum(need) + 7  # a few free ones
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(total), first + max(need)), -1, device=DEV, dtype=torch.int32)
    table[:, :first] = order[:first]
    at = first
    for i, n in enumerate(need):
        table[i, first:first + n] = order[at:at + n]
        at += n
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s.update(table=table, kv_len=torch.tensor(total, device=DEV, dtype=torch.int32), q_start=torch.tensor(start, device=DEV, dtype=torch.int32),
             tokens=start[-1])
    # pages hold what their scale was chosen for; places past a sequence's end hold whatever was there, NaN codes among it
    used = torch.zeros(pages, page, dtype=torch.bool, device=DEV)
    place = torch.arange(table.shape[1] * page, device=DEV)
    inside = (place[None] < s["kv_len"][:, None]).view(len(total), -1, page)
    used[table[table >= 0].long()] = inside[table >= 0]
    for name in ("K", "V"):
        codes = torch.randn(pages, kv, page, d, generator=g, device=DEV).mul_(120.0).clamp_(-TOP, TOP).to(F8).view(torch.uint8)
        s[name] = torch.where(used[:, None, :, None], codes, torch.full_like(codes, 0x7F))
        s["s" + name] = torch.exp2(torch.randint(-9, -5, (pages, kv), generator=g, device=DEV).float())
    s["Q"] = torch.randn(start[-1], h, d, generator=g, device=DEV).to(torch.bfloat16)
    s["O"] = torch.empty(start[-1], h, d, device=DEV, dtype=torch.bfloat16)
    s["lse"] = torch.empty(start[-1], h, device=DEV, dtype=torch.float32)
    return s


# ---------------------------------------------------------------- plain forms
def _sigmoid_of(g, act):
    """(what multiplies g in the activation, the derivative of its argument)."""
    if act == "silu":
        return 1 / (1 + torch.exp(-g)), 1.0
    c = 2 * math.sqrt(2 / math.pi)
    return 1 / (1 + torch.exp(-c * (g + CUBE * g * g * g))), c * (1 + 3 * CUBE * g * g)


def _quantize(x, cols=False):
    """(values of the codes, scales) of x by blocks of 128 along its rows, or down its columns and stored transposed."""
    r, c = x.shape
    if cols:
        x = torch.nn.functional.pad(x, (0, 0, 0, -r % 16)).t()
    n = x.shape[1]
    b = torch.nn.functional.pad(x, (0, -n % 128)).reshape(x.shape[0], -1, 128)
    top = b.abs().amax(2, keepdim=True).clamp(min=LEAST)
    codes = (b * torch.div(torch.full_like(top, TOP), top)).clamp(-TOP, TOP).view(x.shape[0], -1)[:, :n]
    return {"codes": codes.to(F8), "scales": (top / TOP)[..., 0]}


def _gated(s):
    c = s["case"]
    k, n = c["k"], c["n"]
    a = s["A"].view(F8).float() * s["sA"].repeat_interleave(128, 1)[:, :k]

    def product(w, scale):
        if c["rows_k"]:
            return a @ (w.view(F8).float() * scale.repeat_interleave(128, 0)[:k].repeat_interleave(128, 1)[:, :n])
        return a @ (w.view(F8).float() * scale.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]).t()

    g, u = product(s["w_gate"], s["s_gate"]), product(s["w_up"], s["s_up"])
    h = g * _sigmoid_of(g, c["act"])[0] * u
    out = _quantize(h) if c["out"] == "e4m3" else {"h": h.to(s["H"].dtype)}
    return {**out, "gate": g.to(torch.bfloat16), "up": u.to(torch.bfloat16)} if c["keep"] else out


def _gated_grad(s):
    act = s["case"]["act"]
    g, u, dh = s["gate"].float(), s["up"].float(), s["dH"].float()
    p, slope = _sigmoid_of(g, act)
    a = g * p
    dg, du = dh * u * (p + a * (1 - p) * slope), dh * a
    if s["case"]["out"] == "bf16":
        return {"dgate": dg.to(torch.bfloat16), "dup": du.to(torch.bfloat16)}
    return {"dgate_rows": _quantize(dg), "dup_rows": _quantize(du), "dgate_cols": _quantize(dg, True), "dup_cols": _quantize(du, True),
            "hidden_cols": _quantize(a * u, True)}


EPS = 1e-6


def _turn(x, cos, sin, rot, interleaved):
    """The first `rot` values of each head turned by the angles: pairs (i, i + rot / 2), or (2 i, 2 i + 1)."""
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    one, two = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = one, two
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = one, two
    return y


def _angles(s):
    """Cosines and sines of each token's angles times the factor; the angles in 64 bits."""
    w = s["positions"].double()[:, None] * s["freqs"]
    return (torch.cos(w) * s["factor"]).float()[:, None], (torch.sin(w) * s["factor"]).float()[:, None]


def _rotate(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        if c["norm"]:
            x = x / torch.sqrt((x * x).mean(2, keepdim=True) + EPS) * s["w" + name]
        out[name] = _turn(x, cos, sin, c["rot"], c["interleaved"]).to(s[name].dtype)
    return out


def _rotate_grad(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = {}
    for name in ("q", "k"):
        dn = _turn(s["d" + name].float(), cos, -sin, c["rot"], c["interleaved"])
        if c["norm"]:
            x = s[name].float()
            inv = 1 / torch.sqrt((x * x).mean(2, keepdim=True) + EPS)
            hat = x * inv
            out["dw" + name] = (dn * hat).sum((0, 1), dtype=torch.float64).float()
            dn = dn * s["w" + name]
            dn = inv * (dn - hat * (dn * hat).mean(2, keepdim=True))
        out["d" + name] = dn.to(s[name].dtype)
    return out


def _shared(s):
    c = s["case"]
    b, page, h, kv, d, p, most = c["batch"], c["page"], c["heads"], c["kv"], c["d"], c["shared"], c["new"]
    g = h // kv
    n = s["q_start"].diff()
    seq = torch.repeat_interleave(torch.arange(b, device=DEV), n, output_size=s["tokens"])
    at = torch.arange(s["tokens"], device=DEV) - s["q_start"][seq]
    q = s["Q"].float().view(-1, kv, g, d)

    def keys(table):
        return ((s[x][table].view(F8).float() * s["s" + x][table][..., None, None]).transpose(-4, -3).flatten(-3, -2) for x in ("K", "V"))

    # scores against the shared keys, once for all, and against the sequence's own
    k0, v0 = keys(s["table"][0, :p // page].long())
    k1, v1 = keys(s["table"][:, p // page:].clamp(min=0).long())
    place = p + torch.arange(k1.shape[2], device=DEV)
    inside = place < s["kv_len"][:, None]
    v1 = torch.where(inside[:, None, :, None], v1, 0.0)
    own_q = torch.zeros(b, most, kv, g, d, device=DEV)
    own_q[seq, at] = q
    own_q = own_q.permute(0, 2, 3, 1, 4).reshape(b, kv, g * most, d)
    x0 = (q.permute(1, 2, 0, 3).reshape(kv, -1, d) @ k0.transpose(1, 2)).view(kv, g, -1, p).permute(2, 0, 1, 3) / math.sqrt(d)
    x1 = (own_q @ k1.transpose(2, 3)).view(b, kv, g, most, -1).permute(0, 3, 1, 2, 4)[seq, at] / math.sqrt(d)
    pos = (s["kv_len"] - n)[seq] + at
    x1 = torch.where((inside[seq] & (place <= pos[:, None]))[:, None, None], x1, -math.inf)
    top = torch.maximum(x0.amax(3, keepdim=True), x1.amax(3, keepdim=True))
    w0, w1 = torch.exp(x0 - top), torch.exp(x1 - top)
    total = w0.sum(3, keepdim=True) + w1.sum(3, keepdim=True)
    o0 = (w0.permute(1, 2, 0, 3).reshape(kv, -1, p) @ v0).view(kv, g, -1, d).permute(2, 0, 1, 3)
    own_w = torch.zeros(b, most, kv, g, w1.shape[3], device=DEV)
    own_w[seq, at] = w1
    o1 = (own_w.permute(0, 2, 3, 1, 4).reshape(b, kv, g * most, -1) @ v1).view(b, kv, g, most, d).permute(0, 3, 1, 2, 4)[seq, at]
    return {"o": ((o0 + o1) / total).reshape(-1, h, d).to(torch.bfloat16), "lse": (top + torch.log(total)).view(-1, h)}


# ---------------------------------------------------------------- the framework's calls
_kept = {}


def _handle(mx, rows_k=False):
    """The program's handles: one for each way that the weights lie."""
    if rows_k not in _kept:
        h = _kept[rows_k] = mx.mxgemm_create(torch.cuda.current_device())
        mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_K_BY_N if rows_k else mx.B_N_BY_K)
    return _kept[rows_k]


def _as_values(pair):
    return {"codes": pair[0].view(F8), "scales": pair[1]}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"gated": _gated, "gated_grad": _gated_grad, "rotate": _rotate, "rotate_grad": _rotate_grad, "shared": _shared}[op](s)
    import block_scaled_gemm_gb300 as mx
    stream = torch.cuda.current_stream()
    if op in ("gated", "gated_grad"):
        act = mx.ACT_SILU if c["act"] == "silu" else mx.ACT_GELU_TANH
    if op == "gated":
        mx.mxgemm_run_gated_block128(_handle(mx, c["rows_k"]), c["m"], c["n"], c["k"], s["A"], s["sA"], s["w_gate"], s["s_gate"], s["w_up"], s["s_up"],
                                     s["H"], H_scale=s["sH"], act=act, out_dtype={"e4m3": mx.OUT_E4M3, "bf16": mx.OUT_BF16, "f32": mx.OUT_F32}[c["out"]],
                                     gate=s["gate"], up=s["up"], stream=stream)
        out = _as_values((s["H"], s["sH"])) if c["out"] == "e4m3" else {"h": s["H"]}
        return {**out, "gate": s["gate"], "up": s["up"]} if c["keep"] else out
    if op == "gated_grad":
        mx.mxgemm_gated_backward(s["gate"], s["up"], s["dH"], c["r"], c["c"], act=act, stream=stream, **s["out"])
        return s["out"] if c["out"] == "bf16" else {name: _as_values(pair) for name, pair in s["out"].items()}
    if op == "rotate":
        mx.mxgemm_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], positions=s["positions"], freqs=s["freqs"], interleaved=c["interleaved"],
                            factor=s["factor"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS, stream=stream)
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "rotate_grad":
        mx.mxgemm_norm_rope_backward(_handle(mx), s["dq"], s["dk"], s["q_out"], s["k_out"], q=s["q"], k=s["k"], positions=s["positions"],
                                     freqs=s["freqs"], interleaved=c["interleaved"], factor=s["factor"], q_weight=s["wq"], k_weight=s["wk"],
                                     dq_weight=s["dwq"], dk_weight=s["dwk"], eps=EPS, stream=stream)
        out = {"dq": s["q_out"], "dk": s["k_out"]}
        return {"dwq": s["dwq"], "dq": out["dq"], "dwk": s["dwk"], "dk": out["dk"]} if c["norm"] else out
    cache = mx.Cache(s["K"], s["V"], s["sK"], s["sV"])
    starts = s["q_start"] if c["new"] > 1 else None  # one token each: no starts are needed
    mx.mxgemm_cache_attention_shared(_handle(mx), cache, s["table"], s["kv_len"], c["shared"], s["Q"], s["O"], q_start=starts, lse=s["lse"], stream=stream)
    return {"o": s["O"], "lse": s["lse"]}


# ---------------------------------------------------------------- in 64 bits
def _e4m3(y):
    """The nearest E4M3 value, ties to even, in 64 bits."""
    y = y.clamp(-TOP, TOP)
    step = torch.exp2(torch.frexp(y)[1].clamp(min=-5).double() - 4)
    return torch.round(y / step) * step


def _value(codes):
    """The values of E4M3 codes in 64 bits, by the format's definition."""
    c = codes.int()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    v = torch.where((c & 127) == 127, math.nan, v)
    return torch.where(c >= 128, -v, v)


def _blocks64(x, cols=False):
    """Codes' values and scales by the quantizer's definition, a strip of 128 at a time along the blocks."""
    r, c = x.shape
    n = r if cols else c
    codes, scales = [], []
    for j in range(0, n, 128):
        part = x[j:j + 128].t() if cols else x[:, j:j + 128]
        top = part.abs().amax(1, keepdim=True).clamp(min=LEAST)
        codes.append(_e4m3(part * (TOP / top)))
        scales.append(top / TOP)
    if cols and r % 16:
        codes.append(torch.zeros(c, 16 - r % 16, device=DEV, dtype=torch.float64))
    return {"codes": torch.cat(codes, 1), "scales": torch.cat(scales, 1)}


def _act64(g, act):
    """The activation and its derivative."""
    if act == "silu":
        t = torch.tanh(g / 2)
        return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 4
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + CUBE * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 2 * c * (1 + 3 * CUBE * g ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        if m * n * k > 1e12:
            return None
        row = torch.arange(n, device=DEV) // 128
        sums = []
        for name in ("gate", "up"):
            w, scale = s["w_" + name], s["s_" + name].double()
            if case["rows_k"]:
                w, scale = w.t(), scale.t()
            total = torch.zeros(m, n, device=DEV, dtype=torch.float64)
            for j in range(0, k, 1024):  # eight blocks at a time
                at = torch.arange(j, min(k, j + 1024), device=DEV)
                total += (_value(s["A"][:, at]) * s["sA"].double()[:, at // 128]) @ (_value(w[:, at]) * scale[row][:, at // 128]).t()
            sums.append(total)
        g, u = sums
        h = _act64(g, case["act"])[0] * u
        out = _blocks64(h) if case["out"] == "e4m3" else {"h": h}
        return {**out, "gate": g, "up": u} if case["keep"] else out
    if op == "gated_grad":
        g, u, dh = s["gate"].double(), s["up"].double(), s["dH"].double()
        a, slope = _act64(g, case["act"])
        dg, du = dh * u * slope, dh * a
        del slope, g, dh
        if case["out"] == "bf16":
            return {"dgate": dg, "dup": du}
        return {"dgate_rows": _blocks64(dg), "dup_rows": _blocks64(du), "dgate_cols": _blocks64(dg, True), "dup_cols": _blocks64(du, True),
                "hidden_cols": _blocks64(a * u, True)}
    if op in ("rotate", "rotate_grad"):
        rot, d = case["rot"], case["d"]
        i = torch.arange(rot // 2, device=DEV)
        one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        # turned as complex numbers
        angle = s["positions"].double()[:, None] * s["freqs"]
        turn = torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]
        out = {}
        for name in ("q", "k"):
            x = s[name].double()
            w = s["w" + name].double() if case["norm"] else torch.ones(d, device=DEV, dtype=torch.float64)
            rms = torch.sqrt(x.square().mean(2, keepdim=True) + EPS) if case["norm"] else torch.ones_like(x[..., :1])
            if op == "rotate":
                y = x / rms * w
                z = torch.complex(y[..., one], y[..., two]) * turn
                y[..., one], y[..., two] = z.real, z.imag
                out[name] = y
                continue
            dy = s["d" + name].double()
            z = torch.complex(dy[..., one], dy[..., two]) * turn.conj()
            dy[..., one], dy[..., two] = z.real, z.imag
            if case["norm"]:
                out["dw" + name] = (dy * x / rms).sum((0, 1))
                dy = dy * w
                dy = dy / rms - x * (dy * x).sum(2, keepdim=True) / (d * rms ** 3)
            out["d" + name] = dy
        return out
    after, new = _lengths(case)
    page, kv, d, h, p = case["page"], case["kv"], case["d"], case["heads"], case["shared"]
    g = h // kv
    table, start = s["table"].long(), s["q_start"].tolist()
    o = torch.zeros(start[-1], h, d, device=DEV, dtype=torch.float64)
    lse = torch.zeros(start[-1], h, device=DEV, dtype=torch.float64)
    for b, (a, n) in enumerate(zip(after, new)):
        t = p + a
        at = table[b, :-(-t // page)]
        hidden = torch.arange(t - n, t, device=DEV)[:, None] < torch.arange(t, device=DEV)[None]
        for i in range(kv):
            k, v = ((_value(s[x][at, i]) * s["s" + x][at, i].double()[:, None, None]).reshape(-1, d)[:t] for x in ("K", "V"))
            q = s["Q"][start[b]:start[b + 1], i * g:i * g + g].double()
            w = (q @ k.t() / math.sqrt(d)).masked_fill(hidden[:, None], -math.inf)
            lse[start[b]:start[b + 1], i * g:i * g + g] = torch.logsumexp(w, 2)
            o[start[b]:start[b + 1], i * g:i * g + g] = torch.softmax(w, 2) @ v
    return {"o": o, "lse": lse}
