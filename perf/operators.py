"""The operators of 8-bit layers, as they are measured: the product with a scale for each block of 128 (`product`), the quantizer that makes its
operands (`quantize`), and the 8-bit key/value cache's append (`append`) and attention (`attend`).

`run` computes a case in its plain form, or, where `own` is true, through the framework's entry points.  `exact` computes it in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TOP = 448.0          # largest E4M3 value
LEAST = 2.0 ** -100  # the quantizer's least amax
FLOOR = 2.0 ** -64   # the cache's least scale
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a linear layer on a decoding batch of 16: all of the weight is read for little arithmetic
        {"name": "product-decode", "op": "product", "m": 16, "n": 8192, "k": 8192, "b_rows_k": False, "b_block": 128, "out": "bf16"},
        # an MLP up-projection on 8192 tokens
        {"name": "product-forward", "op": "product", "m": 8192, "n": 28672, "k": 8192, "b_rows_k": False, "b_block": 128, "out": "bf16"},
        # the gradient of a layer's input, from the weight as it lies (contracted over its rows); ragged tokens
        {"name": "product-grad-input", "op": "product", "m": 5000, "n": 4112, "k": 8192, "b_rows_k": True, "b_block": 128, "out": "f32"},
        # the gradient of a weight: contracted over 5000 tokens (stored to a multiple of 16), a scale for each column of both operands
        {"name": "product-grad-weight", "op": "product", "m": 4096, "n": 4096, "k": 5008, "b_rows_k": False, "b_block": 1, "out": "f32"},
        # activations before a product
        {"name": "quantize-rows", "op": "quantize", "r": 8192, "c": 8192, "block": "rows", "x": "bf16"},
        # activations for a weight's gradient: blocks of 128 tokens, stored with the tokens along the rows
        {"name": "quantize-columns", "op": "quantize", "r": 5000, "c": 4096, "block": "cols", "x": "f32"},
        # one new token for each of 64 sequences
        {"name": "append-token", "op": "append", "batch": 64, "new": 1, "longest": 4000, "spread": 0.9, "kv": 8, "d": 128, "page": 64, "x": "bf16"},
        # the prompts of four sequences, ragged, after what their caches hold
        {"name": "append-prompt", "op": "append", "batch": 4, "new": 2500, "longest": 6001, "spread": 0.5, "kv": 8, "d": 128, "page": 64, "x": "bf16"},
        # one sequence, a short window and four first tokens: latency alone
        {"name": "attend-token-window", "op": "attend", "batch": 1, "new": 1, "longest": 2047, "spread": 0.0, "heads": 32, "kv": 8, "d": 128,
         "page": 16, "window": 512, "sinks": 4},
        # an ordinary decoding batch
        {"name": "attend-token-batch", "op": "attend", "batch": 64, "new": 1, "longest": 8192, "spread": 0.75, "heads": 64, "kv": 8, "d": 128,
         "page": 64, "window": 0, "sinks": 0},
        # two very long sequences
        {"name": "attend-token-long", "op": "attend", "batch": 2, "new": 1, "longest": 131071, "spread": 0.3, "heads": 32, "kv": 4, "d": 128,
         "page": 128, "window": 0, "sinks": 0},
        # a chunk of a prompt behind a prefix
        {"name": "attend-prompt", "op": "attend", "batch": 2, "new": 2048, "longest": 8190, "spread": 0.3, "heads": 32, "kv": 8, "d": 128,
         "page": 64, "window": 0, "sinks": 0},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["product", "quantize", "append", "attend", "attend"])
    if op == "product":
        while True:
            m, n, k = _spread(rng, 1, 8192), _spread(rng, 16, 16384), _spread(rng, 1, 1024) * 16
            rows_k, block = rng.choice([(False, 128), (True, 128), (False, 1)])
            n = -(-n // 16) * 16 if rows_k else n
            if 2e6 <= m * n * k <= 5e11 and 3072 not in (m, n, k):
                return {"op": op, "m": m, "n": n, "k": k, "b_rows_k": rows_k, "b_block": block, "out": rng.choice(["bf16", "f32"])}
    if op == "quantize":
        while True:
            r, c = _spread(rng, 1, 16384), _spread(rng, 1, 1024) * 16
            if 1e4 <= r * c <= 8192 * 8192 and 3072 not in (r, c):
                return {"op": op, "r": r, "c": c, "block": rng.choice(["rows", "cols", "tiles"]), "x": rng.choice(["bf16", "f32"])}
    d, page, kv = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8])
    while True:
        batch, longest = _spread(rng, 1, 64), _spread(rng, 30, 100000)
        new = 1 if rng.random() < 0.5 else _spread(rng, 2, 2000)
        group = rng.choice([1, 2, 4, 7, 8, 16])
        rows = batch * kv * group * min(new, longest)
        if 3072 in (batch, longest, new) or batch * longest * kv * d > 64 * 8192 * 8 * 128 or batch * min(new, longest) > 16384:
            continue
        if op == "append":
            return {"op": op, "batch": batch, "new": new, "longest": longest, "spread": round(rng.random(), 2), "kv": kv, "d": d, "page": page,
                    "x": rng.choice(["bf16", "f32"])}
        if rows * longest <= 2 * 32 * 2048 * 8190:
            window = rng.choice([0, 0, _spread(rng, 1, longest)])
            return {"op": op, "batch": batch, "new": new, "longest": longest, "spread": round(rng.random(), 2), "heads": kv * group, "kv": kv,
                    "d": d, "page": page, "window": 0 if window == 3072 else window, "sinks": rng.choice([0, 1, 4]) if window else 0}


def _lengths(case):
    """Tokens that each sequence holds after its new ones, and how many of them are new: the longest first."""
    b = case["batch"]
    total = [max(1, round(case["longest"] * (1 - case["spread"] * i / max(1, b - 1)))) for i in range(b)]
    new = [max(1, min(t, round(case["new"] * (1 - 0.5 * case["spread"] * i / max(1, b - 1))))) for i, t in enumerate(total)]
    return total, new


def _visible(total, new, window, sinks):
    """Pairs of a query and a key that it sees, and how many keys any query sees."""
    p = range(total - new, total)
    if not window:
        return sum(i + 1 for i in p), total
    pairs = sum(min(i + 1, window) + min(sinks, max(0, i + 1 - window)) for i in p)
    first = max(0, total - new - window + 1)
    return pairs, total - first + min(sinks, first)


def work(case):
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // 128)
        scales = 4 * kb * (m + (n if case["b_block"] == 1 else -(-n // 128)))
        return {"bytes": m * k + n * k + scales + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    if case["op"] == "quantize":
        r, c = case["r"], case["c"]
        blocks = {"rows": r * -(-c // 128), "cols": c * -(-r // 128), "tiles": -(-r // 128) * -(-c // 128)}[case["block"]]
        return {"bytes": r * c * ((2 if case["x"] == "bf16" else 4) + 1) + 4 * blocks, "flops": 2 * r * c}
    total, new = _lengths(case)
    kv, d, page = case["kv"], case["d"], case["page"]
    if case["op"] == "append":
        t = sum(new)
        pages = sum(-(-a // page) - (a - b) // page for a, b in zip(total, new))
        return {"bytes": 2 * t * kv * d * ((2 if case["x"] == "bf16" else 4) + 1) + 8 * kv * pages, "flops": 4 * t * kv * d}
    seen = [_visible(a, b, case["window"], case["sinks"]) for a, b in zip(total, new)]
    t, h = sum(new), case["heads"]
    return {"bytes": 2 * kv * d * sum(s for _, s in seen) + 8 * kv * sum(-(-s // page) for _, s in seen) + t * h * (4 * d + 4),
            "flops": 4 * h * d * sum(p for p, _ in seen)}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _codes(x, scale):
    return (x / scale).clamp(-TOP, TOP).to(F8).view(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // 128)
        nb = n if case["b_block"] == 1 else -(-n // 128)
        # activations and weights: normal values, each block's largest near 448, scales that differ from block to block
        a = torch.randn(m, k, generator=g, device=DEV).mul_(100.0).clamp_(-TOP, TOP).to(F8)
        b = torch.randn(n, k, generator=g, device=DEV).mul_(100.0).clamp_(-TOP, TOP).to(F8)
        sa = torch.exp(torch.randn(m, kb, generator=g, device=DEV)) * 0.01
        sb = torch.exp(0.3 * torch.randn(nb, kb, generator=g, device=DEV)) * 0.0002
        if case["b_rows_k"]:
            b, sb = b.view(torch.uint8).t().contiguous(), sb.t().contiguous()
        s.update(A=a.view(torch.uint8), B=b.view(torch.uint8), sA=sa, sB=sb,
                 C=torch.empty(m, n, device=DEV, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32))
        return s
    if case["op"] == "quantize":
        r, c = case["r"], case["c"]
        x = torch.randn(r, c, generator=g, device=DEV)
        x *= torch.where(torch.rand(r, c, generator=g, device=DEV) < 0.001, 50.0, 1.0)  # activations have outliers
        shape = {"rows": (r, -(-c // 128)), "cols": (c, -(-r // 128)), "tiles": (-(-r // 128), -(-c // 128))}[case["block"]]
        s.update(X=x.to(torch.bfloat16) if case["x"] == "bf16" else x,
                 codes=torch.empty((c, -(-r // 16) * 16) if case["block"] == "cols" else (r, c), device=DEV, dtype=torch.uint8),
                 scales=torch.empty(shape, device=DEV, dtype=torch.float32))
        return s
    total, new = _lengths(case)
    kv, d, page = case["kv"], case["d"], case["page"]
    width = max(-(-t // page) for t in total)
    need = sum(-(-t // page) for t in total)
    pages = need + 7  # a few free ones
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(total), width), -1, device=DEV, dtype=torch.int32)
    at = 0
    for i, t in enumerate(total):
        k = -(-t // page)
        table[i, :k] = order[at:at + k]
        at += k
    start = [0]
    for b in new:
        start.append(start[-1] + b)
    # pages hold what their scale was chosen for; places past a sequence's end hold whatever was there, NaN codes among it
    s.update(table=table, kv_len=torch.tensor(total, device=DEV, dtype=torch.int32), q_start=torch.tensor(start, device=DEV, dtype=torch.int32), tokens=start[-1])
    for name in ("K", "V"):
        scale = torch.exp2(torch.randint(-9, -5, (pages, kv), generator=g, device=DEV).float())
        codes = torch.randn(pages, kv, page, d, generator=g, device=DEV).mul_(120.0).clamp_(-TOP, TOP).to(F8).view(torch.uint8)
        last, used = order[:need].long(), torch.zeros(pages, page, dtype=torch.bool, device=DEV)
        place = torch.arange(width * page, device=DEV)
        inside = (place[None] < s["kv_len"][:, None]).view(len(total), width, page)
        used[table.clamp(min=0).long()[table >= 0]] = inside[table >= 0]
        codes = torch.where(used[:, None, :, None], codes, torch.full_like(codes, 0x7F))
        s[name], s["s" + name] = codes, scale
    if case["op"] == "append":
        dt = torch.bfloat16 if case["x"] == "bf16" else torch.float32
        # one buffer of a layer's queries, keys and values, as its projection writes it: the keys and values are slices of its rows
        rows = torch.randn(start[-1], 4 * kv * d, generator=g, device=DEV)
        rows *= torch.exp(0.5 * torch.randn(start[-1], 1, generator=g, device=DEV))
        rows = rows.to(dt)
        # the pages that the new tokens touch, as the program that handed them out knows them
        s["pages"] = torch.cat([table[i, (t - b) // page:-(-t // page)] for i, (t, b) in enumerate(zip(total, new))]).long()
        s["newK"] = rows[:, 2 * kv * d:3 * kv * d].view(start[-1], kv, d)
        s["newV"] = rows[:, 3 * kv * d:].view(start[-1], kv, d)
        return s
    h = case["heads"]
    s["Q"] = torch.randn(start[-1], h, d, generator=g, device=DEV).to(torch.bfloat16)
    s["O"] = torch.empty(start[-1], h, d, device=DEV, dtype=torch.bfloat16)
    s["lse"] = torch.empty(start[-1], h, device=DEV, dtype=torch.float32)
    return s


# ---------------------------------------------------------------- plain forms
def _product(s):
    c = s["case"]
    a = s["A"].view(F8).float() * s["sA"].repeat_interleave(128, 1)[:, :c["k"]]
    b, sb = s["B"].view(F8).float(), s["sB"]
    if c["b_rows_k"]:
        b = b * sb.repeat_interleave(128, 0)[:c["k"]].repeat_interleave(128, 1)[:, :c["n"]]
    else:
        sb = sb if c["b_block"] == 1 else sb.repeat_interleave(128, 0)[:c["n"]]
        b = (b * sb.repeat_interleave(128, 1)[:, :c["k"]]).t()
    return (a @ b).to(s["C"].dtype)


def _blocks(x, block):
    """x, padded to whole blocks, as (blocks down, rows of one, blocks across, columns of one)."""
    r, c = x.shape
    br, bc = (1 if block == "rows" else 128), (1 if block == "cols" else 128)
    x = torch.nn.functional.pad(x, (0, -c % bc, 0, -r % br))
    return x.view(x.shape[0] // br, br, x.shape[1] // bc, bc)


def _quantize(s):
    block, (r, c) = s["case"]["block"], s["X"].shape
    x = _blocks(s["X"].float(), block)
    top = x.abs().amax((1, 3), keepdim=True).clamp(min=LEAST)
    codes = (x * torch.div(torch.full_like(top, TOP), top)).clamp(-TOP, TOP).view(-1, x.shape[2] * x.shape[3])[:r, :c]
    scales = (top / TOP)[:, 0, :, 0]
    if block == "cols":
        codes, scales = torch.nn.functional.pad(codes.t(), (0, -r % 16)), scales.t()
    return {"codes": codes.contiguous().to(F8), "scales": scales.contiguous()}


def _pow2(amax):
    """The least power of two that is amax / 448 or more, and FLOOR at least."""
    f, e = torch.frexp(amax)
    least = torch.ldexp(torch.ones_like(amax), torch.where(f <= 0.875, e - 9, e - 8))
    return torch.where(amax > 0, least, 0.0).clamp(min=FLOOR)


def _append(s):
    page, pages = s["case"]["page"], s["pages"]
    n = s["q_start"].diff()
    first = (s["kv_len"] - n).long()
    seq = torch.repeat_interleave(torch.arange(len(n), device=DEV), n, output_size=s["tokens"])
    pos = torch.arange(s["tokens"], device=DEV) - s["q_start"][seq] + first[seq]
    row = pos % page
    at = torch.zeros(s["K"].shape[0], dtype=torch.int64, device=DEV).index_copy_(0, pages, torch.arange(len(pages), device=DEV))
    to = at[s["table"][seq, pos // page].long()]  # the place of a token's page in `pages`
    # tokens that a page held before
    kept = torch.zeros(len(pages), device=DEV).index_reduce_(0, to, (first[seq] - pos + row).clamp(min=0).float(), "amax")
    old = torch.arange(page, device=DEV)[None] < kept[:, None]
    out = {}
    for name in ("K", "V"):
        codes, scale, x = s[name][pages], s["s" + name][pages], s["new" + name].float()
        want = _pow2(torch.zeros_like(scale).index_reduce_(0, to, x.abs().amax(2), "amax"))
        want = torch.where((kept > 0)[:, None], torch.maximum(scale, want), want)
        again = (codes.view(F8).float() * (scale / want)[:, :, None, None]).clamp(-TOP, TOP).to(F8).view(torch.uint8)
        codes = torch.where(old[:, None, :, None], again, codes)
        codes.permute(0, 2, 1, 3)[to, row] = (x / want[to][:, :, None]).clamp(-TOP, TOP).to(F8).view(torch.uint8)
        out[name], out["s" + name] = s[name].index_copy_(0, pages, codes).view(F8), s["s" + name].index_copy_(0, pages, want)
    return out


def _attend(s):
    c = s["case"]
    b, page, h, kv, d = c["batch"], c["page"], c["heads"], c["kv"], c["d"]
    table = s["table"].clamp(min=0).long()
    length = table.shape[1] * page
    n = s["q_start"].diff()
    key = torch.arange(length, device=DEV)
    inside = key[None] < s["kv_len"][:, None]
    k, v = ((s[x][table].view(F8).float() * s["s" + x][table][..., None, None]).transpose(1, 2).reshape(b, kv, length, d) for x in ("K", "V"))
    v = torch.where(inside[:, None, :, None], v, 0.0)
    most = max(_lengths(c)[1])
    seq = torch.repeat_interleave(torch.arange(b, device=DEV), n, output_size=s["tokens"])
    at = torch.arange(s["tokens"], device=DEV) - s["q_start"][seq]
    q = torch.zeros(b, most, h, d, device=DEV)
    q[seq, at] = s["Q"].float()
    q = q.view(b, most, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(b, kv, h // kv * most, d)
    score = ((q @ k.transpose(2, 3)) * (1 / math.sqrt(d))).view(b, h, most, length)
    pos = (s["kv_len"] - n)[:, None] + torch.arange(most, device=DEV)[None]
    far = pos[:, :, None] - key
    seen = inside[:, None] & (far >= 0)
    if c["window"]:
        seen &= (far < c["window"]) | (key < c["sinks"])
    score = torch.where(seen[:, None], score, -math.inf)
    top = score.amax(3, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(3, keepdim=True)
    o = (p.view(b, kv, h // kv * most, length) @ v).view(b, h, most, d) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    return {"o": o.transpose(1, 2)[seq, at].to(torch.bfloat16), "lse": lse.transpose(1, 2)[seq, at]}


# ---------------------------------------------------------------- the framework's calls
_kept = {}


def _handle(mx, b_rows_k):
    """The program's handles: one for each way that the second operand lies."""
    if b_rows_k not in _kept:
        h = _kept[b_rows_k] = mx.mxgemm_create(torch.cuda.current_device())
        mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_K_BY_N if b_rows_k else mx.B_N_BY_K)
    return _kept[b_rows_k]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"product": _product, "quantize": _quantize, "append": _append, "attend": _attend}[op](s)
    import block_scaled_gemm_gb300 as mx
    stream = torch.cuda.current_stream()
    if op == "product":
        mx.mxgemm_run_block128(_handle(mx, c["b_rows_k"]), c["m"], c["n"], c["k"], s["A"], s["sA"], s["B"], s["sB"], s["C"], use_acc=0,
                               out_dtype=mx.OUT_BF16 if c["out"] == "bf16" else mx.OUT_F32, b_block=c["b_block"], stream=stream)
        return s["C"]
    if op == "quantize":
        block = {"rows": mx.BLOCK_ROWS, "cols": mx.BLOCK_COLS, "tiles": mx.BLOCK_TILES}[c["block"]]
        mx.mxgemm_quantize_block128(s["X"], c["r"], c["c"], s["codes"], s["scales"], block=block, stream=stream)
        return {"codes": s["codes"].view(F8), "scales": s["scales"]}
    cache = mx.Cache(s["K"], s["V"], s["sK"], s["sV"])
    starts = s["q_start"] if c["new"] > 1 else None  # one token each: no starts are needed
    if op == "append":
        mx.mxgemm_cache_append(_handle(mx, False), cache, s["table"], s["kv_len"], s["newK"], s["newV"], q_start=starts, stream=stream)
        return {"K": s["K"].view(F8), "sK": s["sK"], "V": s["V"].view(F8), "sV": s["sV"]}
    mx.mxgemm_cache_attention(_handle(mx, False), cache, s["table"], s["kv_len"], s["Q"], s["O"], q_start=starts, causal=True,
                              window=c["window"], sinks=c["sinks"], lse=s["lse"], stream=stream)
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a, b = _value(s["A"]), _value(s["B"])
        if case["b_rows_k"]:
            b, sb = b.t(), s["sB"].t().double()
        else:
            sb = s["sB"].double()
        row = torch.arange(n, device=DEV) // case["b_block"]
        out = torch.zeros(m, n, device=DEV, dtype=torch.float64)
        for j in range(-(-k // 1024)):  # eight blocks at a time
            at = torch.arange(1024 * j, min(k, 1024 * j + 1024), device=DEV)
            out += (a[:, at] * s["sA"].double()[:, at // 128]) @ (b[:, at] * sb[row][:, at // 128]).t()
        return out
    if case["op"] == "quantize":
        x, (r, c) = s["X"].double(), s["X"].shape
        i, j = torch.arange(r, device=DEV), torch.arange(c, device=DEV)
        bi, bj = (i if case["block"] == "rows" else i // 128), (j if case["block"] == "cols" else j // 128)
        top = torch.zeros(int(bi[-1]) + 1, c, device=DEV, dtype=torch.float64).index_reduce_(0, bi, x.abs(), "amax")
        top = torch.zeros(top.shape[0], int(bj[-1]) + 1, device=DEV, dtype=torch.float64).index_reduce_(1, bj, top, "amax").clamp(min=LEAST)
        codes = _e4m3(x * TOP / top[bi][:, bj])
        if case["block"] != "cols":
            return {"codes": codes, "scales": top / TOP}
        wide = torch.zeros(c, -(-r // 16) * 16, device=DEV, dtype=torch.float64)
        wide[:, :r] = codes.t()
        return {"codes": wide, "scales": (top / TOP).t().contiguous()}
    total, new = _lengths(case)
    page, kv, d = case["page"], case["kv"], case["d"]
    table, start = s["table"].long(), s["q_start"].tolist()
    if case["op"] == "append":
        out = {}
        for name in ("K", "V"):
            value, scale, x = _value(s[name]), s["s" + name].double(), s["new" + name].double()
            for b, (t, n) in enumerate(zip(total, new)):
                for p in range((t - n) // page, -(-t // page)):
                    lo, hi, at = max(p * page, t - n), min((p + 1) * page, t), table[b, p]
                    y = x[start[b] + lo - (t - n):start[b] + hi - (t - n)]
                    need = y.abs().amax((0, 2)) / TOP
                    z = torch.exp2(torch.floor(torch.log2(need.clamp(min=1e-300))) - 1)
                    z = torch.where(z < need, 2 * z, z)
                    z = torch.where(z < need, 2 * z, z).clamp(min=FLOOR)
                    if lo > p * page:
                        z = torch.maximum(z, scale[at])
                        value[at, :, :lo - p * page] = _e4m3(value[at, :, :lo - p * page] * (scale[at] / z)[:, None, None])
                    value[at, :, lo - p * page:hi - p * page] = _e4m3(y / z[None, :, None]).transpose(0, 1)
                    scale[at] = z
            out[name], out["s" + name] = value, scale
        return out
    h = case["heads"]
    g = h // kv
    o = torch.zeros(start[-1], h, d, device=DEV, dtype=torch.float64)
    lse = torch.full((start[-1], h), -math.inf, device=DEV, dtype=torch.float64)
    for b, (t, n) in enumerate(zip(total, new)):
        at = table[b, :-(-t // page)]
        far = torch.arange(t - n, t, device=DEV)[:, None] - torch.arange(t, device=DEV)[None]
        hidden = far < 0
        if case["window"]:
            hidden |= (far >= case["window"]) & (torch.arange(t, device=DEV)[None] >= case["sinks"])
        for i in range(kv):
            k, v = ((_value(s[x][at, i]) * s["s" + x][at, i].double()[:, None, None]).reshape(-1, d)[:t] for x in ("K", "V"))
            for j in range(i * g, i * g + g):
                w = (s["Q"][start[b]:start[b + 1], j].double() @ k.t() / math.sqrt(d)).masked_fill(hidden, -math.inf)
                lse[start[b]:start[b + 1], j] = torch.logsumexp(w, 1)
                o[start[b]:start[b + 1], j] = torch.softmax(w, 1) @ v
    return {"o": o, "lse": lse}
