"""Benchmark cases of the FP8 block-scaled operators: quantisation of activations, the matrix product, the
product grouped by expert, and the whole routed-MoE layer after its routing.

``own`` False computes each operator in plain torch operations (fp32), True calls the framework.  Sizes are
those of the framework's workloads (d_model 2816 / 4096, expert width 704 / 1024, shared width 2112 / 4096,
128 / 256 experts top-8, 1 to 4096 tokens) and ragged ones between them."""
import math

import torch

own = False

BLK = 128        # columns (and weight rows) that share a scale
TINY = 2.0 ** -126
LAYER = 0.5      # layer scalar of every workload


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token's activations before a projection: all launch latency
        {"name": "quantize 1x2816", "op": "quantize", "rows": 1, "cols": 2816, "dtype": "bf16", "pow2": False, "pitch": 0},
        # fp32 activations of a short prompt, a slice of a wider buffer, power-of-two scales, a ragged last block
        {"name": "quantize 700x2112 f32", "op": "quantize", "rows": 700, "cols": 2112, "dtype": "f32", "pow2": True, "pitch": 704},
        # a prefill chunk
        {"name": "quantize 4096x4096", "op": "quantize", "rows": 4096, "cols": 4096, "dtype": "bf16", "pow2": False, "pitch": 0},
        # one token through the shared expert's up projection
        {"name": "matmul 1x2112x2816", "op": "matmul", "m": 1, "n": 2112, "k": 2816, "out": "bf16"},
        # a batch of decoding sequences through a square projection
        {"name": "matmul 64x4096x4096", "op": "matmul", "m": 64, "n": 4096, "k": 4096, "out": "bf16"},
        # an odd number of tokens, output columns and inner columns (a last block of 13), fp32 results (a head's logits)
        {"name": "matmul 333x5001x1037 f32", "op": "matmul", "m": 333, "n": 5001, "k": 1037, "out": "f32"},
        # a prefill chunk
        {"name": "matmul 4096x4096x4096", "op": "matmul", "m": 4096, "n": 4096, "k": 4096, "out": "bf16"},
        # 512 tokens top-8 over 128 experts with a skewed routing: gate projection
        {"name": "grouped 4096 E128", "op": "grouped", "rows": 4096, "e": 128, "n": 704, "k": 2816, "skew": 1.0, "spare": 37, "out": "bf16"},
        # 4096 tokens top-8 over 256 experts: gate projection of the large prefill
        {"name": "grouped 32768 E256", "op": "grouped", "rows": 32768, "e": 256, "n": 1024, "k": 4096, "skew": 0.0, "spare": 0, "out": "bf16"},
        # single-token decode
        {"name": "moe T1 E128", "op": "moe", "t": 1, "e": 128, "topk": 8, "d": 2816, "i": 704, "s": 2112, "skew": 0.0, "act": "gelu", "residual": True},
        # a decoding batch whose routing favours a few experts
        {"name": "moe T31 E128", "op": "moe", "t": 31, "e": 128, "topk": 8, "d": 2816, "i": 704, "s": 2112, "skew": 1.0, "act": "silu", "residual": False},
        # the large prefill
        {"name": "moe T4096 E256", "op": "moe", "t": 4096, "e": 256, "topk": 8, "d": 4096, "i": 1024, "s": 4096, "skew": 0.0, "act": "gelu", "residual": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "grouped", "moe"])
    out = rng.choice(["bf16", "f32"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 4096), "cols": _log_int(rng, 100, 4096),
                "dtype": out, "pow2": rng.random() < 0.5, "pitch": rng.choice([0, 0, 8, 129])}
    if op == "matmul":
        return {"op": op, "m": _log_int(rng, 1, 4096), "n": _log_int(rng, 100, 4096),
                "k": _log_int(rng, 100, 4096), "out": out}
    if op == "grouped":
        return {"op": op, "rows": _log_int(rng, 8, 16384), "e": rng.choice([8, 16, 60, 128]), "n": _log_int(rng, 100, 1408),
                "k": 16 * _log_int(rng, 16, 256), "skew": rng.choice([0.0, 0.5, 1.0]), "spare": rng.choice([0, 1, 100]), "out": out}
    e = rng.choice([16, 60, 128])
    return {"op": op, "t": _log_int(rng, 1, 1024), "e": e, "topk": rng.choice([1, 2, 6, 8]), "d": 16 * _log_int(rng, 16, 256),
            "i": 16 * rng.randrange(8, 65), "s": 16 * rng.choice([0, 16, 77, 132]), "skew": rng.choice([0.0, 1.0]),
            "act": rng.choice(["gelu", "silu"]), "residual": rng.random() < 0.5}


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _nb(n):
    return -(-n // BLK)


# ----------------------------------------------------------------- inputs

def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + stream)
    return g


def _activations(rows, cols, dtype, seed):
    """Normal activations with a few louder channels, as a decoder's residual stream has them."""
    g = _gen(seed, 1)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    loud = torch.rand(cols, device="cuda", generator=g) < 0.01
    return (x * torch.where(loud, 12.0, 1.0)).to(dtype)


def _pitched(*shape):
    """e4m3 rows that start at multiples of 16 bytes."""
    wide = torch.empty(*shape[:-1], -(-shape[-1] // 16) * 16, device="cuda", dtype=torch.float8_e4m3fn)
    return wide[..., :shape[-1]]


def _weight(n, rows, cols, seed, stream):
    """n matrices [rows][cols] of e4m3 codes (normal values over a block's range) and their block scales, such
    that the dequantised weights have a deviation of about 1/sqrt(cols)."""
    g = _gen(seed, stream)
    q = _pitched(n, rows, cols)
    v = torch.empty(n, rows, cols, device="cuda", dtype=torch.float16).normal_(0.0, 110.0, generator=g)
    q.copy_(v.clamp_(-448.0, 448.0))
    s = (0.5 + torch.rand(n, _nb(rows), _nb(cols), device="cuda", generator=g)) / (110.0 * math.sqrt(cols))
    return q, s


def _quantized_rows(rows, cols, seed):
    """Activations as the quantiser leaves them: e4m3 rows and their scales (made here without it)."""
    x = _activations(rows, cols, torch.float32, seed)
    x = torch.nn.functional.pad(x, (0, _nb(cols) * BLK - cols)).view(rows, _nb(cols), BLK)
    s = x.abs().amax(-1).div(448.0).clamp_min(TINY)
    q = _pitched(rows, cols)
    q.copy_((x / s.unsqueeze(-1)).view(rows, -1)[:, :cols])
    return q, s.t().contiguous().t()


def _popularity(e, skew, g):
    rank = torch.randperm(e, device="cuda", generator=g).float()
    return -skew * torch.log1p(rank)


def _routing(t, e, k, skew, seed):
    g = _gen(seed, 2)
    logits = torch.randn(t, e, device="cuda", generator=g) + 1.5 * _popularity(e, skew, g)
    top, idx = logits.topk(k, dim=-1)
    return idx.to(torch.int32), torch.softmax(top, -1).contiguous()


def prepare(case, seed):
    op, c = case["op"], dict(case)
    st = {"case": c}
    if op == "quantize":
        rows, cols = c["rows"], c["cols"]
        wide = _activations(rows, cols + c["pitch"], _dt(c["dtype"]), seed)
        st["x"] = wide[:, :cols]
        st["q"] = _pitched(rows, cols)
        st["scales"] = torch.empty(_nb(cols), rows, device="cuda").t()  # block by block, as the products read them
    elif op == "matmul":
        st["q"], st["scales"] = _quantized_rows(c["m"], c["k"], seed)
        st["w"], st["ws"] = (a[0] for a in _weight(1, c["n"], c["k"], seed, 3))
        st["out"] = torch.empty(c["m"], c["n"], device="cuda", dtype=_dt(c["out"]))
    elif op == "grouped":
        rows, e = c["rows"], c["e"]
        g = _gen(seed, 2)
        p = torch.softmax(_popularity(e, c["skew"], g), 0)
        which = torch.multinomial(p, rows, replacement=True, generator=g)
        counts = torch.bincount(which, minlength=e)
        st["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        st["cap"] = int(counts.max())  # the router's host side knows the largest group
        st["q"], st["scales"] = _quantized_rows(rows + c["spare"], c["k"], seed)
        st["w"], st["ws"] = _weight(e, c["n"], c["k"], seed, 3)
        st["out"] = torch.zeros(rows + c["spare"], c["n"], device="cuda", dtype=_dt(c["out"]))
    else:
        t, e, d, i, s = c["t"], c["e"], c["d"], c["i"], c["s"]
        st["x"] = _activations(t, d, torch.bfloat16, seed)
        st["idx"], st["wts"] = _routing(t, e, c["topk"], c["skew"], seed)
        st["cap"] = int(torch.bincount(st["idx"].flatten().long(), minlength=e).max())
        st["gate"], st["up"], st["down"] = (_weight(e, r, k, seed, 3 + j) for j, (r, k) in enumerate(((i, d), (i, d), (d, i))))
        if s:
            st["shared"] = [_weight(1, r, k, seed, 6 + j) for j, (r, k) in enumerate(((s, d), (s, d), (d, s)))]
        st["residual"] = _activations(t, d, torch.bfloat16, seed + 77) if c["residual"] else None
        st["out"] = torch.empty(t, d, device="cuda", dtype=torch.bfloat16)
    if own and op != "quantize":  # the weight handle and the workspace that a program keeps beside its weights
        import expert_ffn_gb300 as mx
        if op == "moe":
            st["layer"] = mx.Fp8Layer(st["gate"], st["up"], st["down"], shared=st.get("shared"), top_k=c["topk"],
                                      activation=mx.MX_GELU_TANH if c["act"] == "gelu" else mx.MX_SILU, layer_scalar=LAYER)
            n = mx.fp8_moe_workspace_bytes(st["layer"], c["t"])
        else:
            st["weight"] = mx.Fp8Weight(st["w"], st["ws"])
            n = mx.fp8_matmul_workspace_bytes(st["weight"], st["q"].shape[0])
        st["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        mx.workspace_init(st["work"], n, stream=torch.cuda.current_stream())
    return st


# ------------------------------------------------------------------- runs

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import expert_ffn_gb300 as mx
    c = st["case"]
    if c["op"] == "quantize":
        mx.fp8_quantize(st["x"], st["q"], st["scales"], pow2=c["pow2"])
        return {"q": st["q"], "scales": st["scales"]}
    if c["op"] == "matmul":
        mx.fp8_matmul(st["q"], st["scales"], st["weight"], st["out"], st["work"])
    elif c["op"] == "grouped":
        mx.fp8_grouped_matmul(st["q"], st["scales"], st["offsets"], st["weight"], st["out"], st["work"])
    else:
        mx.fp8_moe_forward(st["x"], st["idx"], st["wts"], st["layer"], st["out"], st["work"], residual=st["residual"])
    return st["out"]


def _plain_quantize(x, pow2=False):
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _nb(cols) * BLK - cols)).view(rows, _nb(cols), BLK)
    a = v.abs().amax(-1)
    s = a / torch.full_like(a, 448.0)  # by a tensor: torch multiplies by the reciprocal of a number
    s = torch.where(s < TINY, TINY, s)
    if pow2:
        m, e = torch.frexp(s)  # s = m 2^e, m in [1/2, 1)
        s = torch.ldexp(torch.ones_like(s), torch.where(m > 0.5, e, e - 1))
    q = (v / s.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :cols], s


def _plain_values(q, s):
    """Row-quantised values as fp32."""
    return q.float() * s.repeat_interleave(BLK, 1)[:, :q.shape[1]]


def _plain_weights(w, s):
    """Block-scaled matrices as fp32."""
    r, k = w.shape[-2:]
    return w.float() * s.repeat_interleave(BLK, -2)[..., :r, :].repeat_interleave(BLK, -1)[..., :k]


def _plain_groups(group, n_groups, cap):
    """Positions of the items of each group in item order, [n_groups][cap], and n items where a group has fewer."""
    n = group.numel()
    order = torch.argsort(group, stable=True)
    counts = torch.zeros(n_groups + 1, device="cuda", dtype=torch.long).index_add_(0, group, torch.ones_like(group))
    start = torch.cumsum(counts, 0) - counts
    at = torch.arange(n, device="cuda") - start[group[order]]
    slots = torch.full((n_groups + 1, cap), n, device="cuda", dtype=torch.long)
    slots[group[order], at] = order
    return slots[:n_groups]


def _plain_ffn(x, gate, up, down, act):
    g, u = (torch.matmul(x, _plain_weights(*w).transpose(-1, -2)) for w in (gate, up))
    h = (g * torch.sigmoid(g) if act == "silu" else 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))) * u
    shape = h.shape
    h = _plain_values(*_plain_quantize(h.reshape(-1, shape[-1]))).view(shape)
    return torch.matmul(h, _plain_weights(*down).transpose(-1, -2))


def _run_plain(st):
    c = st["case"]
    if c["op"] == "quantize":
        q, s = _plain_quantize(st["x"], c["pow2"])
        return {"q": q, "scales": s}
    if c["op"] == "matmul":
        return torch.matmul(_plain_values(st["q"], st["scales"]), _plain_weights(st["w"], st["ws"]).t()).to(_dt(c["out"]))
    if c["op"] == "grouped":
        n, e = c["rows"], c["e"]
        group = torch.searchsorted(st["offsets"][1:].long(), torch.arange(n, device="cuda"), right=True)
        slots = _plain_groups(group, e, st["cap"])
        x = torch.nn.functional.pad(_plain_values(st["q"], st["scales"])[:n], (0, 0, 0, 1))
        y = torch.matmul(x[slots], _plain_weights(st["w"], st["ws"]).transpose(1, 2))
        out = torch.zeros(n + 1, c["n"], device="cuda")
        out[slots.flatten()] = y.flatten(0, 1)
        return torch.cat([out[:n], st["out"][n:].float()]).to(_dt(c["out"]))
    t, e, k = c["t"], c["e"], c["topk"]
    x = _plain_values(*_plain_quantize(st["x"]))
    flat = st["idx"].flatten().long()
    if t * k < e:  # each slot beside its own expert's matrices
        xg = x.repeat_interleave(k, 0).unsqueeze(1)
        y = _plain_ffn(xg, *((w[0][flat], w[1][flat]) for w in (st["gate"], st["up"], st["down"])), c["act"]).view(t, k, -1)
    else:
        slots = _plain_groups(flat, e, st["cap"])
        xg = torch.nn.functional.pad(x, (0, 0, 0, 1))[torch.div(slots, k, rounding_mode="floor")]
        y = torch.zeros(t * k + 1, c["d"], device="cuda")
        y[slots.flatten()] = _plain_ffn(xg, st["gate"], st["up"], st["down"], c["act"]).flatten(0, 1)
        y = y[:t * k].view(t, k, -1)
    y = (y * st["wts"].unsqueeze(-1)).sum(1)
    if c["s"]:
        y = y + _plain_ffn(x, *((w[0][0], w[1][0]) for w in st["shared"]), c["act"])
    y = LAYER * y
    return (y if st["residual"] is None else st["residual"].float() + y).to(torch.bfloat16)


# -------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "quantize":
        r, k = c["rows"], c["cols"]
        return {"bytes": r * k * (size[c["dtype"]] + 1) + 4 * r * _nb(k), "flops": 2 * r * k}
    if op == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": n * k + m * k + m * n * size[c["out"]] + 4 * (m + _nb(n)) * _nb(k), "flops": 2 * m * n * k}
    if op == "grouped":
        r, n, k = c["rows"], c["n"], c["k"]
        touched = c["e"] * (1 - (1 - 1 / c["e"]) ** r)
        return {"bytes": touched * n * k + r * k + r * n * size[c["out"]] + 4 * r * _nb(k), "flops": 2 * r * n * k}
    t, d, i, s = c["t"], c["d"], c["i"], c["s"]
    touched = c["e"] * (1 - (1 - c["topk"] / c["e"]) ** t)  # experts that some token chose, routing spread evenly
    acts = 6 if c["residual"] else 4  # bytes of x, out and the residual per element
    return {"bytes": 3 * d * (touched * i + s) + acts * t * d + 8 * t * c["topk"],
            "flops": 6 * t * d * (c["topk"] * i + s)}


# ------------------------------------------------------- definition in fp64

def _exact_e4m3(v):
    """fp64 values, |v| about 448 at most, to the nearest e4m3 number (3 mantissa bits, exponents from -6), ties
    to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_blocks(x, pow2=False):
    """(e4m3 values, scales) of fp64 rows, block by block.  The operator defines the scale and the quotient that
    is rounded to e4m3 as fp32 numbers: bf16 activations often lie exactly between two e4m3 numbers."""
    q, scales = torch.empty_like(x), []
    for lo in range(0, x.shape[1], BLK):
        b = x[:, lo:lo + BLK]
        s = (b.abs().max(1, keepdim=True).values / 448.0).clamp_min(TINY).float().double()
        if pow2:
            up = torch.exp2(torch.round(torch.log2(s)))  # the power of two next to s, or half of the one above
            s = torch.where(up >= s, up, 2 * up)
        q[:, lo:lo + BLK] = _exact_e4m3((b / s).float().double())
        scales.append(s)
    return q, torch.cat(scales, 1)


def _exact_scaled(q, s, br):
    """q * s in fp64 for blocks of br rows by 128 columns."""
    v = q.double()
    for b in range(s.shape[1]):
        col = s[:, b].double().repeat_interleave(br)[:v.shape[0]]
        v[:, b * BLK:(b + 1) * BLK] *= col[:, None]
    return v


def _exact_expert(x, gate, up, down, act):
    g, u = (x @ _exact_scaled(*w, BLK).T for w in (gate, up))
    if act == "silu":
        h = g / (1 + torch.exp(-g)) * u
    else:
        h = g / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) * u
    return _exact_scaled(*_exact_blocks(h), 1) @ _exact_scaled(*down, BLK).T


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "quantize":
        q, s = _exact_blocks(st["x"].double(), c["pow2"])
        return {"q": q, "scales": s}
    if c["op"] == "matmul":
        return _exact_scaled(st["q"], st["scales"], 1) @ _exact_scaled(st["w"], st["ws"], BLK).T
    if c["op"] == "grouped":
        out = st["out"].double()
        at = st["offsets"].tolist()
        for e in range(c["e"]):
            r = slice(at[e], at[e + 1])
            out[r] = _exact_scaled(st["q"][r], st["scales"][r], 1) @ _exact_scaled(st["w"][e], st["ws"][e], BLK).T
        return out
    x = _exact_scaled(*_exact_blocks(st["x"].double()), 1)
    y = torch.zeros_like(x)
    for e in range(c["e"]):
        t, k = torch.nonzero(st["idx"] == e, as_tuple=True)
        if len(t):
            part = _exact_expert(x[t], *((w[0][e], w[1][e]) for w in (st["gate"], st["up"], st["down"])), c["act"])
            y.index_add_(0, t, part * st["wts"][t, k].double()[:, None])
    if c["s"]:
        y += _exact_expert(x, *((w[0][0], w[1][0]) for w in st["shared"]), c["act"])
    y *= LAYER
    return y if st["residual"] is None else y + st["residual"].double()
