"""Benchmark cases of the operators around the experts' products: routing from logits, RMS norm with the residual's
addition and an e4m3 output, and the products with microscaled 4-bit weights (one matrix, or one for each expert),
each with the quantisation of its activations.

``own`` False computes each operator in plain torch operations, True calls the framework.  Sizes are those of the
framework's workloads (d_model 2816 / 4096, expert width 704 / 1024, shared width 2112 / 4096, 128 / 256 experts
top-8, 1 to 4096 tokens) and ragged ones between them."""
import math

import torch

own = False

BLK = 128            # columns that share a scale of the e4m3 output
TINY = 2.0 ** -126
EPS = 1e-6           # of the norm
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token, softmax over all experts, the chosen ones' weights renormalised
        {"name": "route 1x128 softmax", "op": "route", "t": 1, "e": 128, "topk": 8, "score": "softmax", "bias": False,
         "groups": 1, "keep": 1, "best": 1, "renorm": True, "scale": 1.0, "dtype": "f32", "group_slots": False},
        # a short prompt of a model with few experts and logits in bf16 (many ties)
        {"name": "route 333x60 bf16", "op": "route", "t": 333, "e": 60, "topk": 4, "score": "softmax", "bias": False,
         "groups": 1, "keep": 1, "best": 1, "renorm": False, "scale": 1.0, "dtype": "bf16", "group_slots": True},
        # a prefill chunk: sigmoid scores, a bias for balance, the best 4 of 8 groups, slots grouped by expert
        {"name": "route 4096x256 groups", "op": "route", "t": 4096, "e": 256, "topk": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "best": 2, "renorm": True, "scale": 2.5, "dtype": "f32", "group_slots": True},
        # one decoded token before a block: residual added, e4m3 rows for the products, bf16 for the router
        {"name": "norm 1x2816", "op": "norm", "rows": 1, "cols": 2816, "dtype": "bf16", "residual": True, "out": True,
         "q": True, "pow2": False, "pitch": 0, "offset": 0.0},
        # fp32 activations of a short prompt, a slice of a wider buffer, no residual, power-of-two scales, a weight stored around 0
        {"name": "norm 700x2112 f32", "op": "norm", "rows": 700, "cols": 2112, "dtype": "f32", "residual": False, "out": False,
         "q": True, "pow2": True, "pitch": 704, "offset": 1.0},
        # a prefill chunk
        {"name": "norm 4096x4096", "op": "norm", "rows": 4096, "cols": 4096, "dtype": "bf16", "residual": True, "out": True,
         "q": True, "pow2": False, "pitch": 0, "offset": 0.0},
        # one token through the shared expert's up projection
        {"name": "linear 1x2112x2816 b16", "op": "linear", "m": 1, "n": 2112, "k": 2816, "block": 16, "dtype": "bf16", "out": "bf16"},
        # a batch of decoding sequences through a square projection
        {"name": "linear 64x4096x4096 b32", "op": "linear", "m": 64, "n": 4096, "k": 4096, "block": 32, "dtype": "bf16", "out": "bf16"},
        # an odd number of tokens, output columns and inner columns, fp32 in and out
        {"name": "linear 333x5001x1037 f32", "op": "linear", "m": 333, "n": 5001, "k": 1037, "block": 16, "dtype": "f32", "out": "f32"},
        # a prefill chunk
        {"name": "linear 4096^3 b16", "op": "linear", "m": 4096, "n": 4096, "k": 4096, "block": 16, "dtype": "bf16", "out": "bf16"},
        # 512 tokens top-8 over 128 experts with a skewed routing: gate projection
        {"name": "experts 4096 E128 b32", "op": "experts", "rows": 4096, "e": 128, "n": 704, "k": 2816, "skew": 1.0, "spare": 37,
         "block": 32, "dtype": "bf16", "out": "bf16"},
        # 4096 tokens top-8 over 256 experts: gate projection of the large prefill
        {"name": "experts 32768 E256 b16", "op": "experts", "rows": 32768, "e": 256, "n": 1024, "k": 4096, "skew": 0.0, "spare": 0,
         "block": 16, "dtype": "bf16", "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "norm", "linear", "experts"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "route":
        e = rng.choice([8, 16, 60, 64, 128, 160, 256])
        groups = rng.choice([1, 1, 4, 8]) if e % 8 == 0 and e >= 16 else 1
        keep = rng.randrange(max(1, groups // 4), groups + 1)
        return {"op": op, "t": _log_int(rng, 1, 4096), "e": e, "topk": min(rng.choice([1, 2, 6, 8]), e * keep // groups),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups, "keep": keep,
                "best": rng.choice([1, 2]), "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]), "dtype": dtype,
                "group_slots": rng.random() < 0.5}
    if op == "norm":
        q = rng.random() < 0.7
        return {"op": op, "rows": _log_int(rng, 1, 4096), "cols": _log_int(rng, 100, 4096), "dtype": dtype if q else "bf16",
                "residual": rng.random() < 0.5, "out": not q or rng.random() < 0.5, "q": q, "pow2": rng.random() < 0.5,
                "pitch": rng.choice([0, 0, 8, 129]), "offset": rng.choice([0.0, 1.0])}
    block, out = rng.choice([16, 32]), rng.choice(["bf16", "f32"])
    if op == "linear":
        return {"op": op, "m": _log_int(rng, 1, 4096), "n": _log_int(rng, 100, 4096), "k": _log_int(rng, 100, 4096),
                "block": block, "dtype": dtype, "out": out}
    return {"op": op, "rows": _log_int(rng, 8, 16384), "e": rng.choice([8, 16, 60, 128]), "n": _log_int(rng, 100, 1408),
            "k": 16 * _log_int(rng, 16, 256), "skew": rng.choice([0.0, 0.5, 1.0]), "spare": rng.choice([0, 1, 100]),
            "block": block, "dtype": dtype, "out": out}


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _nb(n, block=BLK):
    return -(-n // block)


# ----------------------------------------------------------------- inputs

def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + stream)
    return g


def _activations(rows, cols, dtype, seed, stream=1):
    """Normal activations with a few louder channels, as a decoder's residual stream has them."""
    g = _gen(seed, stream)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    loud = torch.rand(cols, device="cuda", generator=g) < 0.01
    return (x * torch.where(loud, 12.0, 1.0)).to(dtype)


def _pitched(rows, cols):
    """e4m3 rows that start at multiples of 16 bytes."""
    return torch.empty(rows, _nb(cols, 16) * 16, device="cuda", dtype=torch.float8_e4m3fn)[:, :cols]


def _codes(v):
    """Codes of the nearest e2m1 numbers, ties to the even code."""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c + 8 * (v < 0)


def _scales_like(n, rows, cols, block):
    """Uninitialised scale rows that start at multiples of 4 bytes."""
    kind = torch.float8_e4m3fn if block == 16 else torch.float8_e8m0fnu
    nb = _nb(cols, block)
    return torch.empty(n, rows, _nb(nb, 4) * 4, device="cuda", dtype=torch.uint8).view(kind)[..., :nb]


def _weight(n, rows, cols, block, seed):
    """n matrices [rows][cols] of e2m1 codes (rounded normal values), two to a byte, with a scale for each block and
    one for each matrix, such that the dequantised weights have a deviation of about 1 / sqrt(cols)."""
    g = _gen(seed, 3)
    v = torch.empty(n, rows, _nb(cols, 32) * 32, device="cuda", dtype=torch.float16).normal_(0.0, 2.0, generator=g)
    v[..., cols:] = 0
    c = _codes(v)
    w = (c[..., 0::2] + 16 * c[..., 1::2])[..., :_nb(cols, 2)]
    s = _scales_like(n, rows, cols, block)
    if block == 16:  # block scales over e4m3's upper range, the matrix's own factor beside them
        s.copy_(torch.rand(s.shape, device="cuda", generator=g) * 400 + 40)
        t = (0.5 + torch.rand(n, device="cuda", generator=g)) / (480.0 * math.sqrt(cols))
    else:
        e = 127 - int(math.log2(math.sqrt(cols)) + 1)
        s.view(torch.uint8).copy_(torch.randint(e - 1, e + 2, s.shape, device="cuda", generator=g, dtype=torch.uint8))
        t = None
    return w, s, t


def _popularity(e, skew, g):
    rank = torch.randperm(e, device="cuda", generator=g).float()
    return -skew * torch.log1p(rank)


def prepare(case, seed):
    op, c = case["op"], dict(case)
    st = {"case": c}
    if op == "route":
        t, e, k = c["t"], c["e"], c["topk"]
        g = _gen(seed, 2)
        st["logits"] = (1.5 * torch.randn(t, e, device="cuda", generator=g) + _popularity(e, 0.7, g)).to(_dt(c["dtype"]))
        st["bias"] = 0.1 * torch.randn(e, device="cuda", generator=g) if c["bias"] else None
        st["idx"] = torch.empty(t, k, device="cuda", dtype=torch.int32)
        st["w"] = torch.empty(t, k, device="cuda")
        if c["group_slots"]:
            st["counts"], st["offsets"], st["perm"] = (torch.empty(n, device="cuda", dtype=torch.int32) for n in (e, e + 1, t * k))
        if own:  # the router's description and the workspace that a program keeps
            import expert_ffn_gb300 as mx
            st["router"] = mx.Router(e, k, score=mx.MX_SOFTMAX if c["score"] == "softmax" else mx.MX_SIGMOID, bias=st["bias"],
                                     n_groups=c["groups"], topk_groups=c["keep"], group_best=c["best"],
                                     renormalise=c["renorm"], scale=c["scale"])
            n = mx.route_logits_workspace_bytes(st["router"], t)
            st["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
            mx.workspace_init(st["work"], n, stream=torch.cuda.current_stream())
        return st
    if op == "norm":
        rows, cols, dt = c["rows"], c["cols"], _dt(c["dtype"])
        st["x"] = _activations(rows, cols + c["pitch"], dt, seed)[:, :cols]
        g = _gen(seed, 4)
        st["weight"] = (1.0 - c["offset"] + 0.1 * torch.randn(cols, device="cuda", generator=g)).to(dt)
        st["residual"] = _activations(rows, cols, dt, seed, 5) if c["residual"] else None
        st["sum"] = torch.empty(rows, cols, device="cuda", dtype=dt) if c["residual"] else None
        st["out"] = torch.empty(rows, cols, device="cuda", dtype=dt) if c["out"] else None
        st["q"] = _pitched(rows, cols) if c["q"] else None
        st["scales"] = torch.empty(_nb(cols), rows, device="cuda").t() if c["q"] else None
        return st
    if op == "linear":
        rows, e, cap = c["m"], 1, c["m"]
        st["x"] = _activations(rows, c["k"], _dt(c["dtype"]), seed)
    else:
        rows, e = c["rows"], c["e"]
        g = _gen(seed, 2)
        p = torch.softmax(_popularity(e, c["skew"], g), 0)
        which = torch.multinomial(p, rows, replacement=True, generator=g)
        counts = torch.bincount(which, minlength=e)
        st["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        st["cap"] = int(counts.max())  # the router's host side knows the largest group
        rows += c["spare"]
        st["x"] = _activations(rows, c["k"], _dt(c["dtype"]), seed)
    st["w"], st["ws"], st["wt"] = _weight(e, c["n"], c["k"], c["block"], seed)
    # the activations' factor, calibrated to leave room above the largest value seen
    st["xt"] = torch.full((1,), 80.0 / (6.0 * 448.0), device="cuda") if c["block"] == 16 else None
    st["out"] = torch.zeros(rows, c["n"], device="cuda", dtype=_dt(c["out"]))
    if own:  # the weight handle, the buffers of quantised activations and the workspace that a program keeps
        import expert_ffn_gb300 as mx
        w = torch.empty(*st["w"].shape[:2], _nb(c["k"], 32) * 16, device="cuda", dtype=torch.uint8)[..., :_nb(c["k"], 2)]
        st["weight"] = mx.Fp4Weight(w.copy_(st["w"]), st["ws"], st["wt"], cols=c["k"])  # rows at multiples of 16 bytes
        st["q"], st["sx"] = mx.fp4_empty(rows, c["k"], c["block"], device="cuda")
        n = mx.fp4_matmul_workspace_bytes(st["weight"], rows)
        st["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        mx.workspace_init(st["work"], n, stream=torch.cuda.current_stream())
    return st


# ------------------------------------------------------------------- runs

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import expert_ffn_gb300 as mx
    c = st["case"]
    if c["op"] == "route":
        if not c["group_slots"]:
            mx.route_logits(st["logits"], st["router"], st["idx"], st["w"])
            return {"idx": st["idx"], "w": st["w"]}
        mx.route_logits(st["logits"], st["router"], st["idx"], st["w"], counts=st["counts"], offsets=st["offsets"],
                        perm=st["perm"], ws=st["work"])
        return {"idx": st["idx"], "w": st["w"], "counts": st["counts"], "offsets": st["offsets"], "perm": st["perm"]}
    if c["op"] == "norm":
        mx.fp8_rmsnorm(st["x"], st["weight"], eps=EPS, weight_offset=c["offset"], residual=st["residual"],
                       residual_out=st["sum"], out=st["out"], q=st["q"], scales=st["scales"], pow2=c["pow2"])
        return {n: st[n] for n in ("sum", "out", "q", "scales") if st[n] is not None}
    mx.fp4_quantize(st["x"], st["q"], st["sx"], tensor_scale=st["xt"])
    if c["op"] == "linear":
        mx.fp4_matmul(st["q"], st["sx"], st["weight"], st["out"], st["work"], tensor_scale=st["xt"])
    else:
        mx.fp4_grouped_matmul(st["q"], st["sx"], st["offsets"], st["weight"], st["out"], st["work"], tensor_scale=st["xt"])
    return st["out"]


def _plain_topk(c, k):
    """The k largest of each row in descending order, ties to the lower index."""
    return torch.sort(c, dim=-1, descending=True, stable=True)[1][..., :k]


def _plain_route(st):
    c = st["case"]
    t, e, k = c["t"], c["e"], c["topk"]
    l = st["logits"].float()

    def scores(x):
        if c["score"] == "sigmoid":
            return 1.0 / (1.0 + torch.exp(-x))
        z = torch.exp(x - x.amax(-1, keepdim=True))
        return z / z.sum(-1, keepdim=True)

    choice = scores(l.double())  # scores next to one another are told apart in 64 bits
    if c["bias"]:
        choice = choice + st["bias"].double()
    if c["groups"] > 1:
        by = choice.view(t, c["groups"], -1)
        score = by.amax(-1) if c["best"] == 1 else torch.sort(by, dim=-1)[0][..., -2:].sum(-1)
        kept = torch.zeros(t, c["groups"], dtype=torch.bool, device="cuda").scatter_(1, _plain_topk(score, c["keep"]), True)
        choice = torch.where(kept.unsqueeze(-1), by, -math.inf).view(t, e)
    idx = _plain_topk(choice, k)
    w = torch.gather(scores(l), 1, idx)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    out = {"idx": idx.to(torch.int32), "w": w * c["scale"]}
    if c["group_slots"]:
        flat = idx.flatten()
        counts = torch.zeros(e, dtype=torch.int32, device="cuda").index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
        out["counts"] = counts
        out["offsets"] = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).to(torch.int32)
        out["perm"] = torch.argsort(flat, stable=True).to(torch.int32)
    return out


def _plain_e4m3_rows(x, pow2):
    rows, cols = x.shape
    v = torch.nn.functional.pad(x, (0, _nb(cols) * BLK - cols)).view(rows, _nb(cols), BLK)
    a = v.abs().amax(-1)
    s = a / torch.full_like(a, 448.0)  # by a tensor: torch multiplies by the reciprocal of a number
    s = torch.where(s < TINY, TINY, s)
    if pow2:
        m, e = torch.frexp(s)  # s = m 2^e, m in [1/2, 1)
        s = torch.ldexp(torch.ones_like(s), torch.where(m > 0.5, e, e - 1))
    q = (v / s.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :cols], s


def _plain_norm(st):
    c, x, out = st["case"], st["x"], {}
    if c["residual"]:
        x = out["sum"] = (x.float() + st["residual"].float()).to(x.dtype)
    h = x.float()
    r = (1.0 / torch.sqrt((h.double() ** 2).mean(-1, keepdim=True) + EPS)).float()  # a long sum
    y = (h * r) * (c["offset"] + st["weight"].float())
    if c["out"]:
        out["out"] = y.to(x.dtype)
    if c["q"]:
        out["q"], out["scales"] = _plain_e4m3_rows(y, c["pow2"])
    return out


def _plain_fp4_rows(x, block, factor):
    """Activations rounded to e2m1 numbers times their scales, as fp32."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _nb(cols, block) * block - cols)).view(rows, -1, block)
    a = v.abs().amax(-1, keepdim=True)
    if block == 16:
        s = (a * (1.0 / (6.0 * factor))).to(torch.float8_e4m3fn).float() * factor
        v = torch.where(s >= TINY, v * (1.0 / s), 0.0)
    else:
        m, e = torch.frexp(a)  # 6 = 0.75 * 2^3
        e = torch.where(a > 0, torch.where(m > 0.75, e - 2, e - 3), -126).clamp(-126, 127)
        s = ((e + 127) << 23).view(torch.float32)
        v = v / s
    g = v.abs()
    step = torch.where(g < 2, 0.5, torch.where(g < 4, 1.0, 2.0))
    v = (torch.round(v / step) * step).clamp(-6.0, 6.0)
    return (v * s).view(rows, -1)[:, :cols]


def _plain_fp4_weights(w, s, factor, cols, block):
    """Block-scaled e2m1 matrices as fp32."""
    one = torch.tensor(FP4 + tuple(-v for v in FP4), device="cuda")
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)  # a byte's two values
    v = pair[w.int()].flatten(-2)
    if block == 16:
        f = s.float() * factor.view(-1, 1, 1)
    else:
        f = (s.view(torch.uint8).int() << 23).view(torch.float32)
    f = f.repeat_interleave(block, -1)
    return v[..., :cols] * f[..., :cols]


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


def _run_plain(st):
    c = st["case"]
    if c["op"] == "route":
        return _plain_route(st)
    if c["op"] == "norm":
        return _plain_norm(st)
    x = _plain_fp4_rows(st["x"], c["block"], st["xt"])
    w = _plain_fp4_weights(st["w"], st["ws"], st["wt"], c["k"], c["block"])
    if c["op"] == "linear":
        return torch.matmul(x, w[0].t()).to(_dt(c["out"]))
    n, e = c["rows"], c["e"]
    group = torch.searchsorted(st["offsets"][1:].long(), torch.arange(n, device="cuda"), right=True)
    slots = _plain_groups(group, e, st["cap"])
    y = torch.matmul(torch.nn.functional.pad(x[:n], (0, 0, 0, 1))[slots], w.transpose(1, 2))
    out = torch.zeros(n + 1, c["n"], device="cuda")
    out[slots.flatten()] = y.flatten(0, 1)
    return torch.cat([out[:n], st["out"][n:].float()]).to(_dt(c["out"]))


# -------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "route":
        t, e, k = c["t"], c["e"], c["topk"]
        slots = 4 * (t * k + 2 * e + 1) if c["group_slots"] else 0
        return {"bytes": t * e * size[c["dtype"]] + 8 * t * k + 4 * e * c["bias"] + slots, "flops": 4 * t * e}
    if op == "norm":
        r, k, b = c["rows"], c["cols"], size[c["dtype"]]
        per = b * (1 + 2 * c["residual"] + c["out"]) + c["q"]
        return {"bytes": r * k * per + b * k + 4 * r * _nb(k) * c["q"], "flops": 5 * r * k}
    n, k, b = c["n"], c["k"], c["block"]
    row = k / 2 + _nb(k, b)  # bytes of a row of weights
    if op == "linear":
        m = c["m"]
        return {"bytes": n * row + m * k * size[c["dtype"]] + m * n * size[c["out"]], "flops": 2 * m * n * k}
    r = c["rows"]
    touched = c["e"] * (1 - (1 - 1 / c["e"]) ** r)  # experts that have a row, spread evenly
    return {"bytes": touched * n * row + r * k * size[c["dtype"]] + r * n * size[c["out"]], "flops": 2 * r * n * k}


# ------------------------------------------------------- definition in fp64

def _exact_grid(v, lowest, bits, top):
    """fp64 values to the nearest number with `bits` bits behind the leading one and exponents from `lowest`, ties to
    even, at most `top`."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** lowest))) - bits)
    return (torch.round(v / step) * step).clamp(-top, top)


def _exact_fp4_rows(x, block, factor):
    """Values of quantised rows.  The operator defines the block scale, its reciprocal and the value that is rounded to
    e2m1 as fp32 numbers."""
    out = torch.empty_like(x)
    f = lambda v: v.float().double()  # noqa: E731
    for lo in range(0, x.shape[1], block):
        b = x[:, lo:lo + block]
        a = b.abs().max(1, keepdim=True).values
        if block == 16:
            g = factor.double()
            s = f(_exact_grid(f(a * f(1.0 / f(6.0 * g))), -6, 3, 448.0) * g)
            v = torch.where(s >= TINY, f(b * f(1.0 / s.clamp_min(TINY))), torch.zeros_like(b))
        else:
            s = torch.exp2(torch.round(torch.log2(a.clamp_min(6 * 2.0 ** -126) / 6.0)))  # the next power of two, or half of the one above
            s = torch.where(6.0 * s >= a, s, 2 * s)
            v = b / s
        out[:, lo:lo + block] = _exact_grid(v, 0, 1, 6.0) * s
    return out


def _exact_fp4_weight(w, s, factor, cols, block):
    v = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device="cuda")
    for half in (0, 1):
        code = (w >> (4 * half)) & 15
        m, e, sign = (code & 1).double(), ((code >> 1) & 3).double(), 1.0 - 2.0 * (code >> 3).double()
        v[:, half::2] = sign * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    v = v[:, :cols].contiguous()
    for b in range(s.shape[1]):
        f = s[:, b].double() * factor.double() if block == 16 else torch.exp2(s[:, b].view(torch.uint8).double() - 127)
        v[:, b * block:(b + 1) * block] *= f[:, None]
    return v


def _exact_route(st):
    c = st["case"]
    l = st["logits"].double()
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, -1)
    choice = s + st["bias"].double() if c["bias"] else s.clone()
    idx = torch.empty(c["t"], c["topk"], dtype=torch.long, device="cuda")
    lower = torch.arange(c["e"], device="cuda")

    def first_largest(v):
        top = v.max(1, keepdim=True).values
        return torch.where(v == top, lower[:v.shape[1]], v.shape[1]).min(1).values

    if c["groups"] > 1:
        by = choice.view(c["t"], c["groups"], -1)
        score = by.max(-1).values if c["best"] == 1 else by.topk(2, dim=-1).values.sum(-1)
        closed = torch.ones_like(score, dtype=torch.bool)
        for _ in range(c["keep"]):
            g = first_largest(score)[:, None]
            closed.scatter_(1, g, False)
            score = score.scatter(1, g, -math.inf)
        choice = by.masked_fill(closed[..., None], -math.inf).reshape(c["t"], -1)
    for k in range(c["topk"]):
        idx[:, k] = first_largest(choice)
        choice = choice.scatter(1, idx[:, k:k + 1], -math.inf)
    w = s.gather(1, idx)
    out = {"idx": idx.int(), "w": c["scale"] * (w / w.sum(1, keepdim=True) if c["renorm"] else w)}
    if c["group_slots"]:
        flat = idx.flatten()
        out["counts"] = torch.bincount(flat, minlength=c["e"]).int()
        out["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), out["counts"].cumsum(0).int()])
        out["perm"] = torch.argsort(flat * flat.numel() + torch.arange(flat.numel(), device="cuda")).int()
    return out


def _exact_norm(st):
    """The operator defines the sum with the residual as a number of its type, the reciprocal root, both products and
    the quotient that is rounded to e4m3 as fp32 numbers."""
    c, out = st["case"], {}
    h = st["x"].double()
    if c["residual"]:
        h = h + st["residual"].double()
        out["sum"] = h.float().to(st["x"].dtype)
        h = out["sum"].double()
    r = (1.0 / torch.sqrt(h.pow(2).sum(1, keepdim=True) / c["cols"] + EPS)).float().double()
    y = ((h * r).float().double() * (c["offset"] + st["weight"].double()).float().double()).float().double()
    if c["out"]:
        out["out"] = y
    if c["q"]:
        q, ss = torch.empty_like(y), []
        for lo in range(0, c["cols"], BLK):
            b = y[:, lo:lo + BLK]
            s = (b.abs().max(1, keepdim=True).values / 448.0).clamp_min(TINY).float().double()
            if c["pow2"]:
                up = torch.exp2(torch.round(torch.log2(s)))
                s = torch.where(up >= s, up, 2 * up)
            q[:, lo:lo + BLK] = _exact_grid((b / s).float().double(), -6, 3, 448.0)
            ss.append(s)
        out["q"], out["scales"] = q, torch.cat(ss, 1)
    return out


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "route":
        return _exact_route(st)
    if c["op"] == "norm":
        return _exact_norm(st)
    x = _exact_fp4_rows(st["x"].double(), c["block"], st["xt"])
    factor = st["wt"] if c["block"] == 16 else [None] * st["w"].shape[0]
    if c["op"] == "linear":
        return x @ _exact_fp4_weight(st["w"][0], st["ws"][0], factor[0], c["k"], c["block"]).T
    out = st["out"].double()
    at = st["offsets"].tolist()
    for e in range(c["e"]):
        r = slice(at[e], at[e + 1])
        out[r] = x[r] @ _exact_fp4_weight(st["w"][e], st["ws"][e], factor[e], c["k"], c["block"]).T
    return out
