"""Work of the microscaled (MX) activation operators of libk3g, and their plain forms.

A microscaled row holds 32-entry groups of e2m1 (MXFP4) or e4m3 (MXFP8) codes with one ue8m0 scale byte each;
weights are MXFP4 as the library stores them (low nibble = even column; scale byte 255 = the group contributes
nothing). Sizes are the library's own layer: hidden 7168, latent 3584, expert intermediate 3072, shared
intermediate 6144, 896 routed experts, 16 per token.
"""
import math

import torch

own = False

HIDDEN, LATENT, INTER, SHARED, EXPERTS, TOP_K = 7168, 3584, 3072, 6144, 896, 16
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


# ---- the cases ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token's hidden state written as MXFP4 ahead of a product: the smallest call
        {"name": "quantize_token", "op": "quantize", "T": 1, "n": HIDDEN, "type": "bf16", "fmt": "fp4", "pad": 0},
        # a prefill chunk of fp32 latents to MXFP8, the rows a slice of a wider buffer
        {"name": "quantize_chunk", "op": "quantize", "T": 8191, "n": LATENT, "type": "f32", "fmt": "fp8", "pad": 96},
        # the pre-norm of a decode batch: residual added, MXFP8 out
        {"name": "norm_batch", "op": "norm", "T": 64, "n": HIDDEN, "type": "bf16", "fmt": "fp8", "pad": 0},
        # the pre-norm of a prefill chunk
        {"name": "norm_chunk", "op": "norm", "T": 8192, "n": HIDDEN, "type": "bf16", "fmt": "fp8", "pad": 0},
        # one token through the latent down-projection's shape
        {"name": "matmul_token", "op": "matmul", "T": 1, "n": HIDDEN, "rows": LATENT, "fmt": "fp8", "out": "f32"},
        # a ragged decode batch through the latent up-projection's shape
        {"name": "matmul_batch", "op": "matmul", "T": 61, "n": LATENT, "rows": HIDDEN, "fmt": "fp4", "out": "f32"},
        # a prefill chunk through a shared expert's up-projection
        {"name": "matmul_chunk", "op": "matmul", "T": 4096, "n": HIDDEN, "rows": SHARED, "fmt": "fp4", "out": "bf16"},
        # pre-norm and down-projection of a small chunk, one after the other as a block runs them
        {"name": "norm_matmul", "op": "norm_matmul", "T": 256, "n": HIDDEN, "rows": LATENT, "type": "bf16", "fmt": "fp4",
         "out": "bf16"},
        # the experts' down products of 64 decode tokens: about one row an expert, every weight read once
        {"name": "grouped_decode", "op": "grouped", "T": 64, "E": EXPERTS, "k": TOP_K, "n": INTER, "rows": LATENT, "fmt": "fp8",
         "out": "f32"},
        # the same of a prefill chunk: ragged groups of about 73 rows
        {"name": "grouped_chunk", "op": "grouped", "T": 4096, "E": EXPERTS, "k": TOP_K, "n": INTER, "rows": LATENT, "fmt": "fp4",
         "out": "bf16"},
        # one token's 16 experts up to the quantised h
        {"name": "glu_token", "op": "glu", "T": 1, "E": EXPERTS, "k": TOP_K, "n": LATENT, "inter": INTER, "fmt": "fp8"},
        # a prefill chunk through all of its experts: gated up-products, h in MXFP4, down-products
        {"name": "experts_chunk", "op": "experts", "T": 4096, "E": EXPERTS, "k": TOP_K, "n": LATENT, "inter": INTER, "fmt": "fp4",
         "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "matmul", "norm_matmul", "grouped", "glu", "experts"])
    fmt = rng.choice(["fp4", "fp8"])
    width = lambda hi: 32 * _log(rng, 2, hi // 32)  # noqa: E731  (whole groups, odd numbers of them among them)
    if op in ("quantize", "norm"):
        return {"op": op, "T": _log(rng, 1, 8192), "n": width(HIDDEN), "type": rng.choice(list(TYPES)),
                "fmt": fmt if op == "quantize" else "fp8", "pad": rng.choice([0, 0, 32, 160])}
    if op in ("matmul", "norm_matmul"):
        c = {"op": op, "T": _log(rng, 1, 4096), "n": 32 * _log(rng, 8, HIDDEN // 32), "rows": _log(rng, 33, SHARED), "fmt": fmt}
        if op == "matmul":
            return c | {"out": rng.choice(["f32", "bf16"])}
        return c | {"type": rng.choice(list(TYPES)), "out": "bf16"}
    E = _log(rng, 8, EXPERTS)
    c = {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(E, TOP_K)), "n": 32 * _log(rng, 8, LATENT // 32),
         "fmt": fmt}
    if op == "grouped":
        return c | {"rows": width(LATENT), "out": rng.choice(["f32", "bf16"])}
    c["inter"] = 32 * _log(rng, 8, INTER // 32)
    return c | ({"fmt": "fp8"} if op == "glu" else {"out": "bf16"})


def work(c):
    T, n, op = c["T"], c["n"], c["op"]
    code = {"fp4": 0.5, "fp8": 1.0}[c["fmt"]] + 1 / 32
    size = {"f32": 4, "bf16": 2, "f16": 2}
    w = 0.5 + 1 / 32
    if op == "quantize":  # there (codes written) and back (codes read, bf16 written)
        return {"bytes": T * n * (size[c["type"]] + 2 * code + 2), "flops": 4 * T * n}
    if op == "norm":
        return {"bytes": T * n * (3 * size[c["type"]] + 2 * code + 2) + 4 * n, "flops": 8 * T * n}
    if op == "matmul":
        return {"bytes": T * n * code + c["rows"] * n * w + T * c["rows"] * size[c["out"]], "flops": 2 * T * n * c["rows"]}
    if op == "norm_matmul":
        return {"bytes": T * n * (3 * size[c["type"]] + 2 * code) + c["rows"] * n * w + T * c["rows"] * 2,
                "flops": 2 * T * n * c["rows"] + 8 * T * n}
    P = T * c["k"]
    active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** T)  # the experts that a flat routing of T tokens meets
    if op == "grouped":
        return {"bytes": P * n * code + active * c["rows"] * n * w + P * c["rows"] * size[c["out"]],
                "flops": 2 * P * n * c["rows"]}
    up = {"bytes": T * n * code + active * 2 * c["inter"] * n * w + P * c["inter"] * code, "flops": 4 * P * n * c["inter"]}
    if op == "glu":  # and h back as values
        return {"bytes": up["bytes"] + P * c["inter"] * (code + 2), "flops": up["flops"]}
    return {"bytes": up["bytes"] + P * c["inter"] * code + active * n * c["inter"] * w + P * n * 2,
            "flops": up["flops"] + 2 * P * n * c["inter"]}


# ---- the inputs --------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, T, n, dtype, pad=0):
    """Rows of a residual stream: unit normals with a few large channels, in a buffer `pad` columns wider."""
    x = torch.randn(T, n + pad, device="cuda", generator=g)
    big = torch.rand(n + pad, device="cuda", generator=g) < 0.002
    return torch.where(big, 12 * x, x).to(dtype)[:, :n]


def _weight_bytes(g, *shape):
    """Packed nibbles uniform over the 16 codes; scale bytes 118..132, one in a thousand 255 (a skipped group)."""
    packed = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.randint(118, 133, (*shape[:-1], shape[-1] // 32), dtype=torch.uint8, device="cuda", generator=g)
    s[torch.rand(s.shape, device="cuda", generator=g) < 0.001] = 255
    return packed, s


def _layout(latent, inter):
    """An expert's six tensors (w1, w3, w2: packed, scales), back to back, each at a multiple of 256 bytes."""
    off, at = [], 0
    for rows, cols in ((inter, latent), (inter, latent), (latent, inter)):
        for b in (rows * cols // 2, rows * cols // 32):
            off.append(at)
            at = (at + b + 255) // 256 * 256
    return off, at


def _bank(g, E, latent, inter, tensors):
    """A bank of E experts [E][stride] with the named tensors drawn (the others are not read)."""
    off, stride = _layout(latent, inter)
    bank = torch.zeros(E, stride, dtype=torch.uint8, device="cuda")
    for t in tensors:
        rows, cols = ((inter, latent), (inter, latent), (latent, inter))[t]
        for e in range(0, E, 128):
            m = min(128, E - e)
            p, s = _weight_bytes(g, m, rows, cols)
            bank[e:e + m, off[2 * t]:off[2 * t] + rows * cols // 2] = p.view(m, -1)
            bank[e:e + m, off[2 * t + 1]:off[2 * t + 1] + rows * cols // 32] = s.view(m, -1)
    return bank


def _routing(g, T, E, k):
    """A near-flat routing: the pairs sorted by expert as the library's bucket has them (offsets [E + 1], and perm:
    sorted position -> pair id token * k + slot), the experts with pairs, and the longest group."""
    score = torch.rand(T, E, device="cuda", generator=g) + 0.1 * torch.randn(E, device="cuda", generator=g)
    idx = score.topk(k, dim=1).indices.reshape(-1)
    perm = torch.sort(idx, stable=True).indices
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, perm.to(torch.int32), counts.nonzero().flatten(), int(counts.max())


def _codes(q):
    """Codes and scale bytes of the grid values and exponents that _grid() gives."""
    v, x = q["v"], q["x"]
    scales = torch.where(x == 128, 255, x + 127).to(torch.uint8)
    if q["fmt"] == "fp8":
        return v.reshape(v.shape[0], -1).to(torch.float8_e4m3fn).view(torch.uint8), scales
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=v.device)
    c = torch.bucketize(v.abs().float(), mags) + 8 * torch.signbit(v)
    c = c.reshape(v.shape[0], -1, 2).to(torch.uint8)
    return c[..., 0] | (c[..., 1] << 4), scales


def prepare(case, seed):
    g, op, fmt = _gen(seed), case["op"], case["fmt"]
    s = {"case": dict(case)}
    T, n = case["T"], case["n"]
    if op in ("quantize", "norm", "norm_matmul"):
        s["x"] = _normal(g, T, n, TYPES[case["type"]], case.get("pad", 0))
    if op in ("norm", "norm_matmul"):
        s["r"] = _normal(g, T, n, TYPES[case["type"]])
        s["gamma"] = 0.5 + torch.rand(n, device="cuda", generator=g)
    if op in ("matmul", "norm_matmul"):
        s["w"] = _weight_bytes(g, case["rows"], n)
    if op in ("grouped", "glu", "experts"):
        s["offsets"], s["perm"], s["active"], s["most"] = _routing(g, T, case["E"], case["k"])
        if op == "grouped":  # a row for each sorted pair, down an expert's w2
            s["dims"] = (case["rows"], n)
            s["bank"] = _bank(g, case["E"], *s["dims"], (2,))
        else:
            s["dims"] = (n, case["inter"])
            s["bank"] = _bank(g, case["E"], *s["dims"], (0, 1, 2) if op == "experts" else (0, 1))
    if op in ("matmul", "grouped", "glu", "experts"):
        rows = T * case["k"] if op == "grouped" else T
        parts = [_codes(_grid(_normal(g, min(8192, rows - i), n, torch.float32), fmt)) for i in range(0, rows, 8192)]
        s["a"] = tuple(torch.cat(p) for p in zip(*parts))
    if own:  # the library's own handles on these tensors, made once by a program as it loads its weights
        import mxfp4_moe_expert_amd as k3g
        if "w" in s:
            s["w_own"] = k3g.mxfp4(*s["w"])
        if "bank" in s:
            s["bank_own"] = k3g.bank_struct(s["bank"].view(-1), case["E"], *s["dims"])
        if "a" in s:
            s["a_own"] = k3g.mx(*s["a"], _own_fmt(k3g, fmt))
    torch.cuda.synchronize()
    return s


# ---- the plain forms, in 32 bits ---------------------------------------------------------------------------------

def _grid(x, fmt):
    """x [T][n] in 32-groups: grid values v [T][n/32][32] and exponents e [T][n/32] (128 = a group with a value that
    is not finite, which has none), 2^e the smallest power of two that fits the group's largest entry."""
    x = x.reshape(x.shape[0], -1, 32)
    m = x.abs().amax(-1)
    frac, e = torch.frexp(m)
    e = (e - 3 + (frac > 0.75) if fmt == "fp4" else e - 9 + (frac > 0.875)).clamp(-126, 127)
    e = torch.where(m == 0, -126, e)
    fine = torch.isfinite(m)
    e = torch.where(fine, e, 0)
    v = torch.where(fine[..., None], x * torch.ldexp(torch.ones_like(m), -e)[..., None], 0.0)
    a = v.abs()
    if fmt == "fp4":
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    else:
        step = torch.ldexp(torch.ones_like(a), torch.frexp(a)[1].clamp(min=-5) - 4)
    return {"v": torch.round(v / step) * step, "x": torch.where(fine, e, 128), "fmt": fmt}


def _grid_values(q):
    v, x = q["v"], q["x"]
    scale = torch.where(x == 128, 0.0, torch.ldexp(torch.ones(x.shape, dtype=v.dtype, device=x.device), x)).to(v.dtype)
    return (v * scale[..., None]).reshape(v.shape[0], -1)


def _e2m1(device, dtype):
    """byte -> its two e2m1 values"""
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    one = torch.tensor(mags + [-m for m in mags], dtype=dtype, device=device)
    b = torch.arange(256, device=device)
    return torch.stack([one[b & 15], one[b >> 4]], 1)


def _values(codes, scales, fmt, dtype=torch.float32):
    """Values of codes [...][n or n/2] and scale bytes [...][n/32]."""
    lead = scales.shape
    v = _e2m1(codes.device, dtype)[codes.int()] if fmt == "fp4" else codes.view(torch.float8_e4m3fn).to(dtype)
    s = scales.int()
    s = torch.where(s == 255, 0.0, torch.ldexp(torch.ones(lead, dtype=dtype, device=s.device), s - 127)).to(dtype)
    return (v.reshape(*lead, 32) * s[..., None]).reshape(*lead[:-1], -1)


def _situ(g, u):
    return 4 * torch.tanh(g / 4) * torch.sigmoid(g) * (25 * torch.tanh(u / 25))


def _norm(s, dtype):
    """The residual sum and its norm."""
    h = s["x"].to(dtype) + s["r"].to(dtype)
    return h, h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["gamma"].to(dtype)


def _bank_tensor(s, t, experts, dtype):
    latent, inter = s["dims"]
    rows, cols = ((inter, latent), (inter, latent), (latent, inter))[t]
    off = _layout(latent, inter)[0]
    p = s["bank"][:, off[2 * t]:off[2 * t] + rows * cols // 2][experts].reshape(-1, rows, cols // 2)
    q = s["bank"][:, off[2 * t + 1]:off[2 * t + 1] + rows * cols // 32][experts].reshape(-1, rows, cols // 32)
    return _values(p, q, "fp4", dtype)


def _grouped(s, a, t, rows, dtype, src=None, step=64):
    """y[p] = W_t of p's expert times a[src[p]], a block of the experts with rows at a time, each group padded to the
    longest."""
    P = s["perm"].numel()
    y = torch.empty(P + 1, rows, dtype=dtype, device=a.device)  # the last row takes the padding
    off = s["offsets"].long()
    at = torch.arange(s["most"], device=a.device)
    for experts in s["active"].split(step):
        p = off[experts, None] + at
        p = torch.where(p < off[experts + 1, None], p, P)
        i = p.clamp(max=P - 1)
        part = torch.bmm(a[i if src is None else src[i]], _bank_tensor(s, t, experts, dtype).transpose(1, 2))
        y[p.reshape(-1)] = part.reshape(-1, rows)
    return y[:P]


def _plain(s):
    c = s["case"]
    op, fmt = c["op"], c["fmt"]
    f32 = torch.float32
    if op == "quantize":
        return _grid_values(_grid(s["x"].float(), fmt)).to(torch.bfloat16)
    if op in ("norm", "norm_matmul"):
        h, y = _norm(s, f32)
        q = _grid_values(_grid(y, fmt))
        if op == "norm":
            return {"sum": h.to(s["x"].dtype), "q": q.to(torch.bfloat16)}
        return {"sum": h.to(s["x"].dtype), "y": (q @ _values(*s["w"], "fp4").t()).to(TYPES[c["out"]])}
    a = _values(*s["a"], fmt)
    if op == "matmul":
        return (a @ _values(*s["w"], "fp4").t()).to(TYPES[c["out"]])
    if op == "grouped":
        return _grouped(s, a, 2, c["rows"], f32).to(TYPES[c["out"]])
    src = s["perm"].long() // c["k"]
    h = _situ(_grouped(s, a, 0, c["inter"], f32, src), _grouped(s, a, 1, c["inter"], f32, src))
    h = _grid_values(_grid(h, fmt))
    if op == "glu":
        return h.to(torch.bfloat16)
    return _grouped(s, h, 2, c["n"], f32).to(TYPES[c["out"]])


# ---- the library's operators -------------------------------------------------------------------------------------

def _own_fmt(k3g, fmt):
    return k3g.MXFP4 if fmt == "fp4" else k3g.MXFP8


def _own(s):
    import mxfp4_moe_expert_amd as k3g
    c = s["case"]
    op, fmt, n = c["op"], _own_fmt(k3g, c["fmt"]), c["n"]
    new = lambda rows, cols, t: torch.empty(rows, cols, dtype=TYPES[t], device="cuda")  # noqa: E731
    if op == "quantize":
        q = k3g.k3g_mx_quantize(k3g.mx_empty(c["T"], n, fmt), s["x"])
        return k3g.k3g_mx_dequantize(new(c["T"], n, "bf16"), q)
    if op in ("norm", "norm_matmul"):
        h, q = new(c["T"], n, c["type"]), k3g.mx_empty(c["T"], n, fmt)
        k3g.k3g_add_rmsnorm(s["x"], s["gamma"], EPS, r=s["r"], sum=h, q=q)
        if op == "norm":
            return {"sum": h, "q": k3g.k3g_mx_dequantize(new(c["T"], n, "bf16"), q)}
        return {"sum": h, "y": k3g.k3g_mx_matmul(new(c["T"], c["rows"], c["out"]), q, s["w_own"])}
    if op == "matmul":
        return k3g.k3g_mx_matmul(new(c["T"], c["rows"], c["out"]), s["a_own"], s["w_own"])
    P = c["T"] * c["k"]
    if op == "grouped":
        return k3g.k3g_mx_grouped_matmul(new(P, c["rows"], c["out"]), s["a_own"], s["bank_own"], k3g.W2, s["offsets"])
    h = k3g.k3g_mx_grouped_glu(k3g.mx_empty(P, c["inter"], fmt), s["a_own"], s["bank_own"], s["offsets"], perm=s["perm"],
                               top_k=c["k"])
    if op == "glu":
        return k3g.k3g_mx_dequantize(new(P, c["inter"], "bf16"), h)
    return k3g.k3g_mx_grouped_matmul(new(P, n, c["out"]), h, s["bank_own"], k3g.W2, s["offsets"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits -----------------------------------------------------------------------------------

def _exact_mx(y, fmt):
    """The values that a 64-bit row becomes: each group on the grid 2^e * (e2m1 or e4m3), nearest, ties to even."""
    y = y.double().reshape(y.shape[0], -1, 32)
    top, emin, bits = (6.0, 0, 1) if fmt == "fp4" else (448.0, -6, 3)
    m = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(m > 0, m, 1.0) / top))
    e = torch.where(torch.exp2(e - 1) * top >= m, e - 1, e)  # log2 is rounded: settle the exponent by comparing
    e = torch.where(torch.exp2(e) * top < m, e + 1, e)
    e = torch.where(m > 0, e, -126.0).clamp(-126, 127)
    a = (y / torch.exp2(e)).abs()
    b = torch.floor(torch.log2(a.clamp(min=2.0 ** emin)))
    b = torch.where(torch.exp2(b) > a.clamp(min=2.0 ** emin), b - 1, b)
    b = torch.where(torch.exp2(b + 1) <= a, b + 1, b)
    ulp = torch.exp2(b - bits)
    r = torch.round(a / ulp) * ulp * torch.exp2(e)
    return torch.copysign(r, y).reshape(r.shape[0], -1)


def _exact_values(codes, scales, fmt):
    """The definition of the format: sign, exponent and mantissa of each code, times 2^(byte - 127)."""
    c = codes.to(torch.int16)
    if fmt == "fp4":
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        sign, e, m, bias, mbits = c >> 3, (c >> 1) & 3, c & 1, 1, 1
    else:
        sign, e, m, bias, mbits = c >> 7, (c >> 3) & 15, c & 7, 7, 3
    frac = m.double() / (1 << mbits)
    v = torch.where(e > 0, (1 + frac) * torch.exp2(e.double() - bias), frac * 2.0 ** (1 - bias))
    v = torch.where(sign > 0, -v, v)
    s = scales.double().repeat_interleave(32, -1)
    return torch.where(s == 255, 0.0, v * torch.exp2(s - 127))


def _exact_bank(s, t, e):
    latent, inter = s["dims"]
    rows, cols = ((inter, latent), (inter, latent), (latent, inter))[t]
    off = _layout(latent, inter)[0]
    b = s["bank"][e]
    return _exact_values(b[off[2 * t]:off[2 * t] + rows * cols // 2].view(rows, -1),
                         b[off[2 * t + 1]:off[2 * t + 1] + rows * cols // 32].view(rows, -1), "fp4")


def _exact_experts(s, a, tensors, src, rows):
    """For each expert with rows: [W_t a for t in tensors] of its rows."""
    off = s["offsets"].tolist()
    outs = [torch.empty(off[-1], rows, dtype=torch.float64, device=a.device) for _ in tensors]
    for e in range(s["case"]["E"]):
        if off[e + 1] > off[e]:
            p = torch.arange(off[e], off[e + 1], device=a.device)
            x = a[p if src is None else src[p]]
            for y, t in zip(outs, tensors):
                y[p] = x @ _exact_bank(s, t, e).t().contiguous()
    return outs


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = case["op"], case["fmt"]
    if op == "quantize":
        return _exact_mx(s["x"], fmt)
    if op in ("norm", "norm_matmul"):
        h = s["x"].double() + s["r"].double()
        q = _exact_mx(h / torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[1] + EPS) * s["gamma"].double(), fmt)
        return {"sum": h, "q": q} if op == "norm" else {"sum": h, "y": q @ _exact_values(*s["w"], "fp4").t().contiguous()}
    a = _exact_values(*s["a"], fmt)
    if op == "matmul":
        return a @ _exact_values(*s["w"], "fp4").t().contiguous()
    if op == "grouped":
        return _exact_experts(s, a, (2,), None, case["rows"])[0]
    src = torch.div(s["perm"].long(), case["k"], rounding_mode="floor")
    g, u = _exact_experts(s, a, (0, 1), src, case["inter"])
    h = _exact_mx(100 * torch.tanh(g / 4) * torch.tanh(u / 25) / (1 + torch.exp(-g)), fmt)
    return h if op == "glu" else _exact_experts(s, h, (2,), None, case["n"])[0]
