"""The fp8 and grouped products as cases to measure: inputs, plain forms and 64-bit references.

Operators (rows of X are tokens, weights are stored [contraction, output] as everywhere in the library):

  quantize          bf16 activations -> e4m3 values and one fp32 scale for each row and block of 128 columns
  quantize_weight   bf16 weights -> e4m3 values and one fp32 scale for each block of 128 x 128
  linear_fp8        the product of the two
  grouped           bf16 product of each expert's rows with that expert's weights (rows sorted by expert, ragged)
  grouped_fp8       the same on fp8 operands with block scales
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0


def _blocks(x):
    return -(-x // BLOCK)


def _up(x, to):
    return -(-x // to) * to


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a 4096-wide model on its way into an fp8 projection
        {"name": "quantize 1 x 4096", "op": "quantize", "n": 1, "d": 4096},
        # an odd batch, a width that is no multiple of the block
        {"name": "quantize 777 x 1000", "op": "quantize", "n": 777, "d": 1000},
        # the MLP's inner activations of a long prompt
        {"name": "quantize 8192 x 14336", "op": "quantize", "n": 8192, "d": 14336},
        # eight experts' weights at load time
        {"name": "quantize weights 8 x 4096 x 14336", "op": "quantize_weight", "groups": 8, "d": 4096, "m": 14336},
        # decoding eight sequences through the MLP-up projection of an 8192-wide model
        {"name": "fp8 8 x 8192 x 28672", "op": "linear_fp8", "n": 8, "d": 8192, "m": 28672},
        # a short prompt and a small layer, nothing a multiple of a tile
        {"name": "fp8 333 x 1000 x 1522", "op": "linear_fp8", "n": 333, "d": 1000, "m": 1522},
        # a prompt of 4096 tokens through the gate projection
        {"name": "fp8 4096 x 4096 x 14336", "op": "linear_fp8", "n": 4096, "d": 4096, "m": 14336},
        # decoding 32 sequences, two of eight experts each
        {"name": "grouped 64 x 4096 x 14336 of 8", "op": "grouped", "n": 64, "d": 4096, "m": 14336, "groups": 8,
         "skew": 0.3, "tail": 0},
        # many small experts, unevenly popular, some rows of the buffer unused
        {"name": "grouped 4096 x 2048 x 1408 of 64", "op": "grouped", "n": 4096, "d": 2048, "m": 1408, "groups": 64,
         "skew": 1.0, "tail": 100},
        # a prompt of 4096 tokens, two of eight experts each
        {"name": "grouped 8192 x 4096 x 14336 of 8", "op": "grouped", "n": 8192, "d": 4096, "m": 14336, "groups": 8,
         "skew": 0.3, "tail": 0},
        # decoding 32 sequences, eight of 128 experts each: most experts see a row or two, some none
        {"name": "grouped fp8 256 x 2048 x 1536 of 128", "op": "grouped_fp8", "n": 256, "d": 2048, "m": 1536,
         "groups": 128, "skew": 0.7, "tail": 0},
        # the down projection of the prompt above, in fp8
        {"name": "grouped fp8 8192 x 14336 x 4096 of 8", "op": "grouped_fp8", "n": 8192, "d": 14336, "m": 4096,
         "groups": 8, "skew": 0.3, "tail": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A width: one in three odd or otherwise unaligned, the others multiples of 64."""
    x = _log(rng, lo, hi)
    return x if rng.random() < 0.34 else max(64, x // 64 * 64)


def draw(rng):
    op = rng.choice(["quantize", "quantize_weight", "linear_fp8", "linear_fp8", "grouped", "grouped", "grouped_fp8",
                     "grouped_fp8"])
    most_weights = 8 * 4096 * 14336
    most_products = 8192 * 4096 * 14336
    if op == "quantize":
        return {"op": op, "n": _log(rng, 1, 8192), "d": _size(rng, 64, 14336)}
    d, m = _size(rng, 64, 14336), _size(rng, 64, 28672)
    if op == "linear_fp8":
        n = min(_log(rng, 1, 8192), most_products // (d * m))
        return {"op": op, "n": n, "d": d, "m": m}
    groups = max(1, min(_log(rng, 1, 128), most_weights // (d * m)))
    if op == "quantize_weight":
        return {"op": op, "groups": groups, "d": d, "m": m}
    n = max(1, min(_log(rng, 1, 16384), most_products // (d * m)))
    return {"op": op, "n": n, "d": d, "m": m, "groups": groups, "skew": round(rng.uniform(0.0, 1.0), 2),
            "tail": rng.choice([0, 0, rng.randrange(1, 200)])}


# ------------------------------------------------------------------ inputs
def _padded(x, to):
    """x in a buffer whose row length is a multiple of `to` elements (the library's rule for leading dimensions)."""
    ld = _up(x.shape[-1], to)
    if ld == x.shape[-1]:
        return x
    buf = torch.zeros((*x.shape[:-1], ld), dtype=torch.bfloat16, device=x.device).to(x.dtype)
    buf[..., : x.shape[-1]] = x
    return buf[..., : x.shape[-1]]


def _activations(g, n, d):
    """Normal values with a spread of channel sizes and a few outlier channels, as activations have; the last row of a
    batch of more than 8 is padding (zeros)."""
    size = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    size = torch.where(torch.rand(d, generator=g, device="cuda") < 0.01, 20 * size, size)
    x = torch.randn(n, d, generator=g, device="cuda") * size
    if n > 8:
        x[-1] = 0
    return x.bfloat16()


def _weights(g, groups, d, m):
    w = torch.empty((groups, d, m), dtype=torch.bfloat16, device="cuda")
    return w.normal_(0.0, d ** -0.5, generator=g)


def _offsets(seed, n, groups, skew):
    """Rows of each expert, drawn from popularities exp(skew * normal): int32 [groups + 1] on the GPU, and the longest."""
    g = torch.Generator().manual_seed(seed)
    p = torch.exp(skew * torch.randn(groups, generator=g))
    counts = torch.bincount(torch.multinomial(p, n, replacement=True, generator=g), minlength=groups)
    off = torch.zeros(groups + 1, dtype=torch.int32)
    off[1:] = counts.cumsum(0)
    return off.cuda(), int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, d = case["op"], case["d"]
    if op == "quantize":
        return {"op": op, "x": _padded(_activations(g, case["n"], d), 8)}
    m = case["m"]
    if op == "quantize_weight":
        return {"op": op, "w": _padded(_weights(g, case["groups"], d, m), 8)}
    s = {"op": op}
    n = case["n"] + case.get("tail", 0)
    x, w = _activations(g, n, d), _weights(g, case.get("groups", 1), d, m)
    if op == "grouped":
        s["x"], s["w"] = _padded(x, 8), _padded(w, 8)
    else:
        xq, s["sx"] = _quantize(x)
        wq, s["sw"] = _quantize_weight(w)
        s["xq"], s["wq"] = _padded(xq, 16), _padded(wq, 16)
    if op == "linear_fp8":
        s["wq"], s["sw"] = s["wq"][0], s["sw"][0]
    else:
        s["offsets"], s["most"] = _offsets(seed, case["n"], case["groups"], case["skew"])
        s["rows"] = case["n"]
        s["out"] = _padded(torch.full((n, m), 0.5, dtype=torch.bfloat16, device="cuda"), 8)
    return s


# ------------------------------------------------------------------ plain forms
def _scale(amax):
    s = amax / torch.full_like(amax, E4M3_MAX)  # a tensor: division by a number multiplies by its reciprocal
    return torch.where(s == 0, torch.ones_like(s), s)


def _quantize(x):
    n, d = x.shape
    nb = _blocks(d)
    x32 = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - d)).view(n, nb, BLOCK)
    s = _scale(x32.abs().amax(2))
    q = (x32 / s[:, :, None]).to(torch.float8_e4m3fn).view(n, nb * BLOCK)[:, :d]
    return q, s.t().contiguous()


def _quantize_weight(w):
    e, d, m = w.shape
    db, mb = _blocks(d), _blocks(m)
    w32 = torch.nn.functional.pad(w.float(), (0, mb * BLOCK - m, 0, db * BLOCK - d)).view(e, db, BLOCK, mb, BLOCK)
    s = _scale(w32.abs().amax((2, 4)))
    q = (w32 / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(e, db * BLOCK, mb * BLOCK)[:, :d, :m]
    return q, s


def _wide_x(xq, sx):
    return xq.float() * sx.t().repeat_interleave(BLOCK, 1)[:, : xq.shape[1]]


def _wide_w(wq, sw):
    return wq.float() * sw.repeat_interleave(BLOCK, -2).repeat_interleave(BLOCK, -1)[..., : wq.shape[-2], : wq.shape[-1]]


def _grouped(x, w, offsets, rows, most, out):
    """Each expert's rows side by side, padded to the longest, one batched product, the rows taken out again."""
    i = torch.arange(rows, device=x.device)
    e = torch.searchsorted(offsets[1:], i, right=True, out_int32=False)
    at = i - offsets[e]
    wide = torch.zeros((w.shape[0], most, x.shape[1]), dtype=torch.float32, device=x.device)
    wide[e, at] = x[:rows]
    out[:rows] = torch.bmm(wide, w)[e, at].bfloat16()
    return out


def run(s):
    op = s["op"]
    if own:
        import input_adaptive_reduced_colnorm_b200 as rmm

        if op == "quantize":
            return rmm.quantize_fp8(s["x"])
        if op == "quantize_weight":
            return rmm.quantize_fp8_weight(s["w"])
        if op == "linear_fp8":
            return rmm.linear_fp8(s["xq"], s["sx"], s["wq"], s["sw"])
        if op == "grouped":
            return rmm.grouped_linear(s["x"], s["w"], s["offsets"], out=s["out"])
        return rmm.grouped_linear_fp8(s["xq"], s["sx"], s["wq"], s["sw"], s["offsets"], out=s["out"])
    if op == "quantize":
        return _quantize(s["x"])
    if op == "quantize_weight":
        return _quantize_weight(s["w"])
    if op == "linear_fp8":
        return (_wide_x(s["xq"], s["sx"]) @ _wide_w(s["wq"], s["sw"])).bfloat16()
    if op == "grouped":
        return _grouped(s["x"].float(), s["w"].float(), s["offsets"], s["rows"], s["most"], s["out"])
    return _grouped(_wide_x(s["xq"], s["sx"]), _wide_w(s["wq"], s["sw"]), s["offsets"], s["rows"], s["most"], s["out"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, d = case["op"], case["d"]
    if op == "quantize":
        n = case["n"]
        return {"bytes": 3 * n * d + 4 * n * _blocks(d), "flops": 3 * n * d}
    m = case["m"]
    if op == "quantize_weight":
        e = case["groups"]
        return {"bytes": 3 * e * d * m + 4 * e * _blocks(d) * _blocks(m), "flops": 3 * e * d * m}
    n = case["n"]
    # experts that a batch of n rows reaches, taken as equally popular
    e = case.get("groups", 1)
    e = e * (1 - (1 - 1 / e) ** n) if e > 1 else 1
    if op == "grouped":
        return {"bytes": 2 * (n * d + e * d * m + n * m), "flops": 2 * n * d * m}
    scales = 4 * (_blocks(d) * n + e * _blocks(d) * _blocks(m))
    return {"bytes": n * d + e * d * m + 2 * n * m + scales, "flops": 2 * n * d * m}


# ------------------------------------------------------------------ 64 bits
def _exact_scale(amax):
    """The stored scale is fp32 by definition: the block's largest size over 448, rounded once; 1 where that is 0."""
    s = (amax / 448.0).float()
    return torch.where(s > 0, s, torch.ones_like(s))


def _exact_codes(x, s):
    """e4m3 values nearest to x / s, where the quotient is an fp32 number by definition; ties to even."""
    v = (x / s.double()).float().double()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "quantize":
        x = s["x"].double()
        scales, codes = [], torch.empty_like(x)
        for b in range(_blocks(d)):
            cols = slice(b * 128, min(d, b * 128 + 128))
            sb = _exact_scale(x[:, cols].abs().amax(1))
            codes[:, cols] = _exact_codes(x[:, cols], sb[:, None])
            scales.append(sb)
        return codes, torch.stack(scales)
    m = case["m"]
    if op == "quantize_weight":
        w = s["w"]
        codes = torch.empty(w.shape, dtype=torch.float32, device=w.device)
        scales = torch.empty((w.shape[0], _blocks(d), _blocks(m)), dtype=torch.float32, device=w.device)
        for e in range(w.shape[0]):
            for b in range(_blocks(d)):
                band = w[e, b * 128:(b + 1) * 128].double()
                top = torch.zeros(_blocks(m) * 128, dtype=torch.float64, device=w.device)
                top[:m] = band.abs().amax(0)
                sb = _exact_scale(top.view(-1, 128).amax(1))
                scales[e, b] = sb
                codes[e, b * 128:(b + 1) * 128] = _exact_codes(band, sb.repeat_interleave(128)[:m])
        return codes, scales
    rows = case["n"] + case.get("tail", 0)
    y = torch.full((rows, m), 0.5, dtype=torch.float64, device="cuda")
    bounds = s["offsets"].tolist() if "offsets" in s else [0, rows]
    for e in range(len(bounds) - 1):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        if op == "grouped":
            y[lo:hi] = s["x"][lo:hi].double() @ s["w"][e].double()
            continue
        wq, sw = (s["wq"], s["sw"]) if op == "linear_fp8" else (s["wq"][e], s["sw"][e])
        wide = torch.empty((d, m), dtype=torch.float64, device="cuda")
        x = torch.empty((hi - lo, d), dtype=torch.float64, device="cuda")
        for b in range(_blocks(d)):
            at = slice(b * 128, min(d, b * 128 + 128))
            wide[at] = wq[at].double() * sw[b].double().repeat_interleave(128)[:m]
            x[:, at] = s["xq"][lo:hi, at].double() * s["sx"][b, lo:hi].double()[:, None]
        y[lo:hi] = x @ wide
    return y
