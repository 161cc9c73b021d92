"""GPU parity of the fp8 and grouped products: quantize_fp8, quantize_fp8_weight,
linear_fp8, grouped_linear, grouped_linear_fp8, against the float64 oracle.

Tolerances.  The quantisers are exact: equal codes and scales.  A product of d
terms summed in fp32 in any order, each step off by at most 2^-23 relative (a
truncating adder; a rounding one is off by 2^-24), is within
    E = (d + 4) 2^-23 sum_j |x_j w_j|
of the exact value (with block scales, two more products per block are in the 4);
the result is then rounded once to bf16, by at most 2^-8 of its value:
    |y - ref| <= 2^-8 (|ref| + E) + E.
"""
import numpy as np
import pytest
import torch

import oracle
import synthetic

pytestmark = pytest.mark.gpu

rmm = pytest.importorskip("input_adaptive_reduced_colnorm_b200")

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from input_adaptive_reduced_colnorm_b200 import build
    build.build()
    yield
    assert rmm.device_error() == 0


def padded(t, unit, extra=0, fill=float("nan")):
    """t on the GPU in a buffer of NaN whose row stride is a multiple of `unit`, `extra` units wider than needed."""
    ld = -(-t.shape[-1] // unit) * unit + extra * unit
    buf = torch.full((*t.shape[:-1], ld), fill, dtype=torch.float32, device="cuda").to(t.dtype)
    buf[..., : t.shape[-1]] = t.cuda()
    return buf[..., : t.shape[-1]]


def wide(t):
    return t.detach().cpu().to(torch.float64).numpy()


def check(Y, ref, mag, d, what):
    """mag = sum_j |x_j w_j| (0 where Y keeps a value of its own)."""
    Y = wide(Y)
    E = (d + 4) * 2.0 ** -23 * mag
    bound = np.where(mag > 0, 2.0 ** -8 * (np.abs(ref) + E) + E, 0.0)
    bad = ~(np.abs(Y - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[:5].tolist()}, " \
                          f"got {Y[bad][:5]} for {ref[bad][:5]}"


def bounds_of(sizes, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(sizes)]), dtype=torch.int32)


# ------------------------------------------------------------------ quantisers
@pytest.mark.parametrize("n,d", [(1, 1), (1, 4096), (3, 129), (15, 130), (16, 128), (17, 640), (40, 1000), (130, 7)])
def test_quantize_matches_the_oracle(n, d):
    g = synthetic.rng(51)
    X = synthetic.to_bf16(synthetic.outlier_activations(g, n, d, 1.5))
    q, s = rmm.quantize_fp8(padded(X, 8, extra=1))
    rq, rs = oracle.quantize_fp8(synthetic.widen(X))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(wide(q), rq)


@pytest.mark.parametrize("groups,d,m", [(1, 1, 1), (1, 128, 128), (2, 300, 520), (3, 129, 77)])
def test_quantize_weight_matches_the_oracle(groups, d, m):
    g = synthetic.rng(52)
    W = synthetic.to_bf16(g.standard_normal((groups, d, m)))
    q, s = rmm.quantize_fp8_weight(padded(W, 8, extra=1))
    for e in range(groups):
        rq, rs = oracle.quantize_fp8_weight(synthetic.widen(W[e]))
        assert np.array_equal(s[e].cpu().numpy(), rs)
        assert np.array_equal(wide(q[e]), rq)
    q2, s2 = rmm.quantize_fp8_weight(padded(W[0], 8))
    assert torch.equal(q2.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s2, s[0])


def test_quantize_every_value_under_many_scales():
    """Every finite bf16 value, next to block maxima of every mantissa and a spread of
    exponents, the smallest and the largest among them: the codes are those of the
    IEEE division."""
    mant = np.arange(128, 256, dtype=np.float64)
    for e in (-133, -120, -100, -97, -60, -8, 0, 30, 119, 120):
        top = np.float32(1) * mant * 2.0 ** e
        top = top[np.isfinite(synthetic.widen(synthetic.to_bf16(top)))]
        rows = []
        for k in range(0, 20):  # values of every mantissa, down to 2^-19 of the maximum's size
            rows.append(mant[None, :127] * 2.0 ** (e - k) * np.where(np.arange(127) % 2, -1.0, 1.0))
        vals = np.concatenate(rows)                                     # [20, 127]
        vals[::7, 5] = mant[127] * 2.0 ** (e - 3)
        X = np.concatenate([np.repeat(vals, len(top), 0), np.tile(top, len(vals))[:, None]], 1)
        X = np.minimum(np.abs(X), X[:, -1:]) * np.sign(X)
        Xb = synthetic.to_bf16(X)
        q, s = rmm.quantize_fp8(Xb.cuda())
        rq, rs = oracle.quantize_fp8(synthetic.widen(Xb))
        assert np.array_equal(s.cpu().numpy(), rs), e
        assert np.array_equal(wide(q), rq), e


def test_quantize_special_values():
    """Zero blocks (scale 1), negative zero, NaN and infinity: only their own block is touched."""
    X = torch.zeros((18, 256), dtype=torch.bfloat16)
    X[:, 128:] = 1.0
    X[1, 5] = -0.0
    X[2, 5] = float("nan")
    X[3, 5], X[3, 6] = float("inf"), 2.0
    X[4, 200] = float("-inf")
    q, s = rmm.quantize_fp8(X.cuda())
    q, s = wide(q), s.cpu().numpy()
    one = np.float32(1) / np.float32(448)
    assert s[0, [0, 1, 4]].tolist() == [1, 1, 1] and (s[1, [0, 1, 2, 3]] == one).all()
    assert np.isnan(s[0, 2]) and np.isinf(s[0, 3]) and np.isinf(s[1, 4])
    assert not q[[0, 1, 4], :128].any() and (q[:4, 128:] == 448).all()
    assert np.isnan(q[2, :128]).all()
    assert np.isnan(q[3, 5]) and q[3, 6] == 0 and np.isnan(q[4, 200]) and q[4, 201] == 0


def test_quantize_leaves_padding_alone():
    X = synthetic.to_bf16(synthetic.rng(53).standard_normal((20, 130)))
    out = torch.full((24, 160), 7.0, device="cuda").to(F8)
    scale = torch.full((3, 32), 5.0, device="cuda")
    rmm.quantize_fp8(padded(X, 8), out=out[:20, :130], scale=scale[:2, :20])
    assert (out[:, 130:].float() == 7).all() and (out[20:].float() == 7).all()
    assert (scale[2:] == 5).all() and (scale[:, 20:] == 5).all()
    rq, rs = oracle.quantize_fp8(synthetic.widen(X))
    assert np.array_equal(wide(out[:20, :130]), rq) and np.array_equal(scale[:2, :20].cpu().numpy(), rs)


# ------------------------------------------------------------------ products
def fp8_operands(seed, n, d, m, groups=None):
    g = synthetic.rng(seed)
    X = synthetic.outlier_activations(g, n, d, 1.0)
    q, s = oracle.quantize_fp8(synthetic.widen(synthetic.to_bf16(X)))
    ws = [oracle.quantize_fp8_weight(synthetic.widen(synthetic.to_bf16(g.standard_normal((d, m)) / np.sqrt(d))))
          for _ in range(groups or 1)]
    to8 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(torch.float32).to(F8)  # noqa: E731
    wq = to8(np.stack([w for w, _ in ws]))
    sw = torch.from_numpy(np.stack([w for _, w in ws])).cuda()
    dev = {"xq": padded(to8(q), 16, extra=1), "sx": torch.from_numpy(s).cuda(), "wq": padded(wq, 16), "sw": sw}
    if groups is None:
        dev["wq"], dev["sw"] = dev["wq"][0], dev["sw"][0]
    return dev, oracle.fp8_widen(q, s), [oracle.fp8_widen_weight(*w) for w in ws]


@pytest.mark.parametrize("n", [1, 16, 17, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("d,m", [(1, 1), (128, 128), (130, 520), (1000, 1522), (512, 2048)])
def test_linear_fp8(n, d, m):
    dev, X, W = fp8_operands(61, n, d, m)
    Y = rmm.linear_fp8(dev["xq"], dev["sx"], dev["wq"], dev["sw"])
    check(Y, X @ W[0], np.abs(X) @ np.abs(W[0]), d, f"fp8 {n} x {d} x {m}")


SIZES = [
    [1],
    [0, 0, 1],
    [5, 0, 16, 3],
    [17, 31, 0, 1, 40],
    [64, 60, 1, 130],
    [0, 128, 100, 129],
    [300, 0, 257, 5],
    [1000],
]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("d,m", [(1, 1), (72, 136), (200, 777), (520, 1100)])
def test_grouped_linear(sizes, d, m):
    """Two rows before the first group and three behind the last keep their values."""
    g = synthetic.rng(62)
    n, E = sum(sizes) + 5, len(sizes)
    X = synthetic.to_bf16(synthetic.outlier_activations(g, n, d, 1.0))
    W = synthetic.to_bf16(g.standard_normal((E, d, m)) / np.sqrt(d))
    X[:2] = float("nan")   # not in a group: never seen
    X[-3:] = float("inf")
    off = bounds_of(sizes, 2)
    out = padded(torch.full((n, m), 3.0, dtype=torch.bfloat16), 8, extra=1, fill=9.0)
    base = out.as_strided((n, out.stride(0)), (out.stride(0), 1))
    Y = rmm.grouped_linear(padded(X, 8, extra=1), padded(W, 8, extra=1), off.cuda(), out=out)
    Xw, Ww = np.nan_to_num(synthetic.widen(X), nan=0, posinf=0), synthetic.widen(W)
    ref = oracle.grouped_product(Xw, Ww, off.numpy(), np.full((n, m), 3.0))
    mag = oracle.grouped_product(np.abs(Xw), np.abs(Ww), off.numpy(), np.zeros((n, m)))
    check(Y, ref, mag, d, f"grouped {sizes} {d} x {m}")
    assert (base[:, m:] == 9).all()


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("d,m", [(1, 1), (130, 520), (520, 1100)])
def test_grouped_linear_fp8(sizes, d, m):
    n, E = sum(sizes) + 3, len(sizes)
    dev, X, W = fp8_operands(63, n, d, m, E)
    dev["xq"][-3:] = float("nan")
    off = bounds_of(sizes)
    out = padded(torch.full((n, m), 3.0, dtype=torch.bfloat16), 8)
    Y = rmm.grouped_linear_fp8(dev["xq"], dev["sx"], dev["wq"], dev["sw"], off.cuda(), out=out)
    ref = oracle.grouped_product(X, W, off.numpy(), np.full((n, m), 3.0))
    mag = oracle.grouped_product(np.abs(X), [np.abs(w) for w in W], off.numpy(), np.zeros((n, m)))
    check(Y, ref, mag, d, f"grouped fp8 {sizes} {d} x {m}")


# (rows of the groups, d, m): the shapes of tile that the library chooses by the rows of
# an average group and the number of tiles, each with groups that end inside a tile
TILES = [
    ([3, 0, 16, 1, 17, 9], 300, 4200),                     # 16 rows x 256 columns
    ([30, 1, 33, 32, 0, 16, 40, 31], 200, 2600),           # 32 x 512
    ([64, 70, 0, 1, 63, 40, 65, 64, 50, 60], 264, 2100),   # 64 x 256
    ([129, 255, 0, 256, 257, 300, 1], 130, 2300),          # 256 x 256 (fp8 128 x 256), one wave
    ([1000, 31, 130], 200, 4100),                          # the same, a last wave of narrow pieces
    ([128, 127, 100, 1, 129, 64], 1100, 3300),             # fp8 128 x 256, more than 8 blocks
    ([150, 20, 300], 4300, 2100),                          # more than 32 blocks
    ([1030], 72, 5000),
    ([200, 513, 290], 1000, 5100),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("sizes,d,m", TILES, ids=str)
def test_every_tile_shape(sizes, d, m, fp8):
    n, E = sum(sizes) + 3, len(sizes)
    off = bounds_of(sizes, 1)
    out = padded(torch.full((n, m), 3.0, dtype=torch.bfloat16), 8)
    if fp8:
        dev, X, W = fp8_operands(71, n, d, m, E)
        Y = rmm.grouped_linear_fp8(dev["xq"], dev["sx"], dev["wq"], dev["sw"], off.cuda(), out=out)
    else:
        g = synthetic.rng(71)
        Xb = synthetic.to_bf16(synthetic.outlier_activations(g, n, d, 1.0))
        Wb = synthetic.to_bf16(g.standard_normal((E, d, m)) / np.sqrt(d))
        X, W = synthetic.widen(Xb), synthetic.widen(Wb)
        Y = rmm.grouped_linear(padded(Xb, 8, extra=1), padded(Wb, 8), off.cuda(), out=out)
    again = Y.clone()
    behind = out.as_strided((n, out.stride(0)), (out.stride(0), 1))[:, m:]
    assert behind.isnan().all()  # the buffer's columns past m are as they were
    ref = oracle.grouped_product(X, W, off.numpy(), np.full((n, m), 3.0))
    mag = oracle.grouped_product(np.abs(X), [np.abs(w) for w in W], off.numpy(), np.zeros((n, m)))
    check(Y, ref, mag, d, f"{sizes} {d} x {m}")
    for _ in range(3):  # the same result every time
        if fp8:
            rmm.grouped_linear_fp8(dev["xq"], dev["sx"], dev["wq"], dev["sw"], off.cuda(), out=out)
        else:
            rmm.grouped_linear(padded(Xb, 8, extra=1), padded(Wb, 8), off.cuda(), out=out)
        assert torch.equal(out, again)


@pytest.mark.parametrize("n,d,m", [(1, 4096, 1000), (20, 2000, 1522), (7, 130, 9000), (40, 8192, 300), (300, 3000, 520)])
@pytest.mark.parametrize("fp8", [False, True])
def test_split_contraction(n, d, m, fp8):
    """Few tiles: the contraction of one is shared by a cluster, with block counts that do
    not divide by its size and row tiles that are not full."""
    if fp8:
        dev, X, W = fp8_operands(72, n, d, m)
        Y = rmm.linear_fp8(dev["xq"], dev["sx"], dev["wq"], dev["sw"])
        W = W[0]
    else:
        g = synthetic.rng(72)
        Xb = synthetic.to_bf16(synthetic.outlier_activations(g, n, d, 1.0))
        Wb = synthetic.to_bf16(g.standard_normal((1, d, m)) / np.sqrt(d))
        X, W = synthetic.widen(Xb), synthetic.widen(Wb)[0]
        Y = rmm.grouped_linear(padded(Xb, 8), padded(Wb, 8), torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    check(Y, X @ W, np.abs(X) @ np.abs(W), d, f"{n} x {d} x {m}")


def test_all_rows_in_one_of_many_groups():
    """An average group of one row, and one that has them all (more tiles than a launch
    that splits the contraction takes them to be)."""
    g = synthetic.rng(73)
    n, d, m, E = 150, 300, 640, 150
    X = synthetic.to_bf16(g.standard_normal((n, d)))
    W = synthetic.to_bf16(g.standard_normal((E, d, m)))
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[78:] = n
    Y = rmm.grouped_linear(padded(X, 8), W.cuda(), off.cuda())
    Xw, Ww = synthetic.widen(X), synthetic.widen(W[77])
    check(Y, Xw @ Ww, np.abs(Xw) @ np.abs(Ww), d, "one group")
    off4 = torch.tensor([0, 0, 0, n, n], dtype=torch.int32)  # three of four groups empty
    Y = rmm.grouped_linear(padded(X, 8), W[:4].cuda(), off4.cuda())
    Ww = synthetic.widen(W[2])
    check(Y, Xw @ Ww, np.abs(Xw) @ np.abs(Ww), d, "one of four")


def test_offsets_past_32_bits():
    """Outputs and weights of more than 2^31 elements: the last rows and the last group."""
    n, d, m = 66000, 16, 33000
    g = torch.Generator(device="cuda").manual_seed(74)
    X = torch.randn((n, d), generator=g, device="cuda").bfloat16()
    W = torch.randn((2, d, m), generator=g, device="cuda").bfloat16()
    off = torch.tensor([0, 40000, n], dtype=torch.int32, device="cuda")
    Y = rmm.grouped_linear(X, W, off)
    xq, sx = rmm.quantize_fp8(X)
    wq, sw = rmm.quantize_fp8_weight(W)
    Yq = rmm.grouped_linear_fp8(xq, sx, wq, sw, off)
    rows = [0, 39999, 40000, n - 1]
    for r in rows:
        e = int(r >= 40000)
        x, w = wide(X[r]), wide(W[e])
        check(Y[r], x @ w, np.abs(x) @ np.abs(w), d, f"row {r}")
        x, w = oracle.fp8_widen(wide(xq[r:r + 1]), sx[:, r:r + 1].cpu().numpy()), oracle.fp8_widen_weight(wide(wq[e]), sw[e].cpu().numpy())
        check(Yq[r:r + 1], x @ w, np.abs(x) @ np.abs(w), d, f"fp8 row {r}")
    del Y, Yq
    E, d, m = 5, 20480, 26624                       # 2.7e9 weights
    W = torch.zeros((E, d, m), dtype=F8, device="cuda")
    W[4, -1, -1] = 2.0
    W[3, 0, 0] = 1.0
    xq = torch.ones((2, d), device="cuda").to(F8)
    sx = torch.ones((d // 128, 2), device="cuda")
    sw = torch.ones((E, d // 128, m // 128), device="cuda")
    off = torch.tensor([0, 0, 0, 0, 1, 2], dtype=torch.int32, device="cuda")
    Y = rmm.grouped_linear_fp8(xq, sx, W, sw, off)
    assert Y[0, 0] == 1 and Y[1, -1] == 2 and Y.abs().sum() == 3


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_offsets_are_clamped(fp8):
    """Negative, falling and too large bounds read and write nothing out of range."""
    n, d, m = 40, 136, 264
    off = torch.tensor([-5, 10, 4, 1 << 30, 20, 2_000_000_000], dtype=torch.int32)
    out = torch.full((n, m), 3.0, dtype=torch.bfloat16, device="cuda")
    if fp8:
        dev, X, W = fp8_operands(64, n, d, m, 5)
        Y = rmm.grouped_linear_fp8(dev["xq"], dev["sx"], dev["wq"], dev["sw"], off.cuda(), out=out)
    else:
        g = synthetic.rng(64)
        Xb = synthetic.to_bf16(g.standard_normal((n, d)))
        Wb = synthetic.to_bf16(g.standard_normal((5, d, m)))
        X, W = synthetic.widen(Xb), synthetic.widen(Wb)
        Y = rmm.grouped_linear(padded(Xb, 8), padded(Wb, 8), off.cuda(), out=out)
    ref = oracle.grouped_product(X, W, off.numpy(), np.full((n, m), 3.0))
    mag = oracle.grouped_product(np.abs(X), [np.abs(w) for w in W], off.numpy(), np.zeros((n, m)))
    check(Y, ref, mag, d, "clamped bounds")


def test_many_groups():
    """The most groups allowed, most of them empty, and bounds on both sides of a scan's chunk of 32."""
    g = synthetic.rng(65)
    E, d, m = 1024, 64, 64
    sizes = (g.random(E) < 0.1).astype(int) * g.integers(1, 60, E)
    sizes[31:34] = [3, 0, 40]
    n = int(sizes.sum())
    X = synthetic.to_bf16(g.standard_normal((n, d)))
    W = synthetic.to_bf16(g.standard_normal((E, d, m)))
    off = bounds_of(sizes)
    Y = rmm.grouped_linear(X.cuda(), W.cuda(), off.cuda())
    Xw, Ww = synthetic.widen(X), synthetic.widen(W)
    check(Y, oracle.grouped_product(Xw, Ww, off.numpy(), np.zeros((n, m))),
          oracle.grouped_product(np.abs(Xw), np.abs(Ww), off.numpy(), np.zeros((n, m))), d, "1024 groups")


def test_no_rows():
    W = torch.zeros((2, 64, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    X = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    assert rmm.grouped_linear(X, W, off).shape == (0, 64)
    q, s = rmm.quantize_fp8(X)
    wq, sw = rmm.quantize_fp8_weight(W)
    assert q.shape == (0, 64) and s.shape == (1, 0)
    assert rmm.linear_fp8(q, s, wq[0], sw[0]).shape == (0, 64)
    assert rmm.grouped_linear_fp8(q, s, wq, sw, off).shape == (0, 64)


def test_all_groups_empty():
    W = torch.ones((3, 64, 64), dtype=torch.bfloat16, device="cuda")
    X = torch.ones((9, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full((9, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    for v in (0, 4, 9):
        rmm.grouped_linear(X, W, torch.full((4,), v, dtype=torch.int32, device="cuda"), out=out)
    assert (out == 3).all()


def test_nan_and_infinity_stay_in_their_rows():
    """A NaN or infinity in one row of X (or in its scale) does not reach its neighbours,
    and NaN in another group's weights is not seen."""
    n, d, m = 48, 256, 256
    X = torch.ones((n, d), dtype=torch.bfloat16, device="cuda")
    X[7, 3], X[20, 100] = float("nan"), float("inf")
    W = torch.ones((3, d, m), dtype=torch.bfloat16, device="cuda")
    W[1] = float("nan")
    off = torch.tensor([0, 30, 30, 48], dtype=torch.int32, device="cuda")
    good = [i for i in range(n) if i not in (7, 20)]
    Y = rmm.grouped_linear(X, W, off)
    assert (Y[good] == d).all() and Y[7].isnan().all() and Y[20].isinf().all()
    q, s = rmm.quantize_fp8(X)
    wq, sw = rmm.quantize_fp8_weight(W)
    Y = rmm.grouped_linear_fp8(q, s, wq, sw, off)
    assert (Y[good].float() - d).abs().max() <= 1 and Y[7].isnan().all() and Y[20].isnan().all()


def test_refused_shapes_and_layouts():
    dev = "cuda"
    X = torch.zeros((8, 64), dtype=torch.bfloat16, device=dev)
    W = torch.zeros((2, 64, 64), dtype=torch.bfloat16, device=dev)
    off = torch.zeros(3, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="offsets"):
        rmm.grouped_linear(X, W, off[:2])
    with pytest.raises(TypeError, match="int32"):
        rmm.grouped_linear(X, W, off.long())
    with pytest.raises(ValueError, match="contraction"):
        rmm.grouped_linear(X[:, :32], W, off)
    with pytest.raises(ValueError, match="unit column stride"):
        rmm.grouped_linear(X, W.transpose(1, 2), off)
    with pytest.raises(rmm.RMMError, match="multiples"):
        rmm.grouped_linear(torch.zeros((8, 68), dtype=torch.bfloat16, device=dev)[:, :64], W, off)
    with pytest.raises(ValueError, match="out must be"):
        rmm.grouped_linear(X, W, off, out=X[:4])
    q, s = rmm.quantize_fp8(X)
    wq, sw = rmm.quantize_fp8_weight(W)
    with pytest.raises(ValueError, match="x_scale"):
        rmm.linear_fp8(q, s.t(), wq[0], sw[0])
    with pytest.raises(TypeError, match="float8"):
        rmm.linear_fp8(X, s, wq[0], sw[0])
    with pytest.raises(ValueError, match="w_scale"):
        rmm.linear_fp8(q, s, wq[0], sw[:, 0])
    with pytest.raises(TypeError, match="CUDA tensor"):
        rmm.grouped_linear(X, W, off.cpu())
    with pytest.raises(ValueError, match="3 dimensions"):
        rmm.grouped_linear(X, W[0], off)


def test_one_block_scales_as_torch_lays_them_out():
    """Scales of a single block, whose row stride torch may give as anything."""
    g = synthetic.rng(75)
    X = synthetic.to_bf16(g.standard_normal((40, 100)))
    W = synthetic.to_bf16(g.standard_normal((100, 200)))
    q, s = rmm.quantize_fp8(padded(X, 8))
    wq, sw = rmm.quantize_fp8_weight(padded(W, 8))
    Y = rmm.linear_fp8(q, s, wq, sw)
    turned = s.clone().t().contiguous().t().contiguous()  # [1, 40] with strides (1, 1)
    assert torch.equal(rmm.linear_fp8(q, turned, wq, sw), Y)
    one = rmm.linear_fp8(q[7:8], s[:, 7:8], wq, sw)        # one row of a wider batch
    assert torch.equal(one[0], Y[7])


# ------------------------------------------------------------------ together, as they are used
def test_moe_block_in_fp8_and_captured():
    """The experts' gate, up and down projections of a small mixture-of-experts block:
    bf16 and fp8, the fp8 run captured in a graph on a side stream and replayed on
    other inputs and other group sizes, equal bit for bit to eager calls."""
    g = synthetic.rng(66)
    n, d, f, E = 96, 512, 768, 6
    Wg, Wu, Wd = (synthetic.to_bf16(g.standard_normal((E, a, b)) / np.sqrt(a)).cuda()
                  for a, b in ((d, f), (d, f), (f, d)))
    q = [rmm.quantize_fp8_weight(w) for w in (Wg, Wu, Wd)]

    def inputs(seed):
        r = synthetic.rng(seed)
        cuts = np.sort(r.integers(0, n + 1, E - 1))
        return (synthetic.to_bf16(synthetic.outlier_activations(r, n, d, 0.5)).cuda(),
                torch.tensor(np.concatenate([[0], cuts, [n]]), dtype=torch.int32, device="cuda"))

    def fp8(X, off):
        xq, sx = rmm.quantize_fp8(X)
        h = torch.nn.functional.silu(rmm.grouped_linear_fp8(xq, sx, *q[0], off)) * \
            rmm.grouped_linear_fp8(xq, sx, *q[1], off)
        hq, sh = rmm.quantize_fp8(h)
        return rmm.grouped_linear_fp8(hq, sh, *q[2], off)

    def bf16(X, off):
        h = torch.nn.functional.silu(rmm.grouped_linear(X, Wg, off)) * rmm.grouped_linear(X, Wu, off)
        return rmm.grouped_linear(h, Wd, off)

    X, off = inputs(1)
    Xf, bounds = X.double(), off.tolist()
    ref = torch.empty((n, d), dtype=torch.float64, device="cuda")
    for e in range(E):
        x = Xf[bounds[e]:bounds[e + 1]]
        ref[bounds[e]:bounds[e + 1]] = (torch.nn.functional.silu(x @ Wg[e].double()) * (x @ Wu[e].double())) @ Wd[e].double()
    rel = lambda y: ((y.double() - ref).norm() / ref.norm()).item()  # noqa: E731
    # bf16: a handful of roundings of 2^-8; e4m3: operands off by at most 2^-4 each, independent errors
    assert rel(bf16(X, off)) <= 2.0 ** -6
    assert rel(fp8(X, off)) <= 4 * 2.0 ** -4

    eager = [fp8(*inputs(s)) for s in (1, 2, 3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8(X, off)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        Y = fp8(X, off)
    for s in (1, 2, 3, 1):
        Xs, offs = inputs(s)
        X.copy_(Xs)
        off.copy_(offs)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, eager[s - 1])
    del graph


@pytest.mark.parametrize("fp8", [False, True])
def test_large_tiles_captured(fp8):
    """The CTA-pair tiles in a graph: a replay on other rows, other group bounds and (fp8)
    other scales, all written by kernels just before it, equals an eager call."""
    g = synthetic.rng(69)
    n, d, m, E = 700, 256, 2600, 2
    W = synthetic.to_bf16(g.standard_normal((E, d, m)) / 16).cuda()
    wq, sw = rmm.quantize_fp8_weight(W)
    X = torch.empty((n, d), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 300, n], dtype=torch.int32, device="cuda")
    out = torch.zeros((n, m), dtype=torch.bfloat16, device="cuda")

    def call(out=None):
        if fp8:
            return rmm.grouped_linear_fp8(*rmm.quantize_fp8(X), wq, sw, off, out=out)
        return rmm.grouped_linear(X, W, off, out=out)

    inputs = [(synthetic.to_bf16(4.0 ** k * g.standard_normal((n, d))).cuda(), 100 + 211 * k) for k in range(3)]
    eager = []
    for x, cut in inputs:
        X.copy_(x)
        off[1] = cut
        eager.append(call())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for k in (0, 1, 2, 1):
        X.copy_(inputs[k][0])
        off[1] = inputs[k][1]
        out.zero_()
        graph.replay()
        assert torch.equal(out, eager[k])
    del graph


# (rows of the groups, d, m) of tiles of 128 x 256 in bf16 (41 to 64 rows an average group,
# tiles that about fill a wave) and 32 x 512 in e4m3 with more than 32 rows a group
MEDIUM = [
    ([128, 60, 0, 1, 33, 31, 100, 64, 17, 16], 200, 3500),   # 140 tiles of 128 x 256
    ([300, 1, 0, 129, 40, 2, 8, 65, 20, 10, 31, 32], 330, 2900),  # 144, a group of three row tiles
    ([62, 0, 90, 33, 1, 47], 136, 6100),                     # e4m3 32 x 512
    ([40, 33, 38, 0, 70, 32, 39, 36], 260, 2100),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("sizes,d,m", MEDIUM, ids=str)
def test_medium_groups(sizes, d, m, fp8):
    test_every_tile_shape(sizes, d, m, fp8)


def test_two_streams_at_once():
    """Calls on two streams share nothing: interleaved results equal those of calls alone."""
    dev, _, _ = fp8_operands(67, 200, 512, 1024, 4)
    off = torch.tensor([0, 50, 60, 130, 200], dtype=torch.int32, device="cuda")
    g = synthetic.rng(68)
    X = synthetic.to_bf16(g.standard_normal((300, 512))).cuda()
    W = synthetic.to_bf16(g.standard_normal((4, 512, 512))).cuda()
    args = (dev["xq"], dev["sx"], dev["wq"], dev["sw"], off)
    a, b = rmm.grouped_linear_fp8(*args), rmm.grouped_linear(X[:200], W, off)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            got.append((rmm.grouped_linear_fp8(*args), a))
        with torch.cuda.stream(s2):
            got.append((rmm.grouped_linear(X[:200], W, off), b))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)


@pytest.mark.parametrize("rows,d,m", [(6, 128, 6400), (256, 128, 2560)])
def test_threads_with_other_group_counts(rows, d, m):
    """Host threads whose calls have few and many groups (whose bounds take more of a
    kernel's shared memory) at once: none is refused, each result is that of a call alone."""
    import threading

    g = torch.Generator(device="cuda").manual_seed(76)
    calls = []
    for E in (3, 300):
        n = rows * E
        X = torch.randn((n, d), generator=g, device="cuda").bfloat16()
        W = torch.randn((E, d, m), generator=g, device="cuda").bfloat16()
        off = torch.arange(0, n + 1, rows, dtype=torch.int32, device="cuda")
        args = (*rmm.quantize_fp8(X), *rmm.quantize_fp8_weight(W), off)
        calls += [(rmm.grouped_linear, (X, W, off)), (rmm.grouped_linear_fp8, args)]
    alone = [f(*a) for f, a in calls]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        f, a = calls[i]
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                out = torch.empty_like(alone[i])
                for _ in range(100):
                    f(*a, out=out)
                torch.cuda.current_stream().synchronize()
                assert torch.equal(out, alone[i])
        except Exception as e:  # noqa: BLE001
            failed.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
