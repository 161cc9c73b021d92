"""Cases of the grouped and fp8 products by the tile that the library takes for them, shared by the CPU test of
that choice and the GPU tests of the kernels, and their operands with 64-bit references.

A tile is (rows of X, columns of W, CTAs that share its contraction).  On 148 SMs.
"""
import ctypes
import zlib

import torch

import input_adaptive_reduced_colnorm_b200 as rmm

BF16, E4M3 = 0, 1
SMS = 148

# (type, rows of the groups, d, m, tile): every kernel and every split that the choice of tiles reaches
CASES = [
    # 32 x 128, alone and over clusters of 2, 4 and 8
    (BF16, [20], 300, 18000, (32, 128, 1)),
    (BF16, [7], 130, 9000, (32, 128, 2)),
    (BF16, [20], 2000, 4200, (32, 128, 4)),
    (BF16, [9, 0, 30, 1], 2100, 300, (32, 128, 8)),
    (E4M3, [20], 300, 18000, (32, 128, 1)),
    (E4M3, [7], 260, 9000, (32, 128, 2)),
    (E4M3, [20], 2000, 1522, (32, 128, 4)),
    (E4M3, [9, 0, 30, 1], 4200, 300, (32, 128, 8)),
    # 16 x 256, two CTAs per SM
    (BF16, [3, 0, 16, 1, 17, 9], 300, 8200, (16, 256, 1)),
    (BF16, [5], 200, 20000, (16, 256, 2)),
    (E4M3, [3, 0, 16, 1, 17, 9], 300, 8200, (16, 256, 1)),
    (E4M3, [5], 1000, 20000, (16, 256, 2)),
    (E4M3, [1], 2176, 14336, (16, 256, 4)),
    (E4M3, [13], 2176, 14336, (16, 256, 4)),
    # bf16 32 x 256, e4m3 32 x 512
    (BF16, [30, 1, 33, 32, 0, 16, 40, 31], 200, 2600, (32, 256, 1)),
    (E4M3, [40, 1, 33, 32, 0, 36, 40, 31] * 2, 300, 6000, (32, 512, 1)),
    (E4M3, [20], 1000, 20000, (32, 512, 2)),
    (E4M3, [20], 2200, 12000, (32, 512, 4)),
    (E4M3, [37], 2200, 9000, (32, 512, 2)),
    # bf16 128 x 256 on one CTA
    (BF16, [128, 60, 0, 1, 33, 31, 100, 64, 17, 16], 200, 3500, (128, 256, 1)),
    # 64 x 256
    (BF16, [64, 70, 0, 1, 63, 40, 65, 64, 50, 60], 264, 4100, (64, 256, 1)),
    (BF16, [200], 600, 2900, (64, 256, 2)),
    (E4M3, [64, 70, 0, 1, 63, 40, 65, 64, 50, 60], 264, 4100, (64, 256, 1)),
    (E4M3, [200], 1000, 2900, (64, 256, 2)),
    (E4M3, [64], 2200, 5000, (64, 256, 4)),
    (E4M3, [50], 2200, 5000, (64, 256, 4)),
    # bf16 256 x 256 on CTA pairs
    (BF16, [150, 20, 300], 1030, 8100, (256, 256, 1)),
    # e4m3 128 x 256, rows on the lanes: fewer than 32 blocks of 128, and on either side of 32, 64 and 96
    (E4M3, [1030], 72, 5000, (128, 256, 1)),
    (E4M3, [150, 20, 300], 4300, 4100, (128, 256, 1)),
    (E4M3, [300], 4096, 5120, (128, 256, 1)),
    (E4M3, [300], 4100, 5120, (128, 256, 1)),
    (E4M3, [150, 20, 300], 8192, 4100, (128, 256, 1)),
    (E4M3, [150, 20, 300], 8400, 4100, (128, 256, 1)),
    (E4M3, [300], 12288, 5120, (128, 256, 1)),
    (E4M3, [300], 12400, 5120, (128, 256, 1)),
]

GROUPED = [c for c in CASES if len(c[1]) > 1]  # tiles hold rows of other groups

# the same tiles, every CTA with more blocks of the contraction than a kernel has stages
LONG = [
    (BF16, [20], 2100, 18000, (32, 128, 1)),
    (BF16, [7], 2100, 9000, (32, 128, 2)),
    (BF16, [20], 4200, 4200, (32, 128, 4)),
    (BF16, [9, 0, 30, 1], 6100, 300, (32, 128, 8)),
    (E4M3, [20], 2048, 18000, (32, 128, 1)),
    (E4M3, [7], 2560, 9000, (32, 128, 2)),
    (E4M3, [20], 4800, 4200, (32, 128, 4)),
    (E4M3, [9, 0, 30, 1], 9300, 300, (32, 128, 8)),
    (BF16, [3, 0, 16, 1, 17, 9], 2100, 8200, (16, 256, 1)),
    (BF16, [5], 2100, 20000, (16, 256, 2)),
    (E4M3, [3, 0, 16, 1, 17, 9], 2100, 8200, (16, 256, 1)),
    (E4M3, [5], 2100, 20000, (16, 256, 2)),
    (E4M3, [13], 2176, 14336, (16, 256, 4)),
    (BF16, [30, 1, 33, 32, 0, 16, 40, 31], 2100, 2600, (32, 256, 1)),
    (E4M3, [40, 1, 33, 32, 0, 36, 40, 31] * 2, 2100, 6000, (32, 512, 1)),
    (E4M3, [20], 2100, 20000, (32, 512, 2)),
    (E4M3, [20], 2200, 12000, (32, 512, 4)),
    (BF16, [128, 60, 0, 1, 33, 31, 100, 64, 17, 16], 2100, 3500, (128, 256, 1)),
    (BF16, [64, 70, 0, 1, 63, 40, 65, 64, 50, 60], 2100, 4100, (64, 256, 1)),
    (BF16, [200], 2100, 2900, (64, 256, 2)),
    (E4M3, [64, 70, 0, 1, 63, 40, 65, 64, 50, 60], 2100, 4100, (64, 256, 1)),
    (E4M3, [200], 2100, 2900, (64, 256, 2)),
    (E4M3, [64], 3200, 5000, (64, 256, 4)),
    (BF16, [150, 20, 300], 2100, 8100, (256, 256, 1)),
    (E4M3, [150, 20, 300], 2100, 4100, (128, 256, 1)),
]


def case_id(c):
    return f"{'e4m3' if c[0] else 'bf16'}-{'x'.join(map(str, c[4]))}-{sum(c[1])}of{len(c[1])}-{c[2]}x{c[3]}"


def plan(dtype, n, d, m, groups, sms=SMS):
    out = (ctypes.c_int32 * 3)()
    assert rmm.lib().rmm_debug_grouped_plan(dtype, n, d, m, groups, sms, ctypes.cast(out, ctypes.c_void_p)) == 0
    return tuple(out)


def wider(shape, unit, dtype):
    """A matrix in a buffer of NaN whose rows are one unit longer than they need; of a batch, one row longer too."""
    ld = -(-shape[-1] // unit) * unit + unit
    rows = (*shape[:-2], shape[-2] + 1) if len(shape) > 2 else shape[:-1]
    buf = torch.full((*rows, ld), float("nan"), device="cuda").to(dtype)
    return buf[..., : shape[-2], : shape[-1]]


def behind_one(t):
    """t at an address that is a multiple of its element's size only."""
    return torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)


class Operands:
    """Random operands of a case: Gaussian bf16 values, or any e4m3 codes with scales that differ from block to block
    (not from a quantiser: any scales are allowed), all in buffers wider than they need; two rows before the first group and three behind the last; and
    what the formula gives for them in 64 bits."""

    def __init__(self, case):
        dtype, sizes, d, m, _ = case
        g = torch.Generator(device="cuda").manual_seed(zlib.crc32(case_id(case).encode()))
        self.dtype, self.d, self.m, self.groups = dtype, d, m, len(sizes)
        self.before, self.behind = (2, 3) if len(sizes) > 1 else (0, 0)
        self.n = sum(sizes) + self.before + self.behind
        self.bounds = [self.before]
        for s in sizes:
            self.bounds.append(self.bounds[-1] + s)
        self.off = behind_one(torch.tensor(self.bounds, dtype=torch.int32, device="cuda"))
        t, unit = (torch.float8_e4m3fn, 16) if dtype else (torch.bfloat16, 8)
        x = torch.randn((self.n, d), generator=g, device="cuda")
        w = torch.randn((self.groups, d, m), generator=g, device="cuda")
        self.X, self.W = wider(x.shape, unit, t), wider(w.shape, unit, t)
        self.X.copy_(x.clamp(-400, 400))
        self.W.copy_(w)
        if dtype:
            nb, mb = -(-d // 128), -(-m // 128)
            sx = torch.exp2(4 * torch.rand((nb, self.n + 3), generator=g, device="cuda") - 2)
            sx[:, self.n:] = float("nan")
            self.sx = behind_one(sx)[:, : self.n]
            self.sw = behind_one(torch.exp2(4 * torch.rand((self.groups, nb, mb), generator=g, device="cuda") - 2))

    def call(self, out=None):
        if self.dtype:
            return rmm.grouped_linear_fp8(self.X, self.sx, self.W, self.sw, self.off, out=out)
        return rmm.grouped_linear(self.X, self.W, self.off, out=out)

    def expire(self, out):
        """The same call with the producers' waits made to run out."""
        sx, lds, sw = (self.sx.data_ptr(), self.sx.stride(0), self.sw.data_ptr()) if self.dtype else (None, 0, None)
        return rmm.lib().rmm_debug_grouped_expire_producer(
            self.dtype, self.X.data_ptr(), self.n, self.d, self.X.stride(0), sx, lds, self.W.data_ptr(), self.groups,
            self.W.stride(0), self.m, self.W.stride(1), sw, self.off.data_ptr(), out.data_ptr(), out.stride(0),
            torch.cuda.current_stream().cuda_stream)

    def out(self, fill=3.0):
        y = wider((self.n, self.m), 8, torch.bfloat16)
        y.fill_(fill)
        return y

    def wide_x(self):
        x = self.X.float().double()
        return x * self.sx.double().t().repeat_interleave(128, 1)[:, : self.d] if self.dtype else x

    def wide_w(self, e):
        w = self.W[e].float().double()
        if self.dtype:
            w *= self.sw[e].double().repeat_interleave(128, 0)[: self.d].repeat_interleave(128, 1)[:, : self.m]
        return w

    def reference(self, fill=3.0):
        """(Y, sum_j |x_j w_j|, 0 in rows of no group)"""
        x = self.wide_x()
        Y = torch.full((self.n, self.m), fill, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(Y)
        for e in range(self.groups):
            lo, hi = self.bounds[e], self.bounds[e + 1]
            if hi > lo:
                w = self.wide_w(e)
                Y[lo:hi] = x[lo:hi] @ w
                mag[lo:hi] = x[lo:hi].abs() @ w.abs()
        return Y, mag

    def check(self, Y, ref, mag, rows=None):
        """d terms (and the scales' products) summed in fp32, each step off by at most 2^-23 of its value, then one
        rounding to bf16, off by at most 2^-8."""
        E = (self.d + 4) * 2.0 ** -23 * mag
        bad = ~((Y.double() - ref).abs() <= torch.where(mag > 0, 2.0 ** -8 * (ref.abs() + E) + E, 0.0))
        if rows is not None:
            bad = bad[rows]
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[:5].tolist()}"
