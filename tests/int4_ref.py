"""INT4 tensors with group scales for tests: random row-major parts, their exact fp64 values, the
packed layout written out element by element, and the error that a product may have.

A product sums K terms t_k = s (16 + q) x and takes away (16 + z) s sum x (or forms s (q - z) x);
its fp32 roundings are relative to partial sums and of independent sign, so they add up to about
2^-24 sqrt(K) of the 2-norm of all terms (both kinds: s (16 + q + 16 + z) x); eight times that is
allowed. Where the weights or activations are rounded to a half's 11 bits first (2^-11 relative
each, `half` roundings), eight times 2^-11 / sqrt(3) of the 2-norm of the products are added."""
import numpy as np
import torch

import bit_quantized_moe_dequant_amd as mq

FMTS = [mq.FMT_INT4_G32, mq.FMT_INT4_G64, mq.FMT_INT4_G128, mq.FMT_INT4Z_G32, mq.FMT_INT4Z_G64, mq.FMT_INT4Z_G128]


def group_of(fmt):
    return 32 << ((fmt - mq.FMT_INT4_G32) % 3)


class Parts:
    """Row-major codes, scales and zero points of n tensors; values() their fp64 matrices."""

    def __init__(self, fmt, n, rows, cols, seed, scale="bf16", spread=0.0, zmax=15):
        g = np.random.default_rng(seed)
        self.fmt, self.n, self.rows, self.cols, self.group = fmt, n, rows, cols, group_of(fmt)
        self.q = g.integers(0, 16, (n, rows, cols), dtype=np.uint8)
        shape = (n, rows, cols // self.group)
        s = (0.5 + g.random(shape)) * np.exp2(spread * g.standard_normal(shape)) / (4.6 * np.sqrt(cols))
        s *= np.where(g.random(shape) < 0.1, -1.0, 1.0)
        self.st = torch.from_numpy(s).to(torch.bfloat16 if scale == "bf16" else torch.float16)
        self.z = g.integers(0, zmax + 1, shape, dtype=np.uint8) if fmt >= mq.FMT_INT4Z_G32 else None

    @property
    def s(self):
        return self.st.double().numpy()

    def codes(self):
        return torch.from_numpy(self.q[..., 0::2] | (self.q[..., 1::2] << 4))

    def wide(self, a):
        return np.repeat(np.asarray(a, dtype=np.float64), self.group, axis=-1)

    def values(self, e=0):
        z = 8.0 if self.z is None else self.wide(self.z[e])
        return (self.q[e].astype(np.float64) - z) * self.wide(self.s[e])

    def pack(self):
        z = None if self.z is None else torch.from_numpy(self.z).cuda()
        return mq.pack_int4(self.codes().cuda(), self.st.cuda(), z)

    def tol(self, x, e=0, half=0):
        """[T, rows] bound of the error of x W^T (x fp64 [T, cols])."""
        z = 8.0 if self.z is None else self.wide(self.z[e])
        s2, x2 = self.wide(self.s[e]) ** 2, np.asarray(x, dtype=np.float64) ** 2
        t = x2 @ (s2 * (32.0 + self.q[e] + z) ** 2).T
        out = 8 * 2.0 ** -24 * np.sqrt(self.cols) * np.sqrt(t)
        if half:
            out += half * 8 * 2.0 ** -11 / np.sqrt(3) * np.sqrt(x2 @ (self.values(e) ** 2).T)
        return out + 1e-37


def packed_reference(p: Parts, e, exponent):
    """(data, scales) planes of tensor e with scales times 2^-exponent, element by element."""
    per, rt, kt = 128 // p.group, -(-p.rows // 16), -(-p.cols // 128)
    data = np.zeros((rt * kt, 64, 4), np.uint32)
    scales, zeros = np.zeros((rt * kt, 16, per), np.uint16), np.full((rt * kt, 16, per), 8, np.uint8)
    for r in range(p.rows):
        for k in range(p.cols):
            tile, c = (r // 16) * kt + k // 128, k % 128
            lane, j, i = r % 16 + 16 * (c % 32 // 8), c // 32, c % 8
            data[tile, lane, j] |= np.uint32(int(p.q[e, r, k]) << (4 * (i // 2) + 16 * (i % 2)))
        for b in range(p.cols // p.group):
            tile, at = (r // 16) * kt + b // per, b % per
            scales[tile, r % 16, at] = np.float16(np.ldexp(p.s[e, r, b], -exponent)).view(np.uint16)
            if p.z is not None:
                zeros[tile, r % 16, at] = p.z[e, r, b]
    side = scales.tobytes() + (zeros.tobytes() if p.z is not None else b"")
    return np.frombuffer(data.tobytes(), np.uint8), np.frombuffer(side, np.uint8)


def bf16(a):
    """A numpy array as a bf16 tensor on the GPU and its exact values."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()
