"""The 4-bit paged cache in plain numpy, from its definition (Z, U, N of
include/cachegen.h): one token, one channel at a time as index arithmetic, no
tensor-core orders. Quantisation steps in binary32 as the definition has
them; attention in binary64, with a bound on what the kernels may be off."""
import numpy as np


def to16(x, bf16):
    """binary32 -> 16-bit pattern, nearest even."""
    x = np.asarray(x, np.float32)
    if not bf16:
        with np.errstate(over="ignore"):
            return x.astype(np.float16).view(np.uint16)
    b = x.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def from16(b, bf16):
    b = np.asarray(b, np.uint16)
    if not bf16:
        return b.view(np.float16).astype(np.float32)
    return (b.astype(np.uint32) << 16).view(np.float32)


def quantise(x, group, bf16):
    """x binary32 [..., D] -> (codes [..., D] int, params uint16 [..., D/group, 2])."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        m, M = g.min(-1, keepdims=True), g.max(-1, keepdims=True)  # NaNs carry over
        span = M - m
        s = ((span / np.float32(15)).view(np.uint32) + np.uint32(0x10000)) & np.uint32(0xFFFE0000)
        s = from16(to16(s.view(np.float32), bf16), bf16)
        c = np.where(s > 0, np.clip(np.rint((g - m) / np.where(s > 0, s, np.float32(1))), 0, 15), 0)
    bad = ~np.isfinite(span)
    s, m, c = np.where(bad, np.float32(np.nan), s), np.where(bad, np.float32(np.nan), m), np.where(bad, 0, c)
    return c.astype(np.int64).reshape(x.shape), np.concatenate([to16(s, bf16), to16(m, bf16)], -1)


def values(codes, params, group, bf16):
    """U in binary32 (s c is exact in it, one rounding)."""
    p = from16(params, bf16)
    c = codes.reshape(*codes.shape[:-1], -1, group).astype(np.float32)
    return (c * p[..., :1] + p[..., 1:]).astype(np.float32).reshape(codes.shape)


class Layout:
    def __init__(self, L, pages, P, H, D, group):
        self.L, self.pages, self.P, self.H, self.D, self.group = L, pages, P, H, D, group
        self.ng = D // group
        self.record = 16 * D + 128 * self.ng
        self.nbytes = L * pages * H * (P // 16) * self.record

    def rec(self, layer, page, head, slot):
        return (((layer * self.pages + page) * self.H + head) * (self.P // 16) + slot // 16) * self.record

    def k_nibbles(self, slot):
        """Byte and shift of each channel's K code of a token at `slot`, from the record's start."""
        d, D, tok = np.arange(self.D), self.D, slot % 16
        w, jj, t, eh, el = d // 32, d // 16 % 2, d % 16 // 4, d % 4 // 2, d % 2
        n = 4 * el + 2 * jj + eh
        return tok * D // 2 + t * (D // 8) + 4 * w + n // 2, 4 * (n % 2)

    def v_nibbles(self, slot):
        d, D, tok = np.arange(self.D), self.D, slot % 16
        g, i = d // (D // 8), d % (D // 8)
        return 8 * D + tok // 8 * 4 * D + ((g * 4 + tok % 8 // 2) * 2 + tok % 2) * (D // 16) + i // 2, 4 * (i % 2)

    def params(self, slot, v):
        return 16 * self.D + (64 * self.ng if v else 0) + (slot % 16) * 4 * self.ng

    def put(self, pool, layer, page, head, slot, v, codes, params):
        at, sh = (self.v_nibbles if v else self.k_nibbles)(slot)
        base = self.rec(layer, page, head, slot)
        pool[base + at] = 0
        np.bitwise_or.at(pool, base + at, (np.asarray(codes) << sh).astype(np.uint8))
        pool[base + self.params(slot, v):][:4 * self.ng] = np.ascontiguousarray(params).reshape(-1).view(np.uint8)

    def get(self, pool, layer, page, head, slot, v):
        at, sh = (self.v_nibbles if v else self.k_nibbles)(slot)
        base = self.rec(layer, page, head, slot)
        p = pool[base + self.params(slot, v):][:4 * self.ng].copy().view(np.uint16).reshape(self.ng, 2)
        return (pool[base + at].astype(np.int64) >> sh) & 15, p


def attention(q, k, v, pos, window, scale, params_k, out_step, codes_step=0.0):
    """One query head's row: q [D], k, v [n, D] (binary64 values of U),
    params_k [n, D]: an upper bound of the terms s c and |m| of each k; pos: the row's
    position. -> (out [D], lse, bound of |out - kernel's|, bound of |lse - kernel's|).

    The bound counts roundings. h = 2^-11 is half a step of binary16, the
    type of the tensor cores' operands; u = 2^-24 of binary32.
    - scores: q is exact (a power of two away from binary16) but for 2^-25 of its
      row's largest, products are exact or round within u, and D + 16 terms are added:
      dS <= scale * ((D + 16) * 4u * sum_d |q_d| t_d + 2^-24 max|q| * sum_d t_d)
      with t_d the larger terms; adding and exponent: 8u |S|.
    - weights: e^dS, exp2 and its argument 2^-21, one rounding to binary16 (h, and 2^-25
      of the largest where that is subnormal), one of the value or its scale (h): the
      output is off by at most sum_j p_j |v_j| (2 dS + 2h + 2^-19) + 2^-24 n max|t|.
    - the sum of the weights is binary32's: dS + 2^-20 on lse, relative to 1.
    - the output's own rounding: out_step.
    """
    j = np.arange(len(k))
    seen = (j <= pos) & ((j > pos - window) if window else True)
    D = q.shape[0]
    if not seen.any():
        return np.zeros(D), -np.inf, np.zeros(D), 0.0
    k, v, t = k[seen], v[seen], params_k[seen]
    s = scale * (k @ q)
    top = s.max()
    p = np.exp(s - top)
    total = p.sum()
    out, lse = p @ v / total, top + np.log(total)
    u, h = 2.0 ** -24, 2.0 ** -11
    ds = abs(scale) * ((D + 16) * 4 * u * (t @ np.abs(q)) + 2.0 ** -24 * np.abs(q).max() * t.sum(1)).max() + 8 * u * np.abs(s).max()
    bound = (p @ np.abs(v) / total) * (2 * ds + 2 * h + 2.0 ** -19) + 2.0 ** -24 * len(k) * np.nanmax(np.abs(v)) / total
    bound = bound * (1 + out_step) + out_step * np.abs(out) + 2.0 ** -25
    return out, lse, bound, ds + 2.0 ** -20 + 2.0 ** -23 * abs(lse)
