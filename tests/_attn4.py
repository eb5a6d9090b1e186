"""Reference for 4-bit caches and rotated appends: the definitions of
include/spec_attn.h, quantisation in float64 and rotation in 32 bits, operation
by operation (numpy, on the CPU)."""
import math

import numpy as np
import torch

from tests import _attn
from tests._attn import E4M3_MAX, EXP_MIN, World

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 16
FOUR = torch.float4_e2m1fn_x2
_E4M3 = _attn.e4m3_value(np.arange(127, dtype=np.uint8))


def nearest_code(values, y):
    """Index of the value nearest to each y >= 0, ties to the even index, the largest beyond it."""
    hi = np.searchsorted(values, y, side="left").clip(0, len(values) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = y - values[lo], values[hi] - y
    c = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(y >= values[-1], len(values) - 1, np.where(values[hi] == y, hi, c))


def quantise4(x):
    """float64 vectors [..., D] -> (bytes of codes [..., D / 2], scales as e4m3 codes [..., D / 16], exponent bytes)."""
    flat = x.reshape(-1, x.shape[-1])
    n, d = flat.shape
    codes, block, scale = np.zeros((n, d // 2), np.uint8), np.zeros((n, d // BLOCK), np.uint8), np.zeros(n, np.uint8)
    for i, v in enumerate(flat):
        if not np.isfinite(v).all():
            block[i], scale[i] = 0x7f, 255
            continue
        top = np.abs(v).max()
        m, e = math.frexp(top / (6 * E4M3_MAX))
        e = EXP_MIN if top == 0 else max(EXP_MIN, e - (m == 0.5))
        y = (v * 2.0 ** -e).reshape(-1, BLOCK)
        block[i] = nearest_code(_E4M3, np.abs(y).max(-1) / 6)
        s = _E4M3[block[i]][:, None]
        c = nearest_code(E2M1, np.abs(y) / np.where(s > 0, s, 1)) * (s > 0) + 8 * np.signbit(y)
        c = c.reshape(-1)
        codes[i], scale[i] = c[::2] | c[1::2] << 4, e + 127
    return codes.reshape(*x.shape[:-1], d // 2), block.reshape(*x.shape[:-1], d // BLOCK), scale.reshape(x.shape[:-1])


def values4(codes, block, scale):
    """float64 values of what quantise4 gives."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    x = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7] * np.repeat(_attn.e4m3_value(block), BLOCK, -1)
    return np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))[..., None] * x


def attention(q, k, v, scale, seen):
    """tests/_attn.py's, with the bounds that weights in f16 need: a weight below 2^-14 of the
    reference is off by up to half of f16's least step, 2^-25 of the reference, which a row's
    largest weight times its vector's 2^e reaches.  In units of 2^e a cached vector's elements
    are at most its largest, so the error of column d is at most
        2^-25 * max_j(p_j 2^e_j) * sum_j |v_jd| / 2^e_j
    (where a token dominates a row but holds 0 in column d, that is all there is to see).  e_j is
    not kept here: with L the format's largest value (448 or 2688) the vector's largest element is
    above L / 2 * 2^e before it is quantised and at most L * 2^e * 17 / 16 in the cache, and at
    least 15 / 16 of the former there, so max_j(p_j max|v_j|) * sum_j |v_jd| / max|v_j| is at least
    15 / 34 of that product: the factor below is 2^-23."""
    out, lse, tol, tol_lse = _attn.attention(q, k, v, scale, seen)
    group = q.shape[1] // k.shape[1]
    top = np.abs(v).max(-1)                                   # [L, hkv]
    with np.errstate(invalid="ignore", divide="ignore"):
        share = np.where(top[..., None] > 0, np.abs(v) / top[..., None], 0)
    for i, n in enumerate(seen):
        for h in range(q.shape[1] if n > 0 else 0):
            p = np.exp(scale * (k[:n, h // group] @ q[i, h]) - lse[i, h])
            tol[i, h] += 2.0 ** -23 * (p * top[:n, h // group]).max() * share[:n, h // group].sum(0)
    return out, lse, tol, tol_lse


class World4(World):
    """A World whose pool holds 4-bit codes; unused slots hold arbitrary codes and exponents with NaN scales."""

    def __init__(self, new, old, hq, hkv, d, page, seed=0, **kw):
        super().__init__(new, old, hq, hkv, d, page, torch.bfloat16, seed=seed, **kw)
        g = np.random.default_rng(seed + 1000)
        shape = (self.num_pages, hkv, page)
        self.raw = {}
        for name, cached in (("k", self.kc), ("v", self.vc)):
            codes = g.integers(0, 256, (*shape, d // 2)).astype(np.uint8)
            block = np.full((*shape, d // BLOCK), 0x7f, np.uint8)
            scale = g.integers(0, 256, shape).astype(np.uint8)
            for b, x in enumerate(cached):
                if len(x) == 0:
                    continue
                c, s, e = quantise4(x)
                x[:] = values4(c, s, e)
                for p in range(len(x)):
                    at = (self.table[b, p // page], slice(None), p % page)
                    codes[at], block[at], scale[at] = c[p], s[p], e[p]
            self.raw[name], self.raw[name + "_block"], self.raw[name + "_scale"] = (torch.from_numpy(t) for t in (codes, block, scale))

    def expect_attention(self, causal=True, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        parts = []
        for b, n in enumerate(self.new):
            q = self.q[self.cu[b]:self.cu[b + 1]].double().numpy()
            seen = [min(self.kv[b], self.kv[b] - n + i + 1) if causal else self.kv[b] for i in range(n)]
            parts.append(attention(q, self.kc[b], self.vc[b], scale, seen))
        return [np.concatenate([p[i] for p in parts]) for i in range(4)]

    def pool(self, lib):
        """A KVPool on the GPU, and cu, kv_len, page_table."""
        r = {name: t.cuda() for name, t in self.raw.items()}
        e4m3 = torch.float8_e4m3fn
        pool = lib.KVPool(r["k"].view(FOUR), r["v"].view(FOUR), r["k_scale"], r["v_scale"], r["k_block"].view(e4m3), r["v_block"].view(e4m3))
        return pool, tuple(torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (self.cu, np.array(self.kv, np.int32), self.table))


def bytes_of(pool):
    return {name: getattr(pool, name).view(torch.uint8).cpu() for name in ("k", "v", "k_scale", "v_scale", "k_block", "v_block")}


def rope_table(positions, rot, theta=10000.0):
    """[positions, rot] float32: cosines, then sines."""
    angle = np.arange(positions)[:, None] * theta ** -(np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))


def rotate(x, table, pos, interleaved):
    """x [n, heads, D] float32 (numpy), turned by rows pos of the table; every operation rounded to 32 bits."""
    rot = table.shape[1]
    c, s = (table.numpy()[pos][:, None, i * (rot // 2):(i + 1) * (rot // 2)] for i in range(2))
    out = x.copy()
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., i], x[..., j]
    with np.errstate(invalid="ignore", over="ignore"):
        out[..., i] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
        out[..., j] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return out
