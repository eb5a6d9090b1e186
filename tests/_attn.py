"""Reference for the cache and attention tests: the definitions of
include/spec_attn.h in float64 (numpy, on the CPU), written position by position."""
import math

import numpy as np
import torch

E4M3_MAX, EXP_MIN = 448.0, -120


def e4m3_value(code):
    """Value of every e4m3 code (uint8 array) from the format's definition."""
    code = code.astype(np.int64)
    sign, e, m = np.where(code & 0x80, -1.0, 1.0), (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where((code & 0x7f) == 0x7f, np.nan, sign * v)


_POSITIVE = e4m3_value(np.arange(127, dtype=np.uint8))


def quantise(x):
    """float64 vectors [..., D] -> (codes, scale bytes), nearest value with ties to the even code."""
    flat = x.reshape(-1, x.shape[-1])
    codes, scale = np.zeros(flat.shape, np.uint8), np.zeros(len(flat), np.uint8)
    for i, v in enumerate(flat):
        if not np.isfinite(v).all():
            codes[i], scale[i] = 0x7f, 255
            continue
        top = np.abs(v).max()
        e = EXP_MIN if top == 0 else max(EXP_MIN, math.frexp(top / E4M3_MAX)[1] - (math.frexp(top / E4M3_MAX)[0] == 0.5))
        y = np.abs(v) * 2.0 ** -e
        hi = np.searchsorted(_POSITIVE, y, side="left").clip(0, 126)
        lo = np.maximum(hi - 1, 0)
        dl, dh = y - _POSITIVE[lo], _POSITIVE[hi] - y
        c = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
        c = np.where(_POSITIVE[hi] == y, hi, c)
        codes[i], scale[i] = c | np.where(np.signbit(v), 0x80, 0), e + 127
    return codes.reshape(x.shape), scale.reshape(x.shape[:-1])


def attention(q, k, v, scale, seen):
    """q [n, hq, D], k and v [L, hkv, D] float64; row i sees keys 0 .. seen[i]-1.
    Returns out, lse, and the bounds their errors are held to."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    spread, reach = np.zeros((n, hq, d)), np.zeros((n, hq))
    for i in range(n):
        if seen[i] <= 0:
            continue
        for h in range(hq):
            kk, vv = k[:seen[i], h // group], v[:seen[i], h // group]
            s = scale * (kk @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            out[i, h], lse[i, h] = p @ vv / l, m + np.log(l)
            spread[i, h] = p @ np.abs(vv) / l
            reach[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    # The output is rounded to bf16 (relative 2^-9) and the weights to 16 bits before their product
    # with the values (at most 2^-9 of sum p|v|); 2^-9 of that sum is left for the rest (the scores' 32-bit
    # sums, exponentials, the accumulation).  A score is a 32-bit sum of D <= 128 exact products: its error
    # is at most 128 * 2^-23 of the sum of their magnitudes, and the log of the sum moves by no more.
    return out, lse, 2.0 ** -9 * np.abs(out) + 2.0 ** -8 * spread + 1e-30, 2.0 ** -16 * (1 + reach)


class World:
    """A pool with a shuffled page table whose unused slots hold NaN (bf16) or NaN
    codes and arbitrary scale bytes, and new tokens for every sequence."""

    def __init__(self, new, old, hq, hkv, d, page, dtype, seed=0, spread=0.5, spare=3, kv_len=None, max_pages=None):
        g = np.random.default_rng(seed)
        self.new, self.hq, self.hkv, self.d, self.page, self.dtype = list(new), hq, hkv, d, page, dtype
        self.kv = [a + b for a, b in zip(new, old)] if kv_len is None else list(kv_len)
        self.n = sum(new)
        need = [-(-max(x, 0) // page) for x in self.kv]
        self.num_pages = sum(need) + spare
        order = g.permutation(self.num_pages)
        width = max(max(need, default=0), 1) if max_pages is None else max_pages
        self.table = np.zeros((len(new), width), np.int32)
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)

        def bf16(shape):
            x = torch.from_numpy((g.standard_normal(shape) * np.exp(spread * g.standard_normal(shape[:-1] + (1,)))).astype(np.float32))
            return x.bfloat16()

        self.q = bf16((self.n, hq, d))
        self.k_new, self.v_new = bf16((self.n, hkv, d)), bf16((self.n, hkv, d))
        # values of every cached token, per sequence: [kv, hkv, D] float64
        self.kc, self.vc = ([bf16((max(x, 0), hkv, d)).double().numpy() for x in self.kv] for _ in range(2))
        shape = (self.num_pages, hkv, page, d)
        self.codes, self.scales = {}, {}
        for name, cached in (("k", self.kc), ("v", self.vc)):
            if dtype == torch.bfloat16:
                pool = np.full(shape, np.nan)
                for b, x in enumerate(cached):
                    for p in range(len(x)):
                        pool[self.table[b, p // page], :, p % page] = x[p]
                self.codes[name], self.scales[name] = torch.from_numpy(pool).bfloat16(), None
            else:
                pool = np.full(shape, 0x7f, np.uint8)
                scale = g.integers(0, 256, shape[:3]).astype(np.uint8)
                for b, x in enumerate(cached):
                    c, s = quantise(x)
                    x[:] = e4m3_value(c) * 2.0 ** (s.astype(np.float64) - 127)[..., None]
                    for p in range(len(x)):
                        pool[self.table[b, p // page], :, p % page] = c[p]
                        scale[self.table[b, p // page], :, p % page] = s[p]
                self.codes[name] = torch.from_numpy(pool).view(torch.float8_e4m3fn)
                self.scales[name] = torch.from_numpy(scale)

    def to(self, device):
        """(pool tensors, cu, kv_len, page_table) on the device."""
        dev = {name: self.codes[name].to(device) for name in ("k", "v")}
        dev.update({name + "_scale": None if self.scales[name] is None else self.scales[name].to(device) for name in ("k", "v")})
        return dev, *(torch.from_numpy(np.ascontiguousarray(x)).to(device) for x in
                      (self.cu, np.array(self.kv, np.int32), self.table))

    def expect_attention(self, causal=True, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        parts = []
        for b, n in enumerate(self.new):
            q = self.q[self.cu[b]:self.cu[b + 1]].double().numpy()
            seen = [min(self.kv[b], self.kv[b] - n + i + 1) if causal else self.kv[b] for i in range(n)]
            parts.append(attention(q, self.kc[b], self.vc[b], scale, seen))
        return [np.concatenate([p[i] for p in parts]) for i in range(4)]


def assert_attention(out, lse, expected):
    ref, ref_lse, tol, tol_lse = expected
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert got.shape == ref.shape and got_lse.shape == ref_lse.shape
    empty = np.isneginf(ref_lse)
    assert (np.isneginf(got_lse) == empty).all() and (got[empty] == 0).all()
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) / tol).max(initial=0)
    assert worst <= 1, f"output {worst:.3g} of its bound"
    worst = (np.abs(got_lse[~empty] - ref_lse[~empty]) / tol_lse[~empty]).max(initial=0)
    assert worst <= 1, f"log of the sum {worst:.3g} of its bound"
