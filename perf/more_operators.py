"""Workloads of a 4-bit cache and of the position rotation on the way into a cache.

A serving step of speculative decoding projects its new tokens to queries, keys
and values; before they are used, queries and keys are rotated by their
positions.  `append_rotated` does that on the way into the paged cache; a 4-bit
cache holds a vector of d values as d codes of 4 bits (e2m1: 0, 0.5, 1, 1.5, 2,
3, 4, 6 and their negatives), one e4m3 scale per 16 of them, and one power of
two, so that a token of 8 heads of 128 takes 1168 bytes where bf16 takes 4096.

A sequence b of a batch has n_b new tokens (packed, cu[b] .. cu[b+1]) and
kv_len[b] cached tokens, the new ones last: new token i is at position
kv_len[b] - n_b + i, in page table[b, position // page_size].

Operations: `rope` rotates queries and keys and appends keys and values to a bf16
or e4m3 cache; `store` appends to a 4-bit cache, with or without rotation, and
reads the tokens back; `attend` is attention of new tokens over a 4-bit cache;
`step` is a verification step's part of a layer, rotation, append and attention.

`run` computes every operator in plain torch (32 bits, rounded once at the
end), or, where `own` is set, by the library's calls.
"""
import math
import random

import torch

own = False

LOWEST = -120           # least exponent of a vector's power of two
BLOCK = 16              # values that share an e4m3 scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def _case(name, op, kv, seqs, n, ctx, heads, d, page, shape, rot=0, pairs=False, want_k=False):
    return dict(name=name, op=op, kv=kv, seqs=seqs, n_lo=n[0], n_hi=n[1], ctx_lo=ctx[0], ctx_hi=ctx[1], hq=heads[0], hkv=heads[1],
                d=d, page=page, shape=shape, rot=rot, pairs=pairs, want_k=want_k)


def listed():
    return [
        # decode of a few dozen sequences, half of each vector rotated, neighbours in pairs: latency
        _case("rope-1tok", "rope", "bf16", 32, (1, 1), (1, 600), (32, 8), 64, 32, 1, rot=32, pairs=True),
        # verification step of k = 7 drafts over an e4m3 cache
        _case("rope-k7", "rope", "e4m3", 256, (8, 8), (8, 500), (64, 8), 128, 16, 2, rot=128),
        # prompts of uneven lengths enter a bf16 cache; the rotated keys go on to prompt attention
        _case("rope-prompts", "rope", "bf16", 12, (1000, 8000), (0, 0), (32, 8), 128, 64, 3, rot=128, want_k=True),
        # a verification step's tokens enter a 4-bit cache
        _case("store-k7", "store", "e2m1", 256, (8, 8), (8, 500), (64, 8), 128, 16, 4, rot=128),
        # prompts enter a 4-bit cache; a draft model with a layout of its own reads them back
        _case("store-prompts", "store", "e2m1", 12, (1000, 8000), (0, 0), (32, 8), 128, 64, 5),
        # plain decode of a few short sequences: latency
        _case("attend-1tok", "attend", "e2m1", 4, (1, 1), (1, 700), (32, 8), 128, 16, 6),
        # plain decode of many long conversations
        _case("attend-1tok-long", "attend", "e2m1", 64, (1, 1), (1000, 16000), (64, 8), 128, 64, 7),
        # verification of k = 7 drafts, ragged contexts
        _case("attend-k7", "attend", "e2m1", 64, (8, 8), (500, 8000), (64, 8), 128, 32, 8),
        # verification of k = 15 drafts over long contexts
        _case("attend-k15", "attend", "e2m1", 64, (16, 16), (1000, 16000), (64, 8), 128, 64, 9),
        # a chunk of a long prompt over what is cached of it
        _case("attend-chunk", "attend", "e2m1", 4, (300, 512), (6000, 16000), (32, 8), 128, 64, 10),
        # a small model's verification of k = 4 drafts: heads of 64 in an odd group
        _case("attend-d64", "attend", "e2m1", 24, (5, 5), (100, 3000), (14, 2), 64, 32, 11),
        # a whole verification step of a layer, k = 7
        _case("step-k7", "step", "e2m1", 32, (8, 8), (300, 5000), (32, 8), 128, 64, 12, rot=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "rope", "store", "attend", "attend", "attend", "attend", "step"))
    hkv, group = rng.choice(((8, 1), (8, 4), (8, 8), (4, 7), (2, 5), (4, 3), (1, 16), (8, 2)))
    d = rng.choice((64, 128))
    c = dict(op=op, kv=rng.choice(("bf16", "e4m3")) if op == "rope" else "e2m1", hkv=hkv, hq=hkv * group, d=d,
             page=rng.choice((16, 32, 64, 128)), shape=rng.randrange(1 << 30),
             rot=0 if op == "attend" else rng.choice((d, d, d // 2, 16)), pairs=rng.random() < 0.3, want_k=op == "rope" and rng.random() < 0.3)
    if op in ("rope", "store"):
        steps = rng.random() < 0.5
        n = rng.choice((1, 1, 2, 4, 5, 8, 16)) if steps else _log(rng, 4, 8000)
        most = 256 if steps else max(2, min(12, 36000 // n))
        c.update(seqs=_log(rng, 2, most), n_lo=n if steps else max(1, n // 4), n_hi=n, ctx_lo=0, ctx_hi=_log(rng, 1, 500))
        if op == "store" and rng.random() < 0.4:
            c["rot"] = 0
    elif op == "step" or rng.random() < 0.75:       # decode and verification steps
        n, hi = rng.choice((1, 1, 2, 4, 5, 8, 16)), _log(rng, 60, 16000)
        c.update(seqs=_log(rng, 1, 64), n_lo=n, n_hi=n, ctx_lo=max(1, hi // 10), ctx_hi=hi)
    else:                                           # chunks of prompts
        n, hi = _log(rng, 20, 512), _log(rng, 60, 16000)
        c.update(seqs=_log(rng, 1, 4), n_lo=max(1, n // 2), n_hi=n, ctx_lo=max(1, hi // 3), ctx_hi=hi)
    return c


def lengths(case):
    """New tokens and cached tokens before them, per sequence: fixed by the case."""
    r = random.Random(case["shape"])
    new = [_log(r, case["n_lo"], case["n_hi"]) for _ in range(case["seqs"])]
    old = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["seqs"])]
    return new, old


def work(case):
    new, old = lengths(case)
    hkv, hq, d, op = case["hkv"], case["hq"], case["d"], case["op"]
    n, kv = sum(new), sum(new) + sum(old)
    vec = {"bf16": 2 * d, "e4m3": d + 1, "e2m1": d // 2 + d // BLOCK + 1}[case["kv"]]    # one cached vector and its scales
    pages = sum(-(-(a + b) // case["page"]) for a, b in zip(new, old))
    rows = 2 * n * hq * d                                                               # queries, or the output
    kv_rows = 2 * (2 * n * hkv * d)                                                     # keys and values
    total, flops = 0, 0
    if case["rot"]:
        at = len(set().union(*(range(b, a + b) for a, b in zip(new, old))))             # distinct positions
        total += 4 * case["rot"] * at
        flops += 3 * n * case["rot"] * hkv
    if op == "rope":
        total += 2 * rows + kv_rows + (kv_rows // 2 if case["want_k"] else 0) + 2 * n * hkv * vec
        flops += 3 * n * case["rot"] * hq
    elif op == "store":
        total += 2 * kv_rows + 2 * n * hkv * vec
        flops += 4 * n * hkv * d
    else:
        total += 2 * rows + 4 * n * hq + 2 * kv * hkv * vec + 4 * pages
        flops += 4 * d * hq * sum(a * b + a * (a + 1) // 2 for a, b in zip(new, old))
        if op == "step":
            total += kv_rows
            flops += 3 * n * case["rot"] * hq + 4 * n * hkv * d
    return {"bytes": total, "flops": flops}


# ---------------------------------------------------------------- inputs
def _exponent(x, limit):
    """Least e >= LOWEST with max|x| <= limit * 2^e, of vectors in 32 bits."""
    amax = x.abs().amax(-1)
    (top, shift), (m, e) = math.frexp(limit), torch.frexp(amax)
    return torch.where(amax > 0, e - shift + (m > top), LOWEST).clamp_min(LOWEST)


def _quantise8(x):
    """[..., d] float32 -> e4m3 codes and a power of two per vector, held as its exponent + 127."""
    e = _exponent(x, 448.0)
    return torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _quantise4(x):
    """[..., d] float32 -> codes (two a byte, the first low), e4m3 scales per 16 values, and a power of two per vector."""
    e = _exponent(x, 6 * 448.0)
    y = torch.ldexp(x, -e.unsqueeze(-1)).unflatten(-1, (-1, BLOCK))
    s = (y.abs().amax(-1) / 6).to(torch.float8_e4m3fn)
    f = s.float().unsqueeze(-1)
    z = torch.where(f > 0, y / f, torch.copysign(torch.zeros_like(y), y))
    a = z.abs()
    code = torch.signbit(z).to(torch.uint8) << 3
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):   # ties to the even code
        code += a >= border if up else a > border
    code = code.flatten(-2)
    return code[..., ::2] | code[..., 1::2] << 4, s, (e + 127).to(torch.uint8)


def _normal(g, shape, spread=None):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if spread is not None:          # vectors of different size, as tokens' keys and values are
        x *= torch.exp(spread * torch.randn(shape[:-1], generator=g, device="cuda")).unsqueeze(-1)
    return x


def _cached(g, kv, shape):
    """A pool's vectors [page, head, slot, d] as held: codes or values, scales per block, scales per vector."""
    if kv == "bf16":
        return _normal(g, shape, 0.3).bfloat16(), None, None
    parts = []
    step = max(1, (1 << 28) // math.prod(shape[1:]))
    for a in range(0, shape[0], step):                  # so that a large pool never exists in 32 bits
        x = _normal(g, (min(step, shape[0] - a), *shape[1:]), 0.3)
        parts.append([y.view(torch.uint8) for y in (_quantise8(x) if kv == "e4m3" else _quantise4(x))])
    held = [torch.cat(x) for x in zip(*parts)]
    if kv == "e4m3":
        return held[0].view(torch.float8_e4m3fn), None, held[1]
    return held[0], held[1].view(torch.float8_e4m3fn), held[2]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, old = lengths(case)
    hkv, hq, d, page, seqs, op = case["hkv"], case["hq"], case["d"], case["page"], case["seqs"], case["op"]
    n = sum(new)
    kv = [a + b for a, b in zip(new, old)]
    st = dict(case=case, new=new, old=old, n=n, max_new=max(new), max_kv=max(kv))
    cu = [0]
    for a in new:
        cu.append(cu[-1] + a)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if op != "store":
        st["q"] = _normal(g, (n, hq, d)).bfloat16()
    if op != "attend":
        st["k"] = _normal(g, (n, hkv, d), 0.3).bfloat16()
        st["v"] = _normal(g, (n, hkv, d), 0.3).bfloat16()
    if case["rot"]:
        # the model's table of cosines and sines, for as many positions as the cache has room for
        angle = torch.arange(max(kv), dtype=torch.float64, device="cuda")[:, None] * 500000.0 ** -(
            torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        st["table_cs"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    need = [-(-x // page) for x in kv]
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((seqs, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, x in enumerate(need):
        table[b, :x] = order[at:at + x]
        at += x
    st["table"], st["kv_len"] = table, torch.tensor(kv, dtype=torch.int32, device="cuda")
    st["pool"] = {}
    for name in ("k", "v"):
        for part, x in zip(("", "_block", "_scale"), _cached(g, case["kv"], (pages, hkv, page, d))):
            st["pool"][name + part] = x
    if own:
        # the handle (and its workspace) that a serving program keeps; it has seen no data
        import speculative_decoding_verification_68_gb300 as sv
        st["attn"] = sv.SpecAttention(hq, hkv, d, seqs)
        p = st["pool"]
        codes = [p[x].view(torch.float4_e2m1fn_x2) if case["kv"] == "e2m1" else p[x] for x in ("k", "v")]
        st["kv_pool"] = sv.KVPool(*codes, p["k_scale"], p["v_scale"], p["k_block"], p["v_block"])
        if case["rot"]:
            st["rope"] = sv.Rope(st["table_cs"], interleaved=case["pairs"])
    return st


# ---------------------------------------------------------------- plain forms
def _token_places(st):
    """Sequence and index in it of every packed token."""
    t = torch.arange(st["n"], device="cuda")
    b = torch.searchsorted(st["cu"][1:].long(), t, right=True)
    return b, t - st["cu"].long()[b]


def _slots(st):
    """Position, page and slot of every packed new token."""
    b, i = _token_places(st)
    pos = st["kv_len"].long()[b] - (st["cu"][1:] - st["cu"][:-1]).long()[b] + i
    page = st["case"]["page"]
    return pos, st["table"].long()[b, pos // page], pos % page


def _rotate(st, x, pos):
    """x [n, heads, d] float32 with its first `rot` elements rotated: pairs of neighbours, or of the two halves."""
    rot, pairs = st["case"]["rot"], st["case"]["pairs"]
    if not rot:
        return x
    cs = st["table_cs"][pos][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * s, b * c + a * s
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1), x[..., rot:]], -1)


def _values4(codes, block, scale):
    """What a 4-bit cache holds, in 32 bits: bytes [..., d / 2], scales [..., d / 16] and exponents [...]."""
    low = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
    both = torch.stack([low.repeat(16), low.repeat_interleave(16)], -1)                 # the two values of every byte
    x = both[codes.int()].flatten(-2).unflatten(-1, (-1, BLOCK)) * block.float().unsqueeze(-1)
    return torch.ldexp(x.flatten(-2), scale.int().unsqueeze(-1) - 127)


def _plain_append(st, pos, page, slot):
    pool = st["pool"]
    for name in ("k", "v"):
        x = st[name].float()
        if name == "k":
            x = _rotate(st, x, pos)
            rotated = x
        if st["case"]["kv"] == "bf16":
            pool[name][page, :, slot] = x.bfloat16()
        elif st["case"]["kv"] == "e4m3":
            codes, scale = _quantise8(x)
            pool[name].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            pool[name + "_scale"][page, :, slot] = scale
        else:
            codes, block, scale = _quantise4(x)
            pool[name][page, :, slot] = codes
            pool[name + "_block"].view(torch.uint8)[page, :, slot] = block.view(torch.uint8)
            pool[name + "_scale"][page, :, slot] = scale
    return rotated


def _take(pool, name, page, slot):
    """Vectors [..., heads, d] of a 4-bit cache as values in 32 bits."""
    codes, block, scale = pool[name], pool[name + "_block"], pool[name + "_scale"]
    return _values4(codes[page, :, slot], block.view(torch.uint8)[page, :, slot].view(block.dtype), scale[page, :, slot])


def _held(pool):
    return {name: x for name, x in pool.items() if x is not None}


def _plain_rope(st):
    pos, page, slot = _slots(st)
    out = {"q": _rotate(st, st["q"].float(), pos).bfloat16()}
    k = _plain_append(st, pos, page, slot)
    if st["case"]["want_k"]:
        out["k"] = k.bfloat16()
    return {**out, "pool": _held(st["pool"])}


def _plain_store(st):
    pos, page, slot = _slots(st)
    _plain_append(st, pos, page, slot)
    return {name: _take(st["pool"], name, page, slot).bfloat16() for name in ("k", "v")}


def _plain_softmax_av(q, k, v, seen, scale):
    """q [B, n, hq, d], k and v [B, L, hkv, d], seen [B, n, L]: output and log of the sum."""
    B, n, hq, d = q.shape
    L, hkv = k.shape[1], k.shape[2]
    group = hq // hkv
    q = q.view(B, n, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, group * n, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, hkv, group, n, L)
    s.mul_(scale).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, hkv, group * n, L), v.permute(0, 2, 1, 3)).view(B, hkv, group, n, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total)).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, hq, d), lse.permute(0, 3, 1, 2).reshape(B, n, hq)


def _padded(st, x):
    """Packed rows [N, ...] as [B, max_new, ...]; what lies past a sequence's end is arbitrary."""
    i = st["cu"][:-1].long()[:, None] + torch.arange(st["max_new"], device="cuda")[None]
    return x[i.clamp_max(st["n"] - 1)].float()


def _plain_attend(st, q):
    case, L = st["case"], st["max_kv"]
    pos = torch.arange(L, device="cuda")
    kv_len = st["kv_len"].long()[:, None]
    held = pos[None] < kv_len
    page = torch.where(held, st["table"].long()[:, pos // case["page"]], torch.zeros_like(pos)[None])
    slot = (pos % case["page"])[None].expand_as(page)
    k, v = (_take(st["pool"], name, page, slot) for name in ("k", "v"))
    new = (st["cu"][1:] - st["cu"][:-1]).long()[:, None]
    last = kv_len - new + torch.arange(st["max_new"], device="cuda")[None]
    seen = (pos[None, None] <= last[:, :, None]) & held[:, None]
    o, lse = _plain_softmax_av(_padded(st, q), k, v, seen, case["d"] ** -0.5)
    at = _token_places(st)
    return {"out": o[at].bfloat16(), "lse": lse[at]}


def _plain_step(st):
    pos, page, slot = _slots(st)
    _plain_append(st, pos, page, slot)
    return _plain_attend(st, _rotate(st, st["q"].float(), pos).bfloat16())


def run(st):
    op = st["case"]["op"]
    if not own:
        return _plain_attend(st, st["q"]) if op == "attend" else {"rope": _plain_rope, "store": _plain_store, "step": _plain_step}[op](st)
    attn, pool, where = st["attn"], st["kv_pool"], (st["cu"], st["kv_len"], st["table"])
    if op == "rope":
        out = attn.append_rotated(pool, st["k"], st["v"], *where, st["rope"], q=st["q"], want_k=st["case"]["want_k"])
        return {**out, "pool": _held(st["pool"])}
    if op == "store":
        if st["case"]["rot"]:
            attn.append_rotated(pool, st["k"], st["v"], *where, st["rope"])
        else:
            attn.append(pool, st["k"], st["v"], *where)
        return attn.read(pool, *where, n_tokens=st["n"])
    q = st["q"]
    if op == "step":
        q = attn.append_rotated(pool, st["k"], st["v"], *where, st["rope"], q=q)["q"]
    return attn.attend(pool, q, *where, want_lse=True, max_kv=st["max_kv"])


# ---------------------------------------------------------------- 64 bits
def _nearest(x, mantissa, least, most):
    """float64 values rounded to the nearest with `mantissa` bits and exponents from `least` on, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -60))).clamp_min(least)
    step = torch.exp2(e - mantissa)
    return (torch.round(x / step) * step).clamp(-most, most)


def _exact_held(x, kv):
    """What a cache of type kv holds of float64 vectors: (values in units of 2^e, values, e)."""
    limit = 448.0 if kv == "e4m3" else 6 * 448.0
    e = torch.ceil(torch.log2(x.abs().amax(-1) / limit)).clamp_min(LOWEST)
    unit = torch.exp2(e).unsqueeze(-1)
    y = x / unit
    if kv == "e4m3":
        y = _nearest(y, 3, -6.0, 448.0)
    else:
        y = y.unflatten(-1, (-1, BLOCK))
        s = _nearest(y.abs().amax(-1, keepdim=True) / 6, 3, -6.0, 448.0)
        y = torch.where(s > 0, _nearest(y / torch.where(s > 0, s, torch.ones_like(s)), 1, 0.0, 6.0) * s, torch.zeros_like(y)).flatten(-2)
    return y, y * unit, e


def _exact_turned(st, x):
    """Vectors [n, heads, d] in float64, turned as complex numbers by their positions' entries of the table."""
    rot = st["case"]["rot"]
    x = x.double()
    if not rot:
        return x
    first = torch.cat([torch.arange(o, kv, device="cuda") for o, kv in zip(st["old"], st["kv_len"].tolist())])
    t = st["table_cs"].double()[first]
    turn = torch.complex(t[:, :rot // 2], t[:, rot // 2:])[:, None]
    head = x[..., :rot].unflatten(-1, (rot // 2, 2) if st["case"]["pairs"] else (2, rot // 2))
    if not st["case"]["pairs"]:
        head = head.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
    if not st["case"]["pairs"]:
        z = z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), x[..., rot:]], -1)


def _exact_rows(q, k, v, first, scale):
    """One sequence and key-value head: q [n, group, d], k and v [L, d], all float64;
    row i sees keys 0 .. first + i."""
    n, group, d = q.shape
    out = torch.empty_like(q)
    lse = torch.empty((n, group), dtype=torch.float64, device=q.device)
    step = max(1, (1 << 26) // (group * max(1, k.shape[0])))
    for a in range(0, n, step):
        b = min(n, a + step)
        L = first + b
        s = torch.einsum("ngd,ld->ngl", q[a:b], k[:L]) * scale
        over = torch.arange(L, device=q.device)[None, :] > torch.arange(first + a, first + b, device=q.device)[:, None]
        s = torch.where(over[:, None], torch.full_like(s, -math.inf), s)
        lse[a:b] = torch.logsumexp(s, -1)
        out[a:b] = torch.einsum("ngl,ld->ngd", torch.exp(s - lse[a:b, :, None]), v[:L])
    return out, lse


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, kv, page, hkv, hq, d = case["op"], case["kv"], case["page"], case["hkv"], case["hq"], case["d"]
    cu, kv_len, table, pool = st["cu"].tolist(), st["kv_len"].tolist(), st["table"].long(), st["pool"]
    if op in ("rope", "store"):
        held = {name: _exact_turned(st, st[name]) if name == "k" else st[name].double() for name in ("k", "v")}
        if op == "store":
            return {name: _exact_held(x, kv)[1] for name, x in held.items()}
        out = {"q": _exact_turned(st, st["q"])}
        if case["want_k"]:
            out["k"] = held["k"]
        after = {}
        for name, x in held.items():
            values = pool[name].double()
            scales = pool[name + "_scale"]
            units, _, e = (x, x, None) if kv == "bf16" else _exact_held(x, kv)
            for b in range(case["seqs"]):
                pos = torch.arange(kv_len[b] - st["new"][b], kv_len[b], device="cuda")
                at = (table[b, pos // page], slice(None), pos % page)
                values[at] = units[cu[b]:cu[b + 1]]
                if e is not None:
                    scales[at] = (e[cu[b]:cu[b + 1]] + 127).to(torch.uint8)
            after[name] = values
            if scales is not None:
                after[name + "_scale"] = scales
        return {**out, "pool": after}
    if sum((a + b) * a for a, b in zip(st["new"], st["old"])) * 4 * d * hq > 8e12:
        return None

    digits = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def cached(name, b):
        pos = torch.arange(kv_len[b], device="cuda")
        at = (table[b, pos // page], slice(None), pos % page)
        c = pool[name][at].long()
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        x = digits[c & 7] * torch.where(c >= 8, -1.0, 1.0)
        x = x * pool[name + "_block"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double().repeat_interleave(BLOCK, -1)
        return x * torch.exp2(pool[name + "_scale"][at].double() - 127).unsqueeze(-1)

    q = st["q"].double()
    if op == "step":
        q = _exact_turned(st, st["q"]).bfloat16().double()      # handed from one call to the other in bf16
        fresh = {"k": _exact_held(_exact_turned(st, st["k"]), kv)[1], "v": _exact_held(st["v"].double(), kv)[1]}
    out = torch.empty((st["n"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((st["n"], hq), dtype=torch.float64, device="cuda")
    group = hq // hkv
    for b in range(case["seqs"]):
        lo, hi = cu[b], cu[b + 1]
        k, v = (cached(x, b) for x in ("k", "v"))
        if op == "step":
            k[st["old"][b]:], v[st["old"][b]:] = fresh["k"][lo:hi], fresh["v"][lo:hi]
        for h in range(hkv):
            at = (slice(lo, hi), slice(h * group, (h + 1) * group))
            out[at], lse[at] = _exact_rows(q[at].double(), k[:, h], v[:, h], st["old"][b], d ** -0.5)
    return {"out": out, "lse": lse}
