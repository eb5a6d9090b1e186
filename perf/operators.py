"""Workloads of the cache and attention operators that surround a verification step.

A serving step of speculative decoding runs the target model over k+1 new
tokens per sequence: their keys and values are written to a paged cache
(append), the new tokens attend over it (attend), and the accepted length then
only moves the sequence's length.  Prompts enter through prompt attention, and
a cached prefix leaves the cache (for another process, or for a draft model
with its own layout) through read.

A sequence b of a batch has n_b new tokens (packed, cu[b] .. cu[b+1]) and
kv_len[b] cached tokens, the new ones last: new token i is at position
kv_len[b] - n_b + i, in page table[b, position // page_size].

`run` computes every operator in plain torch (32 bits, rounded once at the
end), or, where `own` is set, by the library's calls.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
LOWEST = -120           # least exponent of a scale


# ---------------------------------------------------------------- cases
def listed():
    return [
        # decode: one new token for each of a few dozen sequences
        dict(name="append-1tok", op="append", kv="bf16", seqs=32, n_lo=1, n_hi=1, ctx_lo=1, ctx_hi=600, hkv=8, hq=32, d=64, page=32, shape=1),
        # verification step of k = 7 drafts: 8 new tokens per sequence
        dict(name="append-k7", op="append", kv="e4m3", seqs=256, n_lo=8, n_hi=8, ctx_lo=8, ctx_hi=500, hkv=8, hq=64, d=128, page=16, shape=2),
        # prompts of uneven lengths enter the cache
        dict(name="append-prompts", op="append", kv="e4m3", seqs=12, n_lo=1000, n_hi=8000, ctx_lo=0, ctx_hi=0, hkv=8, hq=32, d=128, page=64, shape=3),
        # a few short prefixes are read back
        dict(name="read-short", op="read", kv="bf16", seqs=3, n_lo=20, n_hi=200, ctx_lo=0, ctx_hi=100, hkv=4, hq=12, d=64, page=16, shape=4),
        # whole cached conversations are read back
        dict(name="read-long", op="read", kv="e4m3", seqs=8, n_lo=2000, n_hi=8000, ctx_lo=0, ctx_hi=0, hkv=8, hq=64, d=128, page=32, shape=5),
        # plain decode of a few short sequences: latency
        dict(name="attend-1tok", op="attend", kv="bf16", seqs=4, n_lo=1, n_hi=1, ctx_lo=1, ctx_hi=700, hkv=8, hq=32, d=128, page=16, shape=6),
        # verification of k = 7 drafts, grouped heads, ragged contexts
        dict(name="attend-k7", op="attend", kv="bf16", seqs=64, n_lo=8, n_hi=8, ctx_lo=500, ctx_hi=8000, hkv=8, hq=64, d=128, page=32, shape=7),
        # verification of k = 15 drafts over a quantised cache
        dict(name="attend-k15", op="attend", kv="e4m3", seqs=64, n_lo=16, n_hi=16, ctx_lo=1000, ctx_hi=16000, hkv=8, hq=64, d=128, page=64, shape=8),
        # a chunk of a long prompt over what is cached of it
        dict(name="attend-chunk", op="attend", kv="bf16", seqs=4, n_lo=300, n_hi=512, ctx_lo=6000, ctx_hi=16000, hkv=8, hq=32, d=128, page=64, shape=9),
        # very short prompts, one head per key-value head
        dict(name="prompt-short", op="prompt", kv="bf16", seqs=3, n_lo=1, n_hi=200, ctx_lo=0, ctx_hi=0, hkv=8, hq=8, d=64, page=16, shape=10),
        # a batch of ordinary prompts
        dict(name="prompt-mixed", op="prompt", kv="bf16", seqs=8, n_lo=100, n_hi=2048, ctx_lo=0, ctx_hi=0, hkv=8, hq=32, d=128, page=16, shape=11),
        # long documents
        dict(name="prompt-long", op="prompt", kv="bf16", seqs=3, n_lo=4000, n_hi=8192, ctx_lo=0, ctx_hi=0, hkv=8, hq=32, d=128, page=16, shape=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "read", "attend", "attend", "attend", "prompt", "prompt"))
    hkv, group = rng.choice(((8, 1), (8, 4), (8, 8), (4, 7), (2, 5), (4, 3), (1, 16), (8, 2)))
    c = dict(op=op, kv=rng.choice(("bf16", "e4m3")), hkv=hkv, hq=hkv * group, d=rng.choice((64, 128)),
             page=rng.choice((16, 32, 64, 128)), shape=rng.randrange(1 << 30))
    if op in ("append", "read"):
        kind = rng.randrange(2 if op == "append" else 1)
        n = rng.choice((1, 1, 2, 4, 8, 16)) if kind else _log(rng, 4, 8000)
        c.update(seqs=_log(rng, 2, 256 if kind else 10), n_lo=n if kind else max(1, n // 4), n_hi=n, ctx_lo=0, ctx_hi=_log(rng, 1, 500))
    elif op == "attend":
        if rng.random() < 0.75:     # decode and verification steps
            n, hi = rng.choice((1, 1, 4, 5, 8, 16)), _log(rng, 60, 16000)
            c.update(seqs=_log(rng, 1, 64), n_lo=n, n_hi=n, ctx_lo=max(1, hi // 10), ctx_hi=hi)
        else:                       # chunks of prompts
            n, hi = _log(rng, 20, 512), _log(rng, 60, 16000)
            c.update(seqs=_log(rng, 1, 4), n_lo=max(1, n // 2), n_hi=n, ctx_lo=max(1, hi // 3), ctx_hi=hi)
    else:
        n = _log(rng, 30, 8000)
        c.update(kv="bf16", page=16, seqs=_log(rng, 1, max(1, min(16, 16000 // n))), n_lo=max(1, n // 8), n_hi=n, ctx_lo=0, ctx_hi=0)
    return c


def lengths(case):
    """New tokens and cached tokens before them, per sequence: fixed by the case."""
    r = random.Random(case["shape"])
    new = [_log(r, case["n_lo"], case["n_hi"]) for _ in range(case["seqs"])]
    old = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["seqs"])]
    return new, old


def work(case):
    new, old = lengths(case)
    hkv, hq, d = case["hkv"], case["hq"], case["d"]
    n, kv = sum(new), sum(new) + sum(old)
    vec = 2 * d if case["kv"] == "bf16" else d + 1              # one cached vector and its scale
    pages = sum(-(-(a + b) // case["page"]) for a, b in zip(new, old))
    if case["op"] in ("append", "read"):
        return {"bytes": 2 * n * hkv * (2 * d + vec) + 4 * n // case["page"], "flops": 4 * n * hkv * d}
    rows = 2 * (2 * n * hq * d) + 4 * n * hq                    # q, out and lse
    if case["op"] == "prompt":
        pairs = sum(a * (a + 1) // 2 for a in new)
        return {"bytes": rows + 2 * n * hkv * 2 * d, "flops": 4 * d * hq * pairs}
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, old))
    return {"bytes": rows + 2 * kv * hkv * vec + 4 * pages, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------- inputs
def _quantise(x):
    """[..., d] float32 -> e4m3 codes and one power of two per vector, the least that keeps the codes
    within +-448, held as its exponent + 127 (the definition append implements)."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)                                    # 448 * 2^(e - 9) = 0.875 * 2^e
    e = torch.where(amax > 0, e - 9 + (m > 0.875), LOWEST).clamp_min(LOWEST)
    return torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _normal(g, shape, spread=None):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if spread is not None:          # vectors of different size, as tokens' keys and values are
        x *= torch.exp(spread * torch.randn(shape[:-1], generator=g, device="cuda")).unsqueeze(-1)
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, old = lengths(case)
    hkv, hq, d, page, seqs = case["hkv"], case["hq"], case["d"], case["page"], case["seqs"]
    n, op = sum(new), case["op"]
    st = dict(case=case, new=new, old=old, n=n, max_new=max(new), max_kv=max(a + b for a, b in zip(new, old)))
    cu = [0]
    for a in new:
        cu.append(cu[-1] + a)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if op in ("attend", "prompt"):
        st["q"] = _normal(g, (n, hq, d)).bfloat16()
    if op in ("append", "prompt"):
        st["k"] = _normal(g, (n, hkv, d), 0.3).bfloat16()
        st["v"] = _normal(g, (n, hkv, d), 0.3).bfloat16()
    if op != "prompt":
        kv = [a + b for a, b in zip(new, old)]
        need = [-(-x // page) for x in kv]
        pages = sum(need) + 5
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((seqs, max(need)), dtype=torch.int32, device="cuda")
        at = 0
        for b, x in enumerate(need):
            table[b, :x] = order[at:at + x]
            at += x
        st["table"], st["kv_len"] = table, torch.tensor(kv, dtype=torch.int32, device="cuda")
        # cached tokens: the pools hold [page, head, slot, d]
        pool = {}
        for name in ("k", "v"):
            x = _normal(g, (pages, hkv, page, d), 0.3)
            if case["kv"] == "bf16":
                pool[name], pool[name + "_scale"] = x.bfloat16(), None
            else:
                pool[name], pool[name + "_scale"] = _quantise(x)
            del x
        st["pool"] = pool
    if own:
        # the handle (and its workspace) that a serving program keeps; it has seen no data
        import speculative_decoding_verification_68_gb300 as sv
        st["attn"] = sv.SpecAttention(hq, hkv, d, seqs)
        if op != "prompt":
            st["kv_pool"] = sv.KVPool(pool["k"], pool["v"], pool["k_scale"], pool["v_scale"])
    return st


# ---------------------------------------------------------------- plain forms
def _token_places(st):
    """Sequence and index in it of every packed token."""
    t = torch.arange(st["n"], device="cuda")
    b = torch.searchsorted(st["cu"][1:].long(), t, right=True)
    return b, t - st["cu"].long()[b]


def _slots(st):
    """Page and slot of every packed new token."""
    b, i = _token_places(st)
    pos = st["kv_len"].long()[b] - (st["cu"][1:] - st["cu"][:-1]).long()[b] + i
    page = st["case"]["page"]
    return st["table"].long()[b, pos // page], pos % page


def _plain_append(st):
    page, slot = _slots(st)
    pool = st["pool"]
    for name in ("k", "v"):
        if st["case"]["kv"] == "bf16":
            pool[name][page, :, slot] = st[name]
        else:
            codes, scale = _quantise(st[name].float())
            pool[name].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            pool[name + "_scale"][page, :, slot] = scale
    return pool


def _values(x, scale):
    return x.float() if scale is None else torch.ldexp(x.float(), scale.unsqueeze(-1).int() - 127)


def _take(pool, name, page, slot):
    """Cached vectors [..., heads, d] as values in 32 bits."""
    x, scale = pool[name], pool[name + "_scale"]
    if scale is None:
        return x[page, :, slot].float()
    return _values(x.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn), scale[page, :, slot])


def _plain_read(st):
    page, slot = _slots(st)
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
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, hkv, group * n, L), v.permute(0, 2, 1, 3)).view(B, hkv, group, n, d)
    o = o / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, hq, d), lse.permute(0, 3, 1, 2).reshape(B, n, hq)


def _padded(st, x):
    """Packed rows [N, ...] as [B, max_new, ...]; what lies past a sequence's end is arbitrary."""
    i = st["cu"][:-1].long()[:, None] + torch.arange(st["max_new"], device="cuda")[None]
    return x[i.clamp_max(st["n"] - 1)].float()


def _plain_attend(st):
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
    o, lse = _plain_softmax_av(_padded(st, st["q"]), k, v, seen, case["d"] ** -0.5)
    at = _token_places(st)
    return {"out": o[at].bfloat16(), "lse": lse[at]}


def _plain_prompt(st):
    i = torch.arange(st["max_new"], device="cuda")
    new = (st["cu"][1:] - st["cu"][:-1]).long()
    seen = (i[None, None] <= i[None, :, None]) & (i[None, None] < new[:, None, None])
    o, lse = _plain_softmax_av(_padded(st, st["q"]), _padded(st, st["k"]), _padded(st, st["v"]), seen, st["case"]["d"] ** -0.5)
    at = _token_places(st)
    return {"out": o[at].bfloat16(), "lse": lse[at]}


def run(st):
    op = st["case"]["op"]
    if own:
        attn = st["attn"]
        if op == "prompt":
            return attn.prompt(st["q"], st["k"], st["v"], st["cu"], want_lse=True)
        pool, where = st["kv_pool"], (st["cu"], st["kv_len"], st["table"])
        if op == "append":
            attn.append(pool, st["k"], st["v"], *where)
            return st["pool"]
        if op == "read":
            return attn.read(pool, *where, n_tokens=st["n"])
        return attn.attend(pool, st["q"], *where, want_lse=True)
    return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend, "prompt": _plain_prompt}[op](st)


# ---------------------------------------------------------------- 64 bits
def _round_e4m3(x):
    """float64 values rounded to the nearest e4m3 value, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -40))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


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
    op, page, hkv, hq, d = case["op"], case["page"], case["hkv"], case["hq"], case["d"]
    cu = st["cu"].tolist()
    if op == "prompt":
        table = None
    else:
        table = st["table"].long()
        kv_len = st["kv_len"].tolist()

    def cached(name, b, lo, hi):
        pos = torch.arange(lo, hi, device="cuda")
        x = st["pool"][name]
        x = x.view(torch.uint8)[table[b, pos // page], :, pos % page].view(x.dtype).double() if x.element_size() == 1 else x[table[b, pos // page], :, pos % page].double()
        scale = st["pool"][name + "_scale"]
        return x if scale is None else x * torch.exp2(scale[table[b, pos // page], :, pos % page].double() - 127).unsqueeze(-1)

    if op == "append":
        out = {}
        for name in ("k", "v"):
            values = st["pool"][name].double()
            scales = st["pool"][name + "_scale"]
            for b in range(case["seqs"]):
                x = st[name][cu[b]:cu[b + 1]].double()
                pos = torch.arange(kv_len[b] - x.shape[0], kv_len[b], device="cuda")
                at = (table[b, pos // page], slice(None), pos % page)
                if scales is None:
                    values[at] = x
                else:
                    e = torch.ceil(torch.log2(x.abs().amax(-1) / E4M3_MAX)).clamp_min(LOWEST)
                    values[at] = _round_e4m3(x / torch.exp2(e).unsqueeze(-1))
                    scales[at] = (e + 127).to(torch.uint8)
            out[name], out[name + "_scale"] = values, scales
        return out
    if op == "read":
        return {name: torch.cat([cached(name, b, kv_len[b] - st["new"][b], kv_len[b]) for b in range(case["seqs"])]) for name in ("k", "v")}
    if sum((a + b) * a for a, b in zip(st["new"], st["old"])) * 4 * d * hq > 8e12:
        return None
    out = torch.empty((st["n"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((st["n"], hq), dtype=torch.float64, device="cuda")
    group = hq // hkv
    for b in range(case["seqs"]):
        lo, hi = cu[b], cu[b + 1]
        k, v = (st[x][lo:hi].double() for x in ("k", "v")) if op == "prompt" else (cached(x, b, 0, kv_len[b]) for x in ("k", "v"))
        for h in range(hkv):
            at = (slice(lo, hi), slice(h * group, (h + 1) * group))
            out[at], lse[at] = _exact_rows(st["q"][at].double(), k[:, h], v[:, h], st["old"][b], d ** -0.5)
    return {"out": out, "lse": lse}
