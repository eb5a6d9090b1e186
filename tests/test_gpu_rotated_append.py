"""Appends of rotated keys, with the queries beside them, against the formula in
32 bits (bit for bit) and in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import _attn, _attn4  # noqa: E402
from tests._attn import World  # noqa: E402
from tests._attn4 import FOUR, World4, bytes_of, quantise4, rope_table, rotate  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    return sv


def world(lib, new, old, hq, hkv, d, page, dtype, seed=0, **kw):
    if dtype == FOUR:
        w = World4(new, old, hq, hkv, d, page, seed=seed, **kw)
        pool, where = w.pool(lib)
    else:
        w = World(new, old, hq, hkv, d, page, dtype, seed=seed, **kw)
        t, *where = w.to("cuda")
        pool = lib.KVPool(t["k"], t["v"], t["k_scale"], t["v_scale"])
    return w, lib.SpecAttention(hq, hkv, d, max(1, len(new))), pool, tuple(where)


def positions_of(w):
    return np.concatenate([np.arange(kv - n, kv) for n, kv in zip(w.new, w.kv)] or [np.zeros(0, int)])


def assert_cached(w, pool, k, v):
    """The pool holds k and v [n, heads, D] float32 at the batch's slots, quantised from 32 bits, and nothing else has changed."""
    for name, x in (("k", k), ("v", v)):
        if isinstance(w, World4):
            want = {part: w.raw[name + part].clone() for part in ("", "_block", "_scale")}
            parts = dict(zip(("", "_block", "_scale"), quantise4(x.astype(np.float64))))
            got = {part: bytes_of(pool)[name + part] for part in parts}
        elif w.dtype == E4M3:
            want = {"": w.codes[name].view(torch.uint8).clone(), "_scale": w.scales[name].clone()}
            parts = dict(zip(("", "_scale"), _attn.quantise(x.astype(np.float64))))
            got = {part: getattr(pool, name + part).view(torch.uint8).cpu() for part in parts}
        else:
            want = {"": w.codes[name].view(torch.int16).clone()}
            parts = {"": torch.from_numpy(x).bfloat16().view(torch.int16).numpy()}
            got = {"": getattr(pool, name).view(torch.int16).cpu()}
        for b, n in enumerate(w.new):
            for i in range(n):
                t, pos = w.cu[b] + i, w.kv[b] - n + i
                if pos >= 0:
                    for part in parts:
                        want[part][w.table[b, pos // w.page], :, pos % w.page] = torch.from_numpy(np.asarray(parts[part][t]))
        for part in parts:
            assert torch.equal(got[part], want[part]), name + part


CASES = [  # new, old, hq, hkv, d, page, rot, interleaved
    ([1], [0], 1, 1, 64, 16, 64, False),
    ([1, 1, 1], [0, 15, 16], 8, 2, 128, 16, 128, False),
    ([8, 0, 5, 8], [3, 9, 60, 61], 64, 8, 128, 16, 128, True),
    ([33, 130, 1], [31, 0, 257], 6, 3, 64, 32, 32, False),
    ([16, 16], [100, 127], 28, 4, 128, 64, 96, False),
    ([16, 3], [100, 127], 5, 5, 128, 64, 16, True),
    ([300], [7], 1, 1, 128, 128, 48, False),
    ([40], [0], 16, 1, 64, 16, 16, False),
    ([2] * 60, list(range(0, 600, 10)), 9, 3, 64, 16, 48, True),
]


@pytest.mark.parametrize("dtype", [BF16, E4M3, FOUR])
@pytest.mark.parametrize("new, old, hq, hkv, d, page, rot, interleaved", CASES)
def test_rotated_append(lib, new, old, hq, hkv, d, page, rot, interleaved, dtype):
    w, attn, pool, where = world(lib, new, old, hq, hkv, d, page, dtype, seed=1)
    table = rope_table(max(w.kv), rot)
    fused = torch.cat([w.q, w.k_new, w.v_new], 1).cuda()                   # strided: slices of one tensor
    q, k, v = fused.split([hq, hkv, hkv], 1)
    out = attn.append_rotated(pool, k, v, *where, lib.Rope(table.cuda(), interleaved), q=q, want_k=True)
    assert attn.get_error() == lib.SV_OK
    assert torch.equal(fused.cpu(), torch.cat([w.q, w.k_new, w.v_new], 1))
    pos = positions_of(w)
    want = {name: rotate(x.float().numpy(), table, pos, interleaved) for name, x in (("q", w.q), ("k", w.k_new))}
    for name, x in want.items():
        assert torch.equal(out[name].cpu().view(torch.int16), torch.from_numpy(x).bfloat16().view(torch.int16)), name
    assert_cached(w, pool, want["k"], w.v_new.float().numpy())
    # the formula in 64 bits: the table's entries, two products and a sum of 32 bits are off by 2^-24 of their
    # sizes each (2^-22 of |a| + |b| in all), and bf16's half step is 2^-8 of what is rounded
    x, angle = w.q.double().numpy(), pos[:, None] * 10000.0 ** -(np.arange(0, rot, 2) / rot)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    for place, part in ((i, x[..., i] * c - x[..., j] * s), (j, x[..., j] * c + x[..., i] * s)):
        off = np.abs(out["q"].double().cpu().numpy()[..., place] - part)
        small = 2.0 ** -22 * (np.abs(x[..., i]) + np.abs(x[..., j]))
        worst = (off / (2.0 ** -8 * (np.abs(part) + small) + small + 1e-300)).max()
        assert worst <= 1, worst


@pytest.mark.parametrize("dtype", [BF16, FOUR])
def test_in_place_without_queries_and_with_positions_of_its_own(lib, dtype):
    w, attn, pool, where = world(lib, [5, 3, 9], [100, 0, 33], 8, 2, 128, 16, dtype, seed=2)
    table = rope_table(5000, 128)
    pos = np.random.default_rng(0).integers(0, 5000, w.n).astype(np.int32)
    pos[3] = 4999
    rope = lib.Rope(table.cuda())
    q, k, v = (x.cuda() for x in (w.q, w.k_new, w.v_new))
    out = attn.append_rotated(pool, k, v, *where, rope, q=q, positions=torch.from_numpy(pos).cuda(), out={"q": q, "k": k})
    assert out["q"] is q and out["k"] is k and attn.get_error() == lib.SV_OK
    want_q, want_k = (rotate(x.float().numpy(), table, pos, False) for x in (w.q, w.k_new))
    assert torch.equal(q.cpu(), torch.from_numpy(want_q).bfloat16()) and torch.equal(k.cpu(), torch.from_numpy(want_k).bfloat16())
    assert_cached(w, pool, want_k, w.v_new.float().numpy())
    # the positions of one call do not stay for the next
    w, attn, pool, where = world(lib, [5, 3, 9], [100, 0, 33], 8, 2, 128, 16, dtype, seed=3)
    assert attn.append_rotated(pool, w.k_new.cuda(), w.v_new.cuda(), *where, rope) == {}
    assert attn.get_error() == lib.SV_OK
    assert_cached(w, pool, rotate(w.k_new.float().numpy(), table, positions_of(w), False), w.v_new.float().numpy())


@pytest.mark.parametrize("dtype", [BF16, E4M3, FOUR])
def test_agrees_with_append_where_nothing_turns(lib, dtype):
    """At position 0 the cosines are 1 and the sines 0: the bytes of plain append, zeros' signs aside."""
    w, attn, pool, where = world(lib, [7, 20], [60, 5], 8, 4, 64, 16, dtype, seed=4)
    other = world(lib, [7, 20], [60, 5], 8, 4, 64, 16, dtype, seed=4)[2]
    k, v = w.k_new.cuda(), w.v_new.cuda()
    zero = torch.zeros(w.n, dtype=torch.int32, device="cuda")
    attn.append_rotated(pool, k, v, *where, lib.Rope(rope_table(1, 64).cuda()), positions=zero)
    attn.append(other, k, v, *where)
    assert attn.get_error() == lib.SV_OK
    for name in ("k", "v", "k_scale", "v_scale", "k_block", "v_block"):
        a, b = getattr(pool, name), getattr(other, name)
        assert a is b is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF16, E4M3, FOUR])
def test_positions_that_the_table_does_not_hold(lib, dtype):
    w, attn, pool, where = world(lib, [4, 3], [30, 10], 8, 2, 64, 16, dtype, seed=5)
    rope, q, k, v = lib.Rope(rope_table(20, 64).cuda()), w.q.cuda(), w.k_new.cuda(), w.v_new.cuda()
    before = [t.view(torch.uint8).clone() for t in (pool.k, pool.v)]
    out = attn.append_rotated(pool, k, v, *where, rope, q=q, want_k=True)       # positions 30 .. 33 and 10 .. 12
    assert attn.get_error() == lib.SV_ERR_DATA and attn.get_error() == lib.SV_OK
    assert torch.isnan(out["q"][:4]).all() and torch.isnan(out["k"][:4]).all() and torch.isfinite(out["q"][4:]).all()
    for t, old in zip((pool.k, pool.v), before):
        changed = (t.view(torch.uint8) != old).any(-1).any(1)
        assert changed.sum() == 3 and changed[w.table[1, 0], 10:13].all()
    for bad in (-1, 20, 1 << 30, -(1 << 31)):
        pos = torch.tensor([0, 1, bad, 3, 4, 5, 6], dtype=torch.int32, device="cuda")
        out = attn.append_rotated(pool, k, v, *where, rope, q=q, positions=pos)
        assert attn.get_error() == lib.SV_ERR_DATA
        assert torch.isnan(out["q"]).flatten(1).any(1).tolist() == [i == 2 for i in range(7)]


@pytest.mark.parametrize("dtype", [BF16, FOUR])
def test_tokens_without_a_slot_and_rows_of_no_sequence(lib, dtype):
    w, attn, pool, where = world(lib, [6, 5, 3], None, 4, 2, 64, 16, dtype, kv_len=[4, 0, 3], seed=6)
    table = rope_table(10, 32)
    pad = [torch.cat([x, torch.full((3, *x.shape[1:]), 2.0, dtype=BF16)]).cuda() for x in (w.q, w.k_new, w.v_new)]
    out = {"q": torch.full_like(pad[0], 7.0), "k": torch.full_like(pad[1], 7.0)}
    attn.append_rotated(pool, pad[1], pad[2], *where, lib.Rope(table.cuda()), q=pad[0], out=out)
    assert attn.get_error() == lib.SV_OK                      # neither is an error
    pos = positions_of(w)
    for name, x in (("q", w.q), ("k", w.k_new)):
        want = torch.from_numpy(rotate(x.float().numpy(), table, pos.clip(0), False)).bfloat16()
        want[torch.from_numpy(pos < 0)] = 0
        assert torch.equal(out[name][:w.n].cpu(), want) and (out[name][w.n:] == 7).all()
    assert_cached(w, pool, rotate(w.k_new.float().numpy(), table, pos.clip(0), False), w.v_new.float().numpy())
    bad = where[2].clone()
    bad[0, 0] = -1                                            # an invalid page
    out = attn.append_rotated(pool, pad[1][:w.n], pad[2][:w.n], where[0], where[1], bad, lib.Rope(table.cuda()), q=pad[0][:w.n])
    assert attn.get_error() == lib.SV_ERR_DATA
    assert torch.isnan(out["q"]).flatten(1).all(1).tolist() == [2 <= i < 6 for i in range(14)]


def test_values_that_are_not_finite(lib):
    w, attn, pool, where = world(lib, [4], [0], 2, 2, 64, 16, BF16, seed=7)
    table = rope_table(16, 32)
    q, k, v = w.q.clone(), w.k_new.clone(), w.v_new.clone()
    k[1, 0, 3], k[2, 1, 40], v[0, 0, 5], q[3, 0, 17] = float("inf"), float("nan"), float("-inf"), float("nan")
    k[3, 1, 50] = -0.0                                        # behind the rotated part: as it is
    out = attn.append_rotated(pool, k.cuda(), v.cuda(), *where, lib.Rope(table.cuda()), q=q.cuda(), want_k=True)
    pos = np.arange(4)
    for x, got in ((k, out["k"]), (q, out["q"])):
        want = torch.from_numpy(rotate(x.float().numpy(), table, pos, False)).bfloat16()
        assert np.array_equal(got.double().cpu().numpy(), want.double().numpy(), equal_nan=True)
    page = w.table[0, 0]
    assert torch.equal(pool.v[page, :, :4].cpu().transpose(0, 1), v)
    assert pool.k[page, 1, 3, 50].view(torch.int16).item() == -(1 << 15)
    for dtype in (E4M3, FOUR):
        w2, attn, pool, where = world(lib, [4], [0], 2, 2, 64, 16, dtype, seed=7)
        attn.append_rotated(pool, k.cuda(), v.cuda(), *where, lib.Rope(table.cuda()))
        back = attn.read(pool, *where, n_tokens=4)
        assert attn.get_error() == lib.SV_OK
        nan = torch.isnan(back["k"])
        assert nan.all(-1).tolist() == [[False, False], [True, False], [False, True], [False, False]] and nan.any(-1).equal(nan.all(-1))
        assert torch.isnan(back["v"]).all(-1).tolist() == [[True, False]] + [[False, False]] * 3


def test_refusals(lib):
    attn = lib.SpecAttention(8, 2, 64, 4)
    pool = attn.alloc_pool(4, 16, FOUR)
    q = torch.zeros((2, 8, 64), dtype=BF16, device="cuda")
    k = torch.zeros((2, 2, 64), dtype=BF16, device="cuda")
    cu, kv = torch.tensor([0, 2], dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
    where = (cu, kv, torch.zeros((1, 2), dtype=torch.int32, device="cuda"))
    rope = lib.Rope(torch.zeros((4, 64), device="cuda"))
    for bad, kw, what in ((lib.Rope(torch.zeros((4, 64))), {}, "rope is on"), (lib.Rope(torch.zeros((4, 128), device="cuda")), {}, "turns 128"),
                          (rope, dict(positions=torch.zeros(2, device="cuda")), "dtype"), (rope, dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")), "shape"),
                          (rope, dict(q=q[:1]), "shape"), (rope, dict(q=q, out={}), "go together"), (rope, dict(out={"q": q}), "go together"),
                          (rope, dict(want_k=True, out={}), "output k is required"), (rope, dict(q=q, out={"q": q[:, :2]}), "output q"),
                          (rope, dict(q=q, out={"q": q[:1].expand(2, 8, 64)}), "overlap"), (rope, dict(out={"k": k.float()}), "output k")):
        with pytest.raises(ValueError, match=what):
            attn.append_rotated(pool, k, k, *where, bad, **kw)
    with pytest.raises(ValueError, match="pool of"):
        attn.append_rotated(lib.SpecAttention(8, 4, 64, 4).alloc_pool(4, 16), k, k, *where, rope)
    assert attn.get_error() == lib.SV_OK
    empty = torch.zeros((0, 2, 64), dtype=BF16, device="cuda")
    none = (torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    assert attn.append_rotated(pool, empty, empty, *none, rope, q=empty[:, :1].expand(0, 8, 64), want_k=True)["q"].shape == (0, 8, 64)


# ----------------------------------------------------------------- all together
@pytest.mark.parametrize("dtype", [BF16, E4M3, FOUR])
def test_prompt_cache_and_step_in_a_graph(lib, dtype):
    """Prompts rotated into the cache and attended to, then a captured step of 4 rotated tokens:
    the step's rows are those of attention over what the cache reads back as."""
    hq, hkv, d, page, lens, n = 8, 2, 64, 16, [70, 131, 5], 4
    g = torch.Generator(device="cuda").manual_seed(8)
    attn = lib.SpecAttention(hq, hkv, d, 3)
    pool = attn.alloc_pool(40, page, dtype)
    table = torch.randperm(39, generator=g, device="cuda").int().view(3, 13)
    rope = lib.Rope(rope_table(200, d).cuda())
    cu = torch.tensor([0, 70, 201, 206], dtype=torch.int32, device="cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def rows(m):
        return (torch.randn((m, h, d), generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv))

    q, k, v = rows(206)
    turned = attn.append_rotated(pool, k, v, cu, kv, table, rope, q=q, want_k=True)
    attn.prompt(turned["q"], turned["k"], v, cu)
    step_cu = torch.tensor([0, n, 2 * n, 3 * n], dtype=torch.int32, device="cuda")
    q, k, v = rows(3 * n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = {"out": torch.empty_like(q), "lse": torch.empty((3 * n, hq), device="cuda")}
    turned = {"q": torch.empty_like(q)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        attn.append_rotated(pool, k, v, step_cu, kv, table, rope, q=q, out=turned, stream=side)
        attn.attend(pool, turned["q"], step_cu, kv, table, out=out, stream=side)
    for _ in range(2):                                        # two steps: other tokens, longer sequences
        kv += n
        for x, y in zip((q, k, v), rows(3 * n)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert attn.get_error() == lib.SV_OK
        lens = [x + n for x in lens]
        all_cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        back = attn.read(pool, all_cu, kv, table, n_tokens=sum(lens))
        pos = np.concatenate([np.arange(x - n, x) for x in lens])
        assert torch.equal(turned["q"].cpu(), torch.from_numpy(rotate(q.cpu().float().numpy(), rope.table.cpu(), pos, False)).bfloat16())
        parts = []
        for b, x in enumerate(lens):
            kc, vc = (back[name][all_cu[b]:all_cu[b + 1]].double().cpu().numpy() for name in ("k", "v"))
            parts.append((_attn if dtype == BF16 else _attn4).attention(turned["q"][b * n:b * n + n].double().cpu().numpy(), kc, vc, d ** -0.5, [x - n + i + 1 for i in range(n)]))
        _attn.assert_attention(out["out"], out["lse"], [np.concatenate([p[i] for p in parts]) for i in range(4)])
