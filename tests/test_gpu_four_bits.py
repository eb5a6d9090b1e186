"""4-bit caches against the float64 definitions: append and read bit for bit, and
attention over ragged, empty, long and wrong batches."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import _attn, _attn4  # noqa: E402
from tests._attn import assert_attention  # noqa: E402
from tests._attn4 import FOUR, World4, bytes_of, quantise4, values4  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    return sv


def setup(lib, w):
    return lib.SpecAttention(w.hq, w.hkv, w.d, max(1, len(w.new))), *w.pool(lib)


def attend(lib, w, **kw):
    attn, pool, where = setup(lib, w)
    out = attn.attend(pool, w.q.cuda(), *where, want_lse=True, **kw)
    assert attn.get_error() == lib.SV_OK
    return out["out"], out["lse"]


# ------------------------------------------------------------ append and read
SHAPES = [  # new, old, hkv, d, page
    ([1], [0], 1, 64, 16),
    ([1, 1, 1], [0, 15, 16], 2, 128, 16),
    ([8, 0, 5, 8], [3, 9, 60, 61], 8, 128, 16),
    ([33, 130, 1], [31, 0, 257], 3, 64, 32),
    ([16, 16], [100, 127], 4, 128, 64),
    ([300], [7], 1, 128, 128),
    ([700], [5], 5, 64, 16),
]


def written(w, x, name):
    """The world's bytes of cache `name` after x [n, heads, D] (float64) is appended."""
    raw = {part: w.raw[name + part].clone() for part in ("", "_block", "_scale")}
    c, s, e = quantise4(x)
    for b, n in enumerate(w.new):
        for i in range(n):
            t, pos = w.cu[b] + i, w.kv[b] - n + i
            at = (w.table[b, pos // w.page], slice(None), pos % w.page)
            raw[""][at], raw["_block"][at], raw["_scale"][at] = (torch.from_numpy(y[t]) for y in (c, s, e))
    return raw


@pytest.mark.parametrize("new, old, hkv, d, page", SHAPES)
def test_append_writes_its_slots_and_no_others(lib, new, old, hkv, d, page):
    w = World4(new, old, hkv, hkv, d, page, seed=1)
    attn, pool, where = setup(lib, w)
    fused = torch.zeros((w.n, 3 * hkv, d), dtype=BF16, device="cuda")      # strided: slices of one tensor
    fused[:, hkv:2 * hkv], fused[:, 2 * hkv:] = w.k_new.cuda(), w.v_new.cuda()
    attn.append(pool, fused[:, hkv:2 * hkv], fused[:, 2 * hkv:], *where)
    assert attn.get_error() == lib.SV_OK
    got = bytes_of(pool)
    for name, x in (("k", w.k_new), ("v", w.v_new)):
        for part, want in written(w, x.double().numpy(), name).items():
            assert torch.equal(got[name + part], want), name + part


@pytest.mark.parametrize("new, old, hkv, d, page", SHAPES)
def test_read_gives_the_cached_values(lib, new, old, hkv, d, page):
    w = World4(new, old, hkv, hkv, d, page, seed=2)
    attn, pool, where = setup(lib, w)
    out = attn.read(pool, *where, n_tokens=w.n)
    assert attn.get_error() == lib.SV_OK
    for name, cached in (("k", w.kc), ("v", w.vc)):
        ref = np.concatenate([x[w.kv[b] - n:] for b, (x, n) in enumerate(zip(cached, new))])
        assert np.array_equal(out[name].double().cpu().numpy(), ref)       # exact in bf16: 2 bits times 4


@pytest.mark.parametrize("d", [64, 128])
def test_quantiser_extremes(lib, d):
    x = torch.zeros((14, 1, d), dtype=BF16)
    x[1] = 1e-38
    x[2, 0, 3] = float("inf")
    x[3, 0, 9] = float("nan")
    x[4, 0, :3] = torch.tensor([3e38, -3e38, 1.0])
    x[5] = torch.arange(d) * 2.0 ** -3
    x[6], x[6, 0, 0] = 2688.0, -2704.0
    x[7] = torch.linspace(-1, 1, d)
    x[8, 0, 5] = 2.0 ** -133                                     # bf16 subnormal
    for i, m in enumerate((15.0, 13.0, 11.0, 9.0)):              # ties between codes, whatever the scale's bits
        x[9 + i] = (torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * m).repeat(d // 8)
        x[9 + i, 0, 1::2] *= -1
    x[13, 0, :16], x[13, 0, 16:32], x[13, 0, 32:48] = 1.0, 2.0 ** -18, 2.0 ** -19      # blocks that keep no scale
    w = World4([14], [0], 1, 1, d, 16)
    attn, pool, where = setup(lib, w)
    attn.append(pool, x.cuda(), x.cuda(), *where)
    out = attn.read(pool, *where, n_tokens=14)
    want = quantise4(x.double().numpy())
    got, page = bytes_of(pool), w.table[0, 0]
    for part, y in zip(("", "_block", "_scale"), want):
        for name in ("k", "v"):
            assert np.array_equal(got[name + part][page, 0, :14].numpy(), y[:, 0]), name + part
    ref = torch.from_numpy(values4(*want)).float().bfloat16()
    assert np.array_equal(out["v"].double().cpu().numpy(), ref.double().numpy(), equal_nan=True)


@pytest.mark.parametrize("shift", [0, -100, 100])
def test_every_scale(lib, shift):
    """Blocks that take each of the 126 scales above 0, with ties between codes and other values under it, by append
    and by the append that rotates (by nothing), which quantise in different ways."""
    g = np.random.default_rng(5)
    scales = _attn.e4m3_value(np.arange(1, 127, dtype=np.uint8)).reshape(18, 7)
    x = np.zeros((18, 1, 8, 16))
    x[:, 0, 7] = 2688.0 * np.where(g.random((18, 16)) < 0.5, 1, -1)                 # makes the exponent 0
    x[:, 0, :7, 0] = 6 * scales
    x[:, 0, :7, 1:8] = scales[..., None] * np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x[:, 0, :7, 8:] = scales[..., None] * g.uniform(-6, 6, (18, 7, 8))
    x = (torch.from_numpy(x.reshape(18, 1, 128)) * 2.0 ** shift).bfloat16()
    want = quantise4(x.double().numpy())
    assert np.array_equal(want[1][:, 0, :7].reshape(-1), np.arange(1, 127)) and (want[2] == 127 + shift).all()
    w = World4([18], [0], 1, 1, 128, 32)
    attn, pool, where = setup(lib, w)
    rope = lib.Rope(torch.cat([torch.ones((18, 64)), torch.zeros((18, 64))], 1).cuda())
    for call in (lambda: attn.append(pool, x.cuda(), x.cuda(), *where), lambda: attn.append_rotated(pool, x.cuda(), x.cuda(), *where, rope)):
        pool.k.view(torch.uint8).zero_(), pool.v.view(torch.uint8).zero_()
        call()
        assert attn.get_error() == lib.SV_OK
        got, page = bytes_of(pool), w.table[0, 0]
        for part, y in zip(("", "_block", "_scale"), want):
            for name in ("k", "v"):
                assert np.array_equal(got[name + part][page, 0, :18].numpy(), y[:, 0]), name + part


def test_tokens_before_the_first_position(lib):
    """kv_len below the number of new tokens: the first ones have no slot."""
    w = World4([6, 5, 3], None, 4, 2, 64, 16, kv_len=[4, 0, 3], seed=3)
    attn, pool, where = setup(lib, w)
    out = attn.read(pool, *where, n_tokens=w.n)
    ref = np.zeros((w.n, 2, 64))
    ref[2:6], ref[11:] = w.kc[0], w.kc[2]
    assert np.array_equal(out["k"].double().cpu().numpy(), ref)
    got = attn.attend(pool, w.q.cuda(), *where, want_lse=True)
    assert_attention(got["out"], got["lse"], w.expect_attention())
    before = bytes_of(pool)
    attn.append(pool, w.k_new.cuda(), w.v_new.cuda(), *where)
    assert attn.get_error() == lib.SV_OK
    after = bytes_of(pool)
    assert 0 < (after["k"] != before["k"]).any(-1).any(1).sum() <= 7     # 4 + 0 + 3 slots


# ------------------------------------------------------------------ attention
CASES = [  # new, old, hq, hkv, d, page
    ([1], [0], 1, 1, 64, 16),
    ([1], [31], 8, 1, 128, 16),
    ([1, 1, 1, 1], [0, 15, 16, 300], 32, 8, 128, 16),
    ([1, 1], [126, 127], 8, 8, 64, 32),
    ([1, 1, 1], [128, 640, 33], 8, 1, 64, 64),
    ([2, 1], [1000, 95], 16, 2, 128, 128),
    ([2], [513], 7, 1, 128, 32),
    ([4, 0, 3], [250, 9, 31], 32, 4, 64, 16),
    ([4, 4], [1, 2000], 8, 1, 128, 64),
    ([5, 3], [511, 65], 10, 2, 128, 16),
    ([1, 1], [700, 64], 48, 2, 128, 32),
    ([1], [300], 31, 1, 64, 16),
    ([8, 8, 8], [0, 120, 121], 64, 8, 128, 32),
    ([16, 16], [240, 1000], 64, 8, 128, 64),
    ([5, 0, 3, 1], [130, 50, 0, 511], 28, 4, 64, 16),
    ([9, 2], [64, 255], 16, 1, 128, 128),
    ([40, 7], [10, 128], 15, 3, 128, 64),
    ([130], [70], 10, 2, 64, 64),
    ([129, 257, 64], [0, 130, 700], 4, 1, 128, 128),
    ([3, 12], [300, 90], 64, 1, 128, 16),
    ([1], [4000], 2, 1, 128, 16),
    ([8] * 40, list(range(0, 400, 10)), 8, 2, 64, 16),
    ([1] * 150, list(range(0, 750, 5)), 8, 1, 64, 32),
    ([3] * 30, list(range(0, 1500, 50)), 16, 4, 128, 16),
    ([100], [1000], 4, 4, 128, 16),
    ([3] * 140, list(range(0, 560, 4)), 16, 2, 64, 16),            # more sequences than a warp plans by itself
]


@pytest.mark.parametrize("new, old, hq, hkv, d, page", CASES)
def test_attend(lib, new, old, hq, hkv, d, page):
    w = World4(new, old, hq, hkv, d, page, seed=4)
    assert_attention(*attend(lib, w), w.expect_attention())


@pytest.mark.parametrize("new", [[7, 1, 20], [1, 1, 2]])
def test_attend_without_causality_and_another_scale(lib, new):
    w = World4(new, [0, 200, 130], 12, 4, 128, 32, seed=5)
    assert_attention(*attend(lib, w, causal=False, scale=0.3), w.expect_attention(causal=False, scale=0.3))
    w = World4([4, 3, 2], None, 12, 4, 64, 32, kv_len=[0, 1, 140], seed=6)      # an empty sequence
    assert_attention(*attend(lib, w, causal=False), w.expect_attention(causal=False))


@pytest.mark.parametrize("new", [[8, 64], [1, 2], [4, 4]])
def test_peaked_scores_and_vectors_of_different_size(lib, new):
    w = World4(new, [500, 300], 16, 2, 128, 16, seed=7, spread=1.5)
    assert_attention(*attend(lib, w, scale=0.5), w.expect_attention(scale=0.5))


@pytest.mark.parametrize("new", [[1], [4], [12], [40]])
def test_vectors_far_apart_in_size(lib, new):
    w = World4(new, [520], 8, 2, 64, 16, seed=8)
    for name, cached in (("k", w.kc), ("v", w.vc)):
        for p in range(0, w.kv[0], 3):
            page, slot = w.table[0, p // 16], p % 16
            shift = -60 if p % 2 else (0 if name == "k" else 20)
            w.raw[name + "_scale"][page, :, slot] = (w.raw[name + "_scale"][page, :, slot].int() + shift).to(torch.uint8)
            cached[0][p] *= 2.0 ** shift
    assert_attention(*attend(lib, w), w.expect_attention())


def packed(lib, hq, k, v, q, page=32, causal=True):
    """Sequences of bf16 keys and values [tokens, heads, D] through append, and their last tokens' rows."""
    hkv, d, lens = k[0].shape[1], k[0].shape[2], [len(x) for x in k]
    need = [-(-n // page) for n in lens]
    attn = lib.SpecAttention(hq, hkv, d, len(k))
    pool = attn.alloc_pool(sum(need) + 1, page, FOUR)
    order = np.random.default_rng(0).permutation(sum(need) + 1)
    table = np.zeros((len(k), max(need)), np.int32)
    for b, c in enumerate(need):
        table[b, :c] = order[sum(need[:b]):sum(need[:b]) + c]
    cu, kv_len, new = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in
                       (np.concatenate([[0], np.cumsum(lens)]), lens, np.concatenate([[0], np.cumsum([len(x) for x in q])])))
    table = torch.from_numpy(table).cuda()
    attn.append(pool, torch.cat(k).cuda(), torch.cat(v).cuda(), cu, kv_len, table)
    got = attn.attend(pool, torch.cat(q).cuda(), new, kv_len, table, causal=causal, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    parts = []
    for b, x in enumerate(q):
        n, kv = len(x), len(k[b])
        kc, vc = (values4(*quantise4(y[b].double().numpy())) for y in (k, v))
        parts.append(_attn4.attention(x.double().numpy(), kc, vc, d ** -0.5, [kv - n + i + 1 if causal else kv for i in range(n)]))
    assert_attention(got["out"], got["lse"], [np.concatenate([p[i] for p in parts]) for i in range(4)])


def normal(g, *shape):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).bfloat16()


@pytest.mark.parametrize("n", [1, 4, 20])
@pytest.mark.parametrize("zero_keys", [True, False])
@pytest.mark.parametrize("lens", [[130], [1000, 40], [300] * 12])
def test_values_that_are_all_zero(lib, lens, zero_keys, n):
    g = np.random.default_rng(1)
    k = [normal(g, x, 2, 64) * (0 if zero_keys else 1) for x in lens]
    packed(lib, 8, k, [torch.zeros_like(x) for x in k], [normal(g, n, 8, 64) for _ in lens])


@pytest.mark.parametrize("n", [1, 4, 20])
@pytest.mark.parametrize("size", [2.0 ** -100, 1.0, 2.0 ** 90])
@pytest.mark.parametrize("zeros", [(0, 260), (0, 640), (300, 700)])
def test_stretches_of_zero_values_beside_others(lib, zeros, size, n):
    g = np.random.default_rng(2)
    k, v = normal(g, 900, 2, 128), normal(g, 900, 2, 128) * size
    v[zeros[0]:zeros[1]] = 0
    packed(lib, 8, [k], [v], [normal(g, n, 8, 128)])


@pytest.mark.parametrize("n", [1, 3, 30])
@pytest.mark.parametrize("factor", [2.0 ** 40, 2.0 ** -40])
def test_an_outsized_token(lib, factor, n):
    """One token's values of another size, and the same of its key where that leaves the scores in range."""
    g = np.random.default_rng(3)
    for at in (0, 130, 898):
        k, v = normal(g, 900, 2, 64), normal(g, 900, 2, 64)
        v[at] *= factor
        k[at] *= min(1.0, factor)
        packed(lib, 4, [k], [v], [normal(g, n, 4, 64)])


@pytest.mark.parametrize("hq, hkv, d", [(16, 2, 128), (6, 2, 64), (4, 4, 64)])
@pytest.mark.parametrize("new, old", [([150, 3], [40, 300]), ([8, 8], [250, 500]), ([3, 2], [30, 125]), ([400], [700])])
def test_later_tokens_of_nan_leave_earlier_rows_alone(lib, new, old, hq, hkv, d):
    w = World4(new, old, hq, hkv, d, 32, seed=14)
    expected = w.expect_attention()
    attn, pool, where = setup(lib, w)
    at = [max(1, n // 2) for n in new]                       # new token of each sequence with bad vectors
    for b, i in enumerate(at):
        pos = w.kv[b] - new[b] + i
        page, slot = w.table[b, pos // 32], pos % 32
        pool.k_scale[page, :, slot] = pool.v_scale[page, :, slot] = 255
    got = attn.attend(pool, w.q.cuda(), *where, want_lse=True)
    again = attn.attend(pool, w.q.cuda(), *where, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    assert torch.equal(got["out"].view(torch.int16), again["out"].view(torch.int16))
    for b, i in enumerate(at):
        clean = slice(w.cu[b], w.cu[b] + i)
        assert_attention(got["out"][clean], got["lse"][clean], [x[clean] for x in expected])
        assert torch.isnan(got["out"][w.cu[b] + i:w.cu[b + 1]]).all()      # they see a key of NaN


@pytest.mark.parametrize("n", [1, 4, 40])
def test_values_of_nan_reach_the_rows_that_see_them_and_their_columns(lib, n):
    w = World4([n], [300], 8, 2, 64, 16, seed=15)
    ref = w.expect_attention()
    attn, pool, where = setup(lib, w)
    for pos, block in ((17, 1), (w.kv[0] - max(1, n // 2), 3)):          # a scale of NaN: 16 columns of one token
        pool.v_block.view(torch.uint8)[w.table[0, pos // 16], :, pos % 16, block] = 0x7f
    got = attn.attend(pool, w.q.cuda(), *where, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    out = got["out"].double().cpu().numpy()
    assert np.isnan(out[:, :, 16:32]).all()
    seen = np.arange(n) >= n - max(1, n // 2)
    assert np.isnan(out[seen][:, :, 48:]).all()
    out[:, :, 16:32], out[seen, :, 48:] = ref[0][:, :, 16:32], ref[0][seen][:, :, 48:]
    assert_attention(torch.from_numpy(out), got["lse"], ref)


# ------------------------------------------- streams, graphs, repeats, long ones
@pytest.mark.parametrize("new", [[8, 1, 30], [1, 1, 1], [2, 2, 1]])
def test_calls_repeat_bit_for_bit_and_in_a_graph_on_another_stream(lib, new):
    w = World4(new, [900, 2500, 33], 16, 2, 128, 32, seed=11)
    attn, pool, where = setup(lib, w)
    q = w.q.cuda()
    first = attn.attend(pool, q, *where, want_lse=True)
    out = {name: torch.zeros_like(t) for name, t in first.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    attn.attend(pool, q, *where, out=out, stream=side)
    side.synchronize()
    assert all(torch.equal(out[name], first[name]) for name in first)
    graph = torch.cuda.CUDAGraph()
    k, v = w.k_new.cuda(), w.v_new.cuda()
    with torch.cuda.graph(graph, stream=side):
        attn.append(pool, k, v, *where, stream=side)
        attn.attend(pool, q, *where, out=out, stream=side)
    q.copy_(torch.randn_like(q))                    # new inputs in the captured buffers
    for _ in range(3):
        out["out"].zero_()
        graph.replay()
    torch.cuda.synchronize()
    fresh = attn.attend(pool, q, *where, want_lse=True)
    assert all(torch.equal(out[name], fresh[name]) for name in first)
    assert attn.get_error() == lib.SV_OK


@pytest.mark.parametrize("hq, n", [(64, 16), (64, 8), (64, 1), (32, 1), (32, 5), (16, 200), (40, 3), (128, 2)])
def test_long_ragged_contexts_from_cold_memory(lib, hq, n):
    """Runs of dozens of blocks whose copies keep the products waiting, against a
    float64 softmax on the GPU, with the same bits every time."""
    seqs, hkv, d, page = (24 if n < 100 else 3), 8, 128, 32
    g = torch.Generator(device="cuda").manual_seed(16)
    r = np.random.default_rng(16)
    kv = [int(x) for x in r.integers(max(300, n), 5000, seqs)]
    need = [-(-x // page) for x in kv]
    order = torch.randperm(sum(need), generator=g, device="cuda").int()
    table = torch.zeros((seqs, max(need)), dtype=torch.int32, device="cuda")
    for b, c in enumerate(need):
        table[b, :c] = order[sum(need[:b]):sum(need[:b]) + c]
    attn = lib.SpecAttention(hq, hkv, d, seqs)
    pool = attn.alloc_pool(sum(need), page, FOUR)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(kv)]), dtype=torch.int32, device="cuda")
    kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((sum(kv), hkv, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    attn.append(pool, k, v, cu, kv_len, table)
    back = attn.read(pool, cu, kv_len, table, n_tokens=sum(kv))          # as the cache holds them
    q = torch.randn((seqs * n, hq, d), generator=g, device="cuda").bfloat16()
    new = torch.arange(0, seqs * n + 1, n, dtype=torch.int32, device="cuda")
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(3):
        cold.zero_()
        got.append(attn.attend(pool, q, new, kv_len, table, want_lse=True))
    assert attn.get_error() == lib.SV_OK
    assert all(torch.equal(x[name], got[0][name]) for x in got for name in x)
    for b in range(seqs):
        rows, lo, hi = slice(b * n, b * n + n), sum(kv[:b]), sum(kv[:b + 1])
        kk, vv = (back[x][lo:hi].double().repeat_interleave(hq // hkv, 1) for x in ("k", "v"))
        s = torch.einsum("nhd,lhd->nhl", q[rows].double(), kk) * d ** -0.5
        last = kv[b] - n + torch.arange(n, device="cuda")
        s.masked_fill_(torch.arange(kv[b], device="cuda")[None, None] > last[:, None, None], -float("inf"))
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[..., None])
        ref, spread = torch.einsum("nhl,lhd->nhd", p, vv), torch.einsum("nhl,lhd->nhd", p, vv.abs())
        # the bounds of tests/_attn.py, and of weights in f16 (tests/_attn4.py)
        top = vv.abs().amax(-1, keepdim=True)
        floor = 2.0 ** -23 * (p * top[:, :, 0].T[None]).amax(-1)[..., None] * (vv.abs() / top).sum(0)
        assert ((got[0]["out"][rows].double() - ref).abs() <= 2.0 ** -9 * ref.abs() + 2.0 ** -8 * spread + floor).all()
        reach = torch.einsum("nhd,lhd->nhl", q[rows].double().abs(), kk.abs()).amax(-1) * d ** -0.5
        assert ((got[0]["lse"][rows].double() - lse).abs() <= 2.0 ** -16 * (1 + reach)).all()


@pytest.mark.parametrize("new", [[8, 1], [1, 1]])
def test_offsets_beyond_32_bits(lib, new):
    """Pages whose byte offsets pass 2^32."""
    hkv, d, page = 8, 128, 128
    pages = (1 << 32) // (hkv * page * d // 2) + 8           # 4.3 GB a tensor
    w = World4(new, [200, 140], 16, hkv, d, page, seed=12)
    attn = lib.SpecAttention(16, hkv, d, 2)
    high = pages - w.num_pages
    big = {}
    for name, t in w.raw.items():
        big[name] = torch.empty((pages, *t.shape[1:]), dtype=torch.uint8, device="cuda")
        big[name][high:] = t.cuda()
    e4m3 = torch.float8_e4m3fn
    pool = lib.KVPool(big["k"].view(FOUR), big["v"].view(FOUR), big["k_scale"], big["v_scale"], big["k_block"].view(e4m3), big["v_block"].view(e4m3))
    _, (cu, kv_len, table) = w.pool(lib)
    where = (cu, kv_len, table + high)
    got = attn.attend(pool, w.q.cuda(), *where, want_lse=True)
    assert_attention(got["out"], got["lse"], w.expect_attention())
    attn.append(pool, w.k_new.cuda(), w.v_new.cuda(), *where)
    back = attn.read(pool, *where, n_tokens=w.n)
    assert attn.get_error() == lib.SV_OK
    assert np.array_equal(back["v"].double().cpu().numpy(), values4(*quantise4(w.v_new.double().numpy())))


# ----------------------------------------------------------- wrong metadata
@pytest.mark.parametrize("new", [[8, 4, 2], [2, 1, 1]])
def test_wrong_metadata_is_reported_and_stays_in_bounds(lib, new):
    w = World4(new, [100, 30, 12], 8, 2, 64, 16, seed=13)
    good = w.expect_attention()
    attn, pool, (cu, kv_len, table) = setup(lib, w)
    q = w.q.cuda()
    rows = {b: slice(w.cu[b], w.cu[b + 1]) for b in range(3)}

    def check(where, bad):
        got = attn.attend(pool, q, *where, want_lse=True)
        assert attn.get_error() == lib.SV_ERR_DATA
        assert attn.get_error() == lib.SV_OK
        for b, s in rows.items():
            if b in bad:
                assert torch.isnan(got["out"][s]).all() and torch.isnan(got["lse"][s]).all()
            else:
                assert_attention(got["out"][s], got["lse"][s], [x[s] for x in good])

    for page in (-1, w.num_pages, 1 << 30):
        t = table.clone()
        t[0, 3] = page
        check((cu, kv_len, t), [0])
    for length in (-1, table.shape[1] * 16 + 1):
        n = kv_len.clone()
        n[1] = length
        check((cu, n, table), [1])
    t = table.clone()
    t[0, (w.kv[0] - 1) // 16] = -5                  # the page of sequence 0's newest token
    before = bytes_of(pool)["k"]
    attn.append(pool, w.k_new.cuda(), w.v_new.cuda(), cu, kv_len, t)
    assert attn.get_error() == lib.SV_ERR_DATA
    pages = [p for p in range(w.num_pages) if p not in table.flatten().tolist()]
    assert torch.equal(bytes_of(pool)["k"][pages], before[pages])
    out = attn.read(pool, cu, kv_len, t, n_tokens=w.n)
    assert attn.get_error() == lib.SV_ERR_DATA
    last = int(w.cu[1]) - 1
    assert torch.isnan(out["k"][last]).all() and torch.isfinite(out["k"][last + 1:]).all()
    for bad_cu in ([0, 9, 5, w.n], [-3, new[0], new[0] + new[1], w.n], [0, new[0], new[0] + new[1], 99]):
        attn.attend(pool, q, torch.tensor(bad_cu, dtype=torch.int32, device="cuda"), kv_len, table)
        assert attn.get_error() == lib.SV_ERR_DATA


def test_rows_of_no_sequence_are_not_written(lib):
    for n in (1, 6):
        w = World4([n, n], [40, 300], 8, 2, 64, 16, seed=17)
        attn, pool, where = setup(lib, w)
        q = torch.cat([w.q, torch.full((5, 8, 64), float("nan"), dtype=BF16)]).cuda()
        out = {"out": torch.full((w.n + 5, 8, 64), 7.0, dtype=BF16, device="cuda"), "lse": torch.full((w.n + 5, 8), 7.0, device="cuda")}
        attn.attend(pool, q, *where, out=out)
        kv = torch.full((w.n + 5, 2, 64), float("nan"), dtype=BF16, device="cuda")
        kv[:w.n] = w.k_new.cuda()
        assert (out["out"][w.n:] == 7).all() and (out["lse"][w.n:] == 7).all()
        assert_attention(out["out"][:w.n], out["lse"][:w.n], w.expect_attention())
        attn.append(pool, kv, kv, *where)
        assert attn.get_error() == lib.SV_OK
        assert np.array_equal(bytes_of(pool)["k"].numpy(), written(w, w.k_new.double().numpy(), "k")[""].numpy())


def test_no_sequences_and_no_tokens(lib):
    attn = lib.SpecAttention(8, 2, 64, 4)
    pool = attn.alloc_pool(4, 16, FOUR)
    q = torch.zeros((0, 8, 64), dtype=BF16, device="cuda")
    kv = q[:, :2]
    cu, none = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    table = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    assert attn.attend(pool, q, cu, none, table, want_lse=True)["out"].shape == (0, 8, 64)
    attn.append(pool, kv, kv, cu, none, table)
    assert attn.read(pool, cu, none, table, n_tokens=0)["k"].shape == (0, 2, 64)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")              # sequences without tokens
    attn.attend(pool, q, cu, torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros((2, 1), dtype=torch.int32, device="cuda"))
    assert attn.get_error() == lib.SV_OK
    q = torch.ones((2, 8, 64), dtype=BF16, device="cuda")              # an empty cache: nothing is seen
    got = attn.attend(pool, q, torch.tensor([0, 2], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                      torch.zeros((1, 0), dtype=torch.int32, device="cuda"), want_lse=True)
    assert not got["out"].any() and torch.isneginf(got["lse"]).all() and attn.get_error() == lib.SV_OK
