"""Cache and attention kernels against the float64 definitions: ragged and empty
sequences, pages that end inside a tile, stale slots that hold NaN, grouped
heads, strided inputs, quantised pools, long splits, wrong metadata."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import _attn  # noqa: E402
from tests._attn import World, assert_attention  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    return sv


def setup(lib, w):
    attn = lib.SpecAttention(w.hq, w.hkv, w.d, max(1, len(w.new)))
    tensors, cu, kv_len, table = w.to("cuda")
    return attn, lib.KVPool(tensors["k"], tensors["v"], tensors["k_scale"], tensors["v_scale"]), (cu, kv_len, table)


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
]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("new, old, hkv, d, page", SHAPES)
def test_append_writes_its_slots_and_no_others(lib, new, old, hkv, d, page, dtype):
    w = World(new, old, hkv, hkv, d, page, dtype, seed=1)
    attn, pool, where = setup(lib, w)
    fused = torch.zeros((w.n, 3 * hkv, d), dtype=BF16, device="cuda")      # strided: slices of one tensor
    fused[:, hkv:2 * hkv], fused[:, 2 * hkv:] = w.k_new.cuda(), w.v_new.cuda()
    attn.append(pool, fused[:, hkv:2 * hkv], fused[:, 2 * hkv:], *where)
    assert attn.get_error() == lib.SV_OK
    for name, x in (("k", w.k_new), ("v", w.v_new)):
        codes, scales = w.codes[name].clone(), None if w.scales[name] is None else w.scales[name].clone()
        c, s = _attn.quantise(x.double().numpy()) if dtype == E4M3 else (None, None)
        for b, n in enumerate(new):
            for i in range(n):
                t, pos = w.cu[b] + i, w.kv[b] - n + i
                page_id, slot = w.table[b, pos // page], pos % page
                if dtype == BF16:
                    codes[page_id, :, slot] = x[t]
                else:
                    codes.view(torch.uint8)[page_id, :, slot] = torch.from_numpy(c[t])
                    scales[page_id, :, slot] = torch.from_numpy(s[t])
        bits = torch.int16 if dtype == BF16 else torch.uint8
        assert torch.equal(getattr(pool, name).view(bits).cpu(), codes.view(bits))
        if scales is not None:
            assert torch.equal(getattr(pool, name + "_scale").cpu(), scales)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("new, old, hkv, d, page", SHAPES)
def test_read_gives_the_cached_values(lib, new, old, hkv, d, page, dtype):
    w = World(new, old, hkv, hkv, d, page, dtype, seed=2)
    attn, pool, where = setup(lib, w)
    out = attn.read(pool, *where, n_tokens=w.n)
    assert attn.get_error() == lib.SV_OK
    for name, cached in (("k", w.kc), ("v", w.vc)):
        ref = np.concatenate([x[w.kv[b] - n:] for b, (x, n) in enumerate(zip(cached, new))])
        assert np.array_equal(out[name].double().cpu().numpy(), ref)       # exact in bf16


def test_quantiser_extremes(lib):
    d = 64
    x = torch.zeros((10, 1, d), dtype=BF16)
    x[1] = 1e-38
    x[2, 0, 3] = float("inf")
    x[3, 0, 9] = float("nan")
    x[4, 0, :3] = torch.tensor([3e38, -3e38, 1.0])
    x[5] = torch.arange(d) * 2.0 ** -3
    x[6], x[6, 0, 0] = 448.0, -449.0 - 63.0
    x[7] = torch.linspace(-1, 1, d)
    x[8, 0, 5] = 2.0 ** -133                      # bf16 subnormal
    x[9], x[9, 0, 0] = 17.0 * 2.0 ** -12, 448.0    # ties between codes
    w = World([10], [0], 1, 1, d, 16, E4M3)
    attn, pool, where = setup(lib, w)
    attn.append(pool, x.cuda(), x.cuda(), *where)
    out = attn.read(pool, *where, n_tokens=10)
    codes, scale = _attn.quantise(x.double().numpy())
    slots = w.table[0, 0]
    assert np.array_equal(pool.k.view(torch.uint8)[slots, 0, :10].cpu().numpy(), codes[:, 0])
    assert np.array_equal(pool.k_scale[slots, 0, :10].cpu().numpy(), scale[:, 0])
    ref = _attn.e4m3_value(codes) * 2.0 ** (scale.astype(np.float64) - 127)[..., None]
    ref = torch.from_numpy(ref).float().bfloat16()
    assert np.array_equal(out["v"].double().cpu().numpy(), ref.double().numpy(), equal_nan=True)


def test_tokens_before_the_first_position(lib):
    """kv_len below the number of new tokens: the first ones have no slot."""
    for dtype in (BF16, E4M3):
        w = World([6, 5, 3], None, 4, 2, 64, 16, dtype, kv_len=[4, 0, 3], seed=3)
        attn, pool, where = setup(lib, w)
        out = attn.read(pool, *where, n_tokens=w.n)
        ref = np.zeros((w.n, 2, 64))
        ref[2:6], ref[11:] = w.kc[0], w.kc[2]
        assert np.array_equal(out["k"].double().cpu().numpy(), ref)
        before = [t.clone() for t in (pool.k.view(torch.uint8), pool.v.view(torch.uint8))]
        got = attn.attend(pool, w.q.cuda(), *where, want_lse=True)
        assert_attention(got["out"], got["lse"], w.expect_attention())
        attn.append(pool, w.k_new.cuda(), w.v_new.cuda(), *where)
        assert attn.get_error() == lib.SV_OK
        changed = (pool.k.view(torch.uint8) != before[0]).any(-1).any(1).sum().item()
        assert 0 < changed <= 7                     # 4 + 0 + 3 slots


# ------------------------------------------------------------------ attention
CASES = [  # new, old, hq, hkv, d, page
    ([1], [0], 1, 1, 64, 16),
    ([1, 1, 1, 1], [0, 15, 16, 300], 32, 8, 128, 16),
    ([1, 1], [126, 127], 8, 8, 64, 32),
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
]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("new, old, hq, hkv, d, page", CASES)
def test_attend(lib, new, old, hq, hkv, d, page, dtype):
    w = World(new, old, hq, hkv, d, page, dtype, seed=4)
    assert_attention(*attend(lib, w), w.expect_attention())


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_attend_without_causality_and_another_scale(lib, dtype):
    w = World([7, 1, 20], [0, 200, 130], 12, 4, 128, 32, dtype, seed=5)
    assert_attention(*attend(lib, w, causal=False, scale=0.3), w.expect_attention(causal=False, scale=0.3))
    w = World([4, 3, 2], None, 12, 4, 64, 32, dtype, kv_len=[0, 1, 140], seed=6)      # an empty sequence
    assert_attention(*attend(lib, w, causal=False), w.expect_attention(causal=False))


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_peaked_scores_and_vectors_of_different_size(lib, dtype):
    w = World([8, 64], [500, 300], 16, 2, 128, 16, dtype, seed=7, spread=1.5)
    assert_attention(*attend(lib, w, scale=0.5), w.expect_attention(scale=0.5))


def test_quantised_vectors_far_apart_in_size(lib):
    """Scale bytes that differ by more than a 16-bit float's range inside one tile."""
    w = World([4], [120], 8, 2, 64, 16, E4M3, seed=8)
    for name, cached in (("k", w.kc), ("v", w.vc)):
        for p in range(0, w.kv[0], 3):
            page, slot = w.table[0, p // 16], p % 16
            shift = -60 if p % 2 else (0 if name == "k" else 20)
            w.scales[name][page, :, slot] = (w.scales[name][page, :, slot].int() + shift).to(torch.uint8)
            cached[0][p] *= 2.0 ** shift
    assert_attention(*attend(lib, w), w.expect_attention())


PROMPTS = [  # lengths, hq, hkv, d
    ([1], 1, 1, 64),
    ([1, 2, 3], 8, 8, 64),
    ([37, 0, 200, 128], 8, 2, 128),
    ([129, 127, 5], 28, 4, 64),
    ([513], 4, 1, 128),
    ([300, 1, 301], 15, 3, 128),
    ([64] * 20, 16, 1, 64),
]


@pytest.mark.parametrize("lengths, hq, hkv, d", PROMPTS)
def test_prompt(lib, lengths, hq, hkv, d):
    w = World(lengths, [0] * len(lengths), hq, hkv, d, 16, BF16, seed=9)
    attn = lib.SpecAttention(hq, hkv, d, len(lengths))
    for b, n in enumerate(lengths):
        w.kc[b], w.vc[b] = (x[w.cu[b]:w.cu[b + 1]].double().numpy() for x in (w.k_new, w.v_new))
    fused = torch.cat([w.q, w.k_new, w.v_new], 1).cuda()               # strided: slices of one tensor
    q, k, v = fused.split([hq, hkv, hkv], 1)
    got = attn.prompt(q, k, v, torch.from_numpy(w.cu).cuda(), want_lse=True)
    assert attn.get_error() == lib.SV_OK
    assert_attention(got["out"], got["lse"], w.expect_attention())
    heads_first = [x.transpose(0, 1).contiguous().cuda().transpose(0, 1) for x in (w.q, w.k_new, w.v_new)]
    again = attn.prompt(*heads_first, torch.from_numpy(w.cu).cuda(), want_lse=True)
    assert torch.equal(again["out"], got["out"]) and torch.equal(again["lse"], got["lse"])


def test_one_path_from_prompt_to_verification_step(lib):
    """Prompt, cache, then a step of 8 new tokens: the cached step equals the prompt of all tokens."""
    hq, hkv, d, lens, k = 8, 2, 128, [70, 131], 8
    w = World([n + k for n in lens], [0, 0], hq, hkv, d, 16, BF16, seed=10)
    attn = lib.SpecAttention(hq, hkv, d, 2)
    pool = attn.alloc_pool(w.num_pages, 16)
    table = torch.from_numpy(w.table).cuda()
    q, kk, vv = (x.cuda() for x in (w.q, w.k_new, w.v_new))
    whole = attn.prompt(q, kk, vv, torch.from_numpy(w.cu).cuda())["out"]
    is_new = torch.cat([torch.arange(n + k) >= n for n in lens]).cuda()

    def cu(ns):
        return torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32, device="cuda")

    attn.append(pool, kk[~is_new], vv[~is_new], cu(lens), torch.tensor(lens, dtype=torch.int32, device="cuda"), table)
    step = (cu([k, k]), torch.tensor([n + k for n in lens], dtype=torch.int32, device="cuda"), table)
    attn.append(pool, kk[is_new], vv[is_new], *step)
    got = attn.attend(pool, q[is_new], *step)["out"]
    assert attn.get_error() == lib.SV_OK
    # two roundings of the same values to bf16, with weights rounded to 16 bits in each
    assert ((got - whole[is_new]).abs().float() <= 2.0 ** -6 * vv.abs().amax().float()).all()


# ------------------------------------------- what a row does not see is not there
@pytest.mark.parametrize("hq, hkv, d, dtype", [(16, 2, 128, BF16), (10, 2, 64, BF16), (8, 8, 128, BF16), (16, 2, 128, E4M3), (6, 2, 64, E4M3)])
@pytest.mark.parametrize("new, old", [([150, 3], [40, 300]), ([8, 8], [250, 500]), ([400], [700])])
def test_later_tokens_that_are_not_finite_leave_earlier_rows_alone(lib, new, old, hq, hkv, d, dtype):
    w = World(new, old, hq, hkv, d, 32, dtype, seed=14)
    expected = w.expect_attention()
    attn, pool, where = setup(lib, w)
    at = [max(1, n // 2) for n in new]                       # new token of each sequence with bad vectors
    cols = {5: float("nan"), 6: float("inf"), d - 1: float("-inf")}
    q = w.q.cuda()
    for b, i in enumerate(at):
        pos = w.kv[b] - new[b] + i
        page, slot = w.table[b, pos // 32], pos % 32
        if dtype == BF16:
            pool.k[page, :, slot, 3] = float("nan")
            for col, x in cols.items():
                pool.v[page, :, slot, col] = x
        else:
            pool.k_scale[page, :, slot] = pool.v_scale[page, :, slot] = 255
            pool.k.view(torch.uint8)[page, :, slot] = pool.v.view(torch.uint8)[page, :, slot] = 0x7f
    got = attn.attend(pool, q, *where, want_lse=True)
    again = attn.attend(pool, q, *where, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    assert torch.equal(got["out"].view(torch.int16), again["out"].view(torch.int16))
    for b, i in enumerate(at):
        clean = slice(w.cu[b], w.cu[b] + i)
        assert_attention(got["out"][clean], got["lse"][clean], [x[clean] for x in expected])
        assert torch.isnan(got["out"][w.cu[b] + i:w.cu[b + 1]]).all()      # they see a key of NaN


@pytest.mark.parametrize("hq, hkv, d", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("n", [100, 300, 900])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(lib, n, hq, hkv, d):
    w = World([n], [0], hq, hkv, d, 16, BF16, seed=15)
    bad = {3: (n // 3, float("nan")), 4: (n // 2, float("inf")), 5: (n - 1, float("-inf")), d - 2: (0, float("inf"))}
    v = w.v_new.clone()
    for col, (i, x) in bad.items():
        v[i, :, col] = x
    w.kc[0], w.vc[0] = w.k_new.double().numpy(), w.v_new.double().numpy()
    attn = lib.SpecAttention(hq, hkv, d, 1)
    got = attn.prompt(w.q.cuda(), w.k_new.cuda(), v.cuda(), torch.from_numpy(w.cu).cuda(), want_lse=True)
    assert attn.get_error() == lib.SV_OK
    out = got["out"].float().cpu()
    for col, (i, x) in bad.items():
        seen = out[i:, :, col]
        assert torch.isnan(seen).all() if x != x else (seen == x).all()
        assert torch.isfinite(out[:i, :, col]).all()
    ref = w.expect_attention()
    keep = np.ones(d, bool)
    keep[list(bad)] = False
    fixed = np.where(keep, got["out"].double().cpu().numpy(), ref[0])
    assert_attention(torch.from_numpy(fixed), got["lse"], ref)


# --------------------------------------------------- streams, graphs, repeats
def test_calls_repeat_bit_for_bit_and_in_a_graph_on_another_stream(lib):
    w = World([8, 1, 30], [900, 2500, 33], 16, 2, 128, 32, BF16, seed=11)
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
    with torch.cuda.graph(graph, stream=side):
        attn.attend(pool, q, *where, out=out, stream=side)
    q.copy_(torch.randn_like(q))                    # new inputs in the captured buffers
    fresh = attn.attend(pool, q, *where, want_lse=True)
    for _ in range(3):
        out["out"].zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[name], fresh[name]) for name in first)
    assert not torch.equal(fresh["out"], first["out"])
    assert attn.get_error() == lib.SV_OK


@pytest.mark.parametrize("dtype, hq, n", [(BF16, 64, 8), (E4M3, 64, 16), (BF16, 32, 1), (BF16, 32, 200)])
def test_long_ragged_contexts_from_cold_memory(lib, dtype, hq, n):
    """Runs of dozens of blocks whose copies keep the products waiting, against a
    float64 softmax on the GPU, twice with the same bits."""
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
    pool = attn.alloc_pool(sum(need), page, dtype)
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
        # the bounds of tests/_attn.py
        assert ((got[0]["out"][rows].double() - ref).abs() <= 2.0 ** -9 * ref.abs() + 2.0 ** -8 * spread).all()
        reach = torch.einsum("nhd,lhd->nhl", q[rows].double().abs(), kk.abs()).amax(-1) * d ** -0.5
        assert ((got[0]["lse"][rows].double() - lse).abs() <= 2.0 ** -16 * (1 + reach)).all()


def test_offsets_beyond_32_bits(lib):
    """Pages whose byte and element offsets pass 2^32 and 2^31."""
    hkv, d, page = 8, 128, 128
    per = hkv * page * d
    pages = (1 << 32) // per // 2 * 2 + 8           # > 2^32 elements: 8.6 GB a tensor in bf16
    w = World([8, 1], [200, 140], 16, hkv, d, page, BF16, seed=12)
    attn = lib.SpecAttention(16, hkv, d, 2)
    big = [torch.empty((pages, hkv, page, d), dtype=BF16, device="cuda") for _ in range(2)]
    high = pages - w.num_pages
    for t, name in zip(big, ("k", "v")):
        t[high:] = w.codes[name].cuda()
    pool = lib.KVPool(*big)
    _, cu, kv_len, table = w.to("cuda")
    where = (cu, kv_len, table + high)
    got = attn.attend(pool, w.q.cuda(), *where, want_lse=True)
    assert_attention(got["out"], got["lse"], w.expect_attention())
    back = attn.read(pool, *where, n_tokens=w.n)
    ref = np.concatenate([x[w.kv[b] - n:] for b, (x, n) in enumerate(zip(w.kc, w.new))])
    assert np.array_equal(back["k"].double().cpu().numpy(), ref)
    attn.append(pool, w.k_new.cuda(), w.v_new.cuda(), *where)
    assert attn.get_error() == lib.SV_OK
    back = attn.read(pool, *where, n_tokens=w.n)
    assert torch.equal(back["v"].cpu(), w.v_new)


# ----------------------------------------------------------- wrong metadata
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_wrong_metadata_is_reported_and_stays_in_bounds(lib, dtype):
    w = World([8, 4, 2], [100, 30, 12], 8, 2, 64, 16, dtype, seed=13)
    good = w.expect_attention()
    attn, pool, (cu, kv_len, table) = setup(lib, w)
    q = w.q.cuda()
    rows = {0: slice(0, 8), 1: slice(8, 12), 2: slice(12, 14)}

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
    t[0, -1] = -5                                   # the page of sequence 0's newest tokens
    before = pool.k.view(torch.uint8).clone()
    attn.append(pool, w.k_new.cuda(), w.v_new.cuda(), cu, kv_len, t)
    assert attn.get_error() == lib.SV_ERR_DATA
    pages = [p for p in range(w.num_pages) if p not in table.tolist()[0][:6] + table.tolist()[1] + table.tolist()[2]]
    assert torch.equal(pool.k.view(torch.uint8)[pages], before[pages])
    out = attn.read(pool, cu, kv_len, t, n_tokens=w.n)
    assert attn.get_error() == lib.SV_ERR_DATA
    assert torch.isnan(out["k"][7]).all() and torch.isfinite(out["k"][8:]).all()
    for bad_cu in ([0, 9, 5, 14], [-3, 8, 12, 14], [0, 8, 12, 99]):
        attn.attend(pool, q, torch.tensor(bad_cu, dtype=torch.int32, device="cuda"), kv_len, table)
        assert attn.get_error() == lib.SV_ERR_DATA


def test_refusals(lib):
    with pytest.raises(lib.SpecVerifyError):
        lib.SpecAttention(9, 2, 64, 1)
    with pytest.raises(lib.SpecVerifyError):
        lib.SpecAttention(8, 2, 80, 1)
    attn = lib.SpecAttention(8, 2, 64, 4)
    pool = attn.alloc_pool(4, 16)
    q = torch.zeros((2, 8, 64), dtype=BF16, device="cuda")
    cu, kv = torch.tensor([0, 2], dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(ValueError, match="scale"):
            attn.attend(pool, q, cu, kv, table, scale=scale)
    with pytest.raises(ValueError, match="shape"):
        attn.attend(pool, q[:, :4], cu, kv, table)
    with pytest.raises(ValueError, match="expected cuda"):
        attn.attend(pool, q, cu.cpu(), kv, table)
    with pytest.raises(ValueError, match="pool of"):
        attn.attend(lib.SpecAttention(8, 4, 64, 4).alloc_pool(4, 16), q, cu, kv, table)
    with pytest.raises(ValueError, match="lse"):
        attn.attend(pool, q, cu, kv, table, want_lse=True, out={"out": torch.empty_like(q)})
    with pytest.raises(ValueError, match="shape"):
        attn.append(pool, q[:, :2], q[:1, :2], cu, kv, table)
    with pytest.raises(ValueError, match="output"):
        attn.read(pool, cu, kv, table, n_tokens=2, out={"k": q, "v": q})
    assert attn.get_error() == lib.SV_OK


def test_no_sequences_and_no_tokens(lib):
    attn = lib.SpecAttention(8, 2, 64, 4)
    pool = attn.alloc_pool(4, 16, E4M3)
    q = torch.zeros((0, 8, 64), dtype=BF16, device="cuda")
    kv = q[:, :2]
    cu, none = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    table = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    assert attn.attend(pool, q, cu, none, table, want_lse=True)["out"].shape == (0, 8, 64)
    assert attn.prompt(q, kv, kv, cu)["out"].shape == (0, 8, 64)
    attn.append(pool, kv, kv, cu, none, table)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")              # sequences without tokens
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    attn.attend(pool, q, cu, none, torch.zeros((2, 1), dtype=torch.int32, device="cuda"))
    assert attn.get_error() == lib.SV_OK
