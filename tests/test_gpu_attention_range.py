"""Attention over e4m3 caches whose vectors differ far in size: zero values, vectors at the
ends of the format's range, and outsized tokens that a row does not see or hardly weighs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import _attn  # noqa: E402

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    return sv


def normal(g, *shape):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).bfloat16()


def cache(lib, hq, k, v, page=32):
    """k, v: lists of [tokens, heads, D] bf16.  Returns handle, pool, kv_len, table and the
    sequences' cached values in float64."""
    hkv, d, lens = k[0].shape[1], k[0].shape[2], [len(x) for x in k]
    need = [-(-n // page) for n in lens]
    attn = lib.SpecAttention(hq, hkv, d, len(k))
    pool = attn.alloc_pool(sum(need) + 1, page, E4M3)
    order = np.random.default_rng(0).permutation(sum(need) + 1)
    table = np.zeros((len(k), max(need)), np.int32)
    for b, c in enumerate(need):
        table[b, :c] = order[sum(need[:b]):sum(need[:b]) + c]
    table = torch.from_numpy(table).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    attn.append(pool, torch.cat(k).cuda(), torch.cat(v).cuda(), cu, kv_len, table)
    values = []
    for x in (k, v):
        parts = []
        for y in x:
            codes, scale = _attn.quantise(y.double().numpy())
            parts.append(_attn.e4m3_value(codes) * 2.0 ** (scale.astype(np.float64) - 127)[..., None])
        values.append(parts)
    assert attn.get_error() == lib.SV_OK
    return attn, pool, kv_len, table, *values


def check(lib, hq, q, k, v, causal=True):
    """q: list of [new tokens, hq, D]; the new tokens are the last ones of k and v."""
    attn, pool, kv_len, table, kc, vc = cache(lib, hq, k, v)
    cu = torch.tensor(np.concatenate([[0], np.cumsum([len(x) for x in q])]), dtype=torch.int32, device="cuda")
    got = attn.attend(pool, torch.cat(q).cuda(), cu, kv_len, table, causal=causal, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    parts = []
    for b, x in enumerate(q):
        n, kv = len(x), len(k[b])
        seen = [kv - n + i + 1 if causal else kv for i in range(n)]
        parts.append(_attn.attention(x.double().numpy(), kc[b], vc[b], x.shape[-1] ** -0.5, seen))
    _attn.assert_attention(got["out"], got["lse"], [np.concatenate([p[i] for p in parts]) for i in range(4)])


# --------------------------------------------------------------- small values
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("zero_keys", [True, False])
@pytest.mark.parametrize("lens", [[130], [256], [1000, 3], [6000], [300] * 40])
def test_values_that_are_all_zero(lib, lens, zero_keys, d):
    g = np.random.default_rng(1)
    k = [normal(g, n, 2, d) * (0 if zero_keys else 1) for n in lens]
    v = [torch.zeros_like(x) for x in k]
    check(lib, 8, [normal(g, 2, 8, d) for _ in lens], k, v)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** -100, 1.0, 2.0 ** 30, 2.0 ** 90])
@pytest.mark.parametrize("n, zeros", [(300, (0, 260)), (1000, (0, 640)), (6000, (0, 3000)), (6000, (2000, 5000)), (700, (300, 700))])
def test_stretches_of_zero_values_beside_others(lib, n, zeros, size, d):
    """The zeros count in the sum of weights, whatever the size of the other values."""
    g = np.random.default_rng(2)
    k, v = normal(g, n, 1, d) * 0.1, normal(g, n, 1, d) * size
    v[zeros[0]:zeros[1]] = 0
    check(lib, 4, [normal(g, 3, 4, d)], [k], [v])


def test_largest_scales(lib):
    """Scale bytes up to 254: values at the end of the format's range."""
    d, n = 64, 200
    g = np.random.default_rng(3)
    k, v = normal(g, n, 1, d), normal(g, n, 1, d)
    attn, pool, kv_len, table, kc, vc = cache(lib, 2, [k], [v])
    pool.v.view(torch.uint8).fill_(1)                                    # 2^-9 each
    for byte in (240, 253, 254):
        pool.v_scale.fill_(byte)
        q = normal(g, 1, 2, d)
        got = attn.attend(pool, q.cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"), kv_len, table, want_lse=True)
        value = 2.0 ** (byte - 127 - 9)
        ref = _attn.attention(q.double().numpy(), kc[0], np.ones_like(vc[0]), d ** -0.5, [n])
        assert (np.abs(got["out"].double().cpu().numpy() / value - 1) <= 2.0 ** -7).all()
        assert (np.abs(got["lse"].double().cpu().numpy() - ref[1]) <= ref[3]).all()


# ------------------------------------------------------------ outsized tokens
def shifted(x, at, shift):
    x = x.clone()
    x[at] *= 2.0 ** shift
    return x


@pytest.mark.parametrize("d, hq, hkv", [(64, 4, 2), (128, 8, 1), (128, 15, 3)])
@pytest.mark.parametrize("shift", [13, 15, 20, 30, 60, 100])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
def test_later_tokens_of_another_size_leave_earlier_rows_alone(lib, which, shift, d, hq, hkv):
    g = np.random.default_rng(4)
    q, k, v = [], [], []
    for n, old in ((8, 100), (150, 40), (5, 260)):
        kk, vv = normal(g, old + n, hkv, d), normal(g, old + n, hkv, d)
        for at in (old + n - 1, old + n // 2):
            kk = shifted(kk, at, shift) if "k" in which else kk
            vv = shifted(vv, at, shift) if "v" in which else vv
        q.append(normal(g, n, hq, d)), k.append(kk), v.append(vv)
    check(lib, hq, q, k, v)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shift", [20, 40, 70, 100])
@pytest.mark.parametrize("n, at", [(100, 7), (500, 3), (500, 499), (500, 200), (9000, 1000)])
def test_outsized_values_that_hardly_weigh(lib, n, at, shift, d):
    """One token's value is 2^shift times the others', its weight e^-100: what the others give remains."""
    g = np.random.default_rng(6)
    q, k, v = normal(g, 1, 1, d), normal(g, n, 1, d) * 0.3, shifted(normal(g, n, 1, d), at, shift)
    u = q[0, 0].double()
    k[at, 0] = (-100.0 * d ** 0.5 / (u @ u) * u).bfloat16()
    check(lib, 1, [q], [k], [v])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shift", [20, 40, 100])
@pytest.mark.parametrize("n, at", [(100, 7), (500, 200), (9000, 1000)])
def test_outsized_keys_whose_scores_are_far_below(lib, n, at, shift, d):
    g = np.random.default_rng(7)
    q, k, v = normal(g, 1, 1, d), normal(g, n, 1, d), normal(g, n, 1, d)
    u = q[0, 0].double()
    k[at, 0] = (-(2.0 ** shift) * u / (u @ u) ** 0.5).bfloat16()
    attn, pool, kv_len, table, kc, vc = cache(lib, 1, [k], [v])
    got = attn.attend(pool, q.cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"), kv_len, table, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    # that key's weight is 0 in float64 too; without it the bound on a score is that of the others
    kept = [np.delete(x[0], at, 0) for x in (kc, vc)]
    _attn.assert_attention(got["out"], got["lse"], _attn.attention(q.double().numpy(), *kept, d ** -0.5, [n - 1]))


@pytest.mark.parametrize("causal", [True, False])
def test_sizes_spread_over_the_whole_range(lib, causal):
    """Every vector its own size, keys and values: 2^-60 to 2^60."""
    g = np.random.default_rng(8)
    q, k, v = [], [], []
    for n, old in ((7, 300), (40, 1000), (1, 2)):
        kk, vv = normal(g, old + n, 2, 64), normal(g, old + n, 2, 64)
        for x, hi in ((kk, 0), (vv, 60)):
            x *= torch.from_numpy(2.0 ** g.integers(-60, hi + 1, (old + n, 2, 1)).astype(np.float32)).bfloat16()
        q.append(normal(g, n, 8, 64)), k.append(kk), v.append(vv)
    check(lib, 8, q, k, v, causal=causal)


# -------------------------------------------- scale bytes of another program
@pytest.mark.parametrize("d", [64, 128])
def test_scale_byte_255_is_nan_whatever_the_codes(lib, d):
    """read and attend agree on a vector whose byte is 255 and whose codes are numbers."""
    g = np.random.default_rng(9)
    n, new, at, page = 300, 20, 290, 32
    q, k, v = normal(g, new, 4, d), normal(g, n, 2, d), normal(g, n, 2, d)
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    for name in ("k", "v"):
        attn, pool, kv_len, table, kc, vc = cache(lib, 4, [k], [v], page)
        where = table[0, at // page].item(), slice(None), at % page
        getattr(pool, name + "_scale")[where] = 255
        back = attn.read(pool, cu, kv_len, table, n_tokens=new)[name]
        assert torch.isnan(back[at - (n - new)]).all() and torch.isfinite(back).sum().item() == (new - 1) * 2 * d
        got = attn.attend(pool, q.cuda(), cu, kv_len, table, want_lse=True)
        assert attn.get_error() == lib.SV_OK
        clean = at - (n - new)                       # rows that do not see the token
        expected = _attn.attention(q.double().numpy(), kc[0], vc[0], d ** -0.5, [n - new + i + 1 for i in range(new)])
        _attn.assert_attention(got["out"][:clean], got["lse"][:clean], [x[:clean] for x in expected])
        assert torch.isnan(got["out"][clean:]).all()


def test_scale_byte_0_is_read_as_2_to_the_minus_127(lib):
    g = np.random.default_rng(10)
    n, d = 40, 64
    attn, pool, kv_len, table, _, _ = cache(lib, 2, [normal(g, n, 1, d)], [normal(g, n, 1, d)])
    pool.k_scale.fill_(0), pool.v_scale.fill_(0)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    got = attn.read(pool, cu, kv_len, table, n_tokens=n)
    for name in ("k", "v"):
        codes = getattr(pool, name).view(torch.uint8).cpu().numpy()
        ref = np.stack([_attn.e4m3_value(codes[table[0, p // 32].item(), :, p % 32]) for p in range(n)]) * 2.0 ** -127
        assert torch.equal(got[name].float().cpu(), torch.from_numpy(ref).float().bfloat16().float())
