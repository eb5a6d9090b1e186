"""Attention over e4m3 caches whose values are zero, or at the ends of the format's range."""
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
