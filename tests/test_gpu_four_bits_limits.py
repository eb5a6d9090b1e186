"""The limits of calls on 4-bit caches: lengths near 2^31, factors at the ends of a
float's range, and schedules too long for the short plan."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests._attn4 import FOUR, rope_table  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    return sv


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hq", [2, 40])                                        # up to 16 rows, more
def test_lengths_near_2_31_are_invalid_data(lib, hq):
    attn = lib.SpecAttention(hq, 1, 64, 1)
    pool = attn.alloc_pool(2, 128, FOUR)
    table = torch.zeros((1, 1 << 24), dtype=torch.int32, device="cuda")        # pages enough for 2^31 tokens
    q, k = torch.ones((1, hq, 64), dtype=BF16, device="cuda"), torch.ones((1, 1, 64), dtype=BF16, device="cuda")
    got = attn.attend(pool, q, ints(0, 1), ints(2 ** 31 - 511), table, want_lse=True)
    assert attn.get_error() == lib.SV_ERR_DATA
    assert torch.isnan(got["out"]).all() and torch.isnan(got["lse"]).all()
    assert torch.isnan(attn.read(pool, ints(0, 1), ints(2 ** 31 - 511), table, n_tokens=1)["k"]).all()
    assert attn.get_error() == lib.SV_ERR_DATA
    rope = lib.Rope(rope_table(4, 64).cuda())
    before = pool.k.view(torch.uint8).clone()
    turned = attn.append_rotated(pool, k, k, ints(0, 1), ints(2 ** 31 - 511), table, rope, q=q, positions=ints(0))
    assert attn.get_error() == lib.SV_ERR_DATA
    assert torch.isnan(turned["q"]).all() and torch.equal(pool.k.view(torch.uint8), before)
    turned = attn.append_rotated(pool, k, k, ints(0, 1), ints(2 ** 31 - 512), table, rope, q=q, positions=ints(0))
    assert attn.get_error() == lib.SV_OK and torch.equal(turned["q"], q)
    # 1/6 is not an e4m3 number: a block's largest element, its scale times 6, is off by 2^-4 at most
    assert ((attn.read(pool, ints(0, 1), ints(2 ** 31 - 512), table, n_tokens=1)["k"] - k).abs() <= 2.0 ** -4).all()


@pytest.mark.parametrize("hq", [2, 20])
@pytest.mark.parametrize("scale", [1e-40, 1e-38, 2.9e38])
def test_scales_at_the_ends_of_the_range(lib, scale, hq):
    """Queries of zero give every key the same weight, whatever the factor."""
    n, d = 150, 64
    attn = lib.SpecAttention(hq, 1, d, n)
    pool = attn.alloc_pool(10, 16, FOUR)
    g = torch.Generator(device="cuda").manual_seed(41)
    k, v = (torch.randn((n, 1, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.arange(10, dtype=torch.int32, device="cuda")[None]
    attn.append(pool, k, v, ints(0, n), ints(n), table)
    values = attn.read(pool, ints(0, n), ints(n), table, n_tokens=n)["v"].double()
    seen = torch.arange(1, n + 1, device="cuda")[:, None].double()
    mean, spread = values.cumsum(0) / seen[..., None], values.abs().cumsum(0) / seen[..., None]
    q = torch.zeros((n, hq, d), dtype=BF16, device="cuda")
    whole = attn.attend(pool, q, ints(0, n), ints(n), table, scale=scale, want_lse=True)
    # and a sequence for every token of them, over the same pages
    single = attn.attend(pool, q, ints(*range(n + 1)), ints(*range(1, n + 1)), table.expand(n, 10).contiguous(), scale=scale, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    for got in (whole, single):
        # rounding to bf16 (2^-8) of the result, and less of the weights and sums
        assert ((got["out"].double() - mean).abs() <= 2.0 ** -7 * mean.abs() + 2.0 ** -8 * spread).all()
        assert ((got["lse"].double() - seen.log()).abs() <= 2.0 ** -16).all()


@pytest.mark.parametrize("hq", [2, 20])
def test_a_schedule_of_more_than_2_17_units(lib, hq):
    """30.7 million tokens that all lie in one page: the softmax over the page, each of its weights 240,000 times."""
    d, page, times = 64, 128, 240000
    attn = lib.SpecAttention(hq, 1, d, 2)
    pool = attn.alloc_pool(1, page, FOUR)
    g = torch.Generator(device="cuda").manual_seed(42)
    k, v = (torch.randn((page, 1, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.zeros((1, times), dtype=torch.int32, device="cuda")
    attn.append(pool, k, v, ints(0, page), ints(page), table)
    back = attn.read(pool, ints(0, page), ints(page), table, n_tokens=page)
    q = torch.randn((1, hq, d), generator=g, device="cuda").bfloat16()
    got = attn.attend(pool, q, ints(0, 1), ints(page * times), table, causal=False, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    s = torch.einsum("nhd,ld->nhl", q.double(), back["k"][:, 0].double()) * d ** -0.5
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    ref, spread = p @ back["v"][:, 0].double(), p @ back["v"][:, 0].double().abs()
    # sums of 32 bits over at most 30.7e6 / 152 / 128 blocks in a row are off by 1,600 * 2^-24 = 2^-13.4 of their size
    assert ((got["out"].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * spread).all()
    assert ((got["lse"].double() - lse - math.log(times)).abs() <= 2.0 ** -12).all()
