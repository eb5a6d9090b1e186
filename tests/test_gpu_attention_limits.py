"""The limits of the cache and attention calls: lengths near 2^31, factors at the ends of a float's
range, and handles of another GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
SV_ERR_SIZE = 3


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    return sv


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_lengths_near_2_31_are_invalid_data(lib, dtype):
    attn = lib.SpecAttention(2, 1, 64, 1)
    pool = attn.alloc_pool(2, 128, dtype)
    table = torch.zeros((1, 1 << 24), dtype=torch.int32, device="cuda")    # pages enough for 2^31 tokens
    q = torch.ones((1, 2, 64), dtype=BF16, device="cuda")
    got = attn.attend(pool, q, ints(0, 1), ints(2 ** 31 - 511), table, want_lse=True)
    assert attn.get_error() == lib.SV_ERR_DATA
    assert torch.isnan(got["out"]).all() and torch.isnan(got["lse"]).all()
    back = attn.read(pool, ints(0, 1), ints(2 ** 31 - 511), table, n_tokens=1)
    assert attn.get_error() == lib.SV_ERR_DATA
    assert torch.isnan(back["k"]).all()
    attn.read(pool, ints(0, 1), ints(2 ** 31 - 512), table, n_tokens=1)
    assert attn.get_error() == lib.SV_OK


def test_token_counts_near_2_31_are_refused(lib):
    from speculative_decoding_verification_68_gb300 import attention
    attn = lib.SpecAttention(1, 1, 64, 1)
    pool = attn.alloc_pool(1, 16)
    batch, rows, cu = attention._CBatch(), attention._CRows(), ints(0, 0)
    batch.cu = batch.kv_len = batch.page_table = cu.data_ptr()
    batch.n_seqs, batch.max_pages, batch.n_tokens = 1, 1, 2 ** 31 - 511
    rows.ptr, rows.token_stride, rows.head_stride = pool.k.data_ptr(), 64, 64
    b, r, out = ctypes.byref(batch), ctypes.byref(rows), pool.v.data_ptr()
    assert attn._lib.spec_attn_append(attn._h, pool._ref, b, r, r, None) == SV_ERR_SIZE
    assert attn._lib.spec_attn_read(attn._h, pool._ref, b, out, out, None) == SV_ERR_SIZE
    assert attn._lib.spec_attn_chunk(attn._h, pool._ref, b, r, 1, 1.0, out, None, None) == SV_ERR_SIZE
    assert attn._lib.spec_attn_prompt(attn._h, 1, batch.n_tokens, batch.cu, r, r, r, 1.0, out, None, None) == SV_ERR_SIZE
    assert attn.get_error() == lib.SV_OK


def test_a_handle_of_another_device_is_refused(lib):
    from tests.test_attention_checks import calls_of_another_devices_handle
    assert calls_of_another_devices_handle(lib._native.load()) == [lib.SV_ERR_ARG] * 5


def test_calls_on_a_stream_that_waits_for_no_other_right_after_init_and_get_error(lib):
    """What init and get_error clear is clear when they return: a call whose items are split over the
    GPU's SMs, merged by counters, follows at once on a non-blocking stream."""
    g = torch.Generator(device="cuda").manual_seed(40)
    lens, page = [3000, 700], 64
    kv_len, cu = ints(*lens), ints(0, 2, 4)
    table = torch.arange(2 * 47, dtype=torch.int32, device="cuda").view(2, 47)
    q = torch.randn((4, 8, 128), generator=g, device="cuda").bfloat16()
    pool = lib.SpecAttention(8, 2, 128, 2).alloc_pool(94, page)
    pool.k.normal_(generator=g), pool.v.normal_(generator=g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.empty_like(q) for _ in range(60)]
    for i, out in enumerate(outs):
        if i % 20 == 0:
            attn = lib.SpecAttention(8, 2, 128, 2)
        bad = i % 3 == 1                               # a flag to clear
        attn.attend(pool, q, cu, ints(-1, -1) if bad else kv_len, table, out={"out": torch.empty_like(q)})
        assert attn.get_error() == (lib.SV_ERR_DATA if bad else lib.SV_OK)
        attn.attend(pool, q, cu, kv_len, table, out={"out": out}, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(out, outs[0]) for out in outs) and torch.isfinite(outs[0]).all()
    assert attn.get_error() == lib.SV_OK


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("scale", [1e-40, 1e-38, 2.9e38])
def test_scales_at_the_ends_of_the_range(lib, scale, dtype):
    """Queries of zero give every key the same weight, whatever the factor."""
    n, d = 150, 64
    attn = lib.SpecAttention(2, 1, d, 1)
    pool = attn.alloc_pool(10, 16, dtype)
    g = torch.Generator(device="cuda").manual_seed(41)
    k, v = (torch.randn((n, 1, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.zeros((n, 2, d), dtype=BF16, device="cuda")
    table = torch.arange(10, dtype=torch.int32, device="cuda")[None]
    attn.append(pool, k, v, ints(0, n), ints(n), table)
    values = attn.read(pool, ints(0, n), ints(n), table, n_tokens=n)["v"].double()
    seen = torch.arange(1, n + 1, device="cuda")[:, None].double()
    mean, spread = values.cumsum(0) / seen[..., None], values.abs().cumsum(0) / seen[..., None]
    calls = [attn.attend(pool, q, ints(0, n), ints(n), table, scale=scale, want_lse=True)]
    if dtype == BF16:
        calls.append(attn.prompt(q, k, v, ints(0, n), scale=scale, want_lse=True))
    assert attn.get_error() == lib.SV_OK
    for got in calls:
        # rounding to bf16 (2^-8) of the weights, of the sum they are divided by, of the result
        assert ((got["out"].double() - mean).abs() <= 2.0 ** -7 * mean.abs() + 2.0 ** -8 * spread).all()
        assert ((got["lse"].double() - seen.log()).abs() <= 2.0 ** -16).all()
