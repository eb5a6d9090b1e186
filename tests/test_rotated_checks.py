"""4-bit pools and rotated appends without a GPU: checks of arguments, and the
references that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_68_gb300 as sv  # noqa: E402
from speculative_decoding_verification_68_gb300 import _native  # noqa: E402
from speculative_decoding_verification_68_gb300.attention import KVPool, Rope, _CBatch, _CPool, _CRope, _CRows  # noqa: E402
from tests import _attn, _attn4  # noqa: E402
from tests.test_attention_checks import _FakeHandle, lib  # noqa: E402, F401

FOUR, E4M3 = torch.float4_e2m1fn_x2, torch.float8_e4m3fn


def four(pages=3, heads=2, page=16, d=64):
    codes = torch.zeros((pages, heads, page, d // 2), dtype=torch.uint8).view(FOUR)
    return [codes, codes.clone(), torch.zeros((pages, heads, page), dtype=torch.uint8), torch.zeros((pages, heads, page), dtype=torch.uint8),
            torch.zeros((pages, heads, page, d // 16), dtype=E4M3), torch.zeros((pages, heads, page, d // 16), dtype=E4M3)]


def test_four_bit_pool_checks():
    pool = KVPool(*four())
    assert (pool.head_dim, pool.page_size, pool.kv_heads, pool.quantised) == (64, 16, 2, True)
    for i, bad, what in ((4, None, "k_block is required"), (5, None, "v_block is required"), (2, None, "k_scale is required"),
                         (4, torch.zeros((3, 2, 16, 4), dtype=torch.uint8), "dtype"), (5, torch.zeros((3, 2, 16, 8), dtype=E4M3), "shape"),
                         (1, torch.zeros((3, 2, 16, 64), dtype=torch.uint8).view(FOUR), "shape"), (1, torch.zeros((3, 2, 16, 32), dtype=torch.uint8), "dtype"),
                         (4, torch.zeros(3 * 2 * 16 * 4 + 8, dtype=torch.uint8)[8:].view(E4M3).view(3, 2, 16, 4), "aligned"),
                         (3, torch.zeros(3 * 2 * 16 + 8, dtype=torch.uint8)[8:].view(3, 2, 16), "aligned")):
        args = four()
        args[i] = bad
        with pytest.raises(ValueError, match=what):
            KVPool(*args)
    bf16 = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="only a 4-bit pool"):
        KVPool(bf16, bf16, None, None, four()[4], four()[5])


@pytest.mark.parametrize("table, what", [
    (None, "must be"), (torch.zeros(32), "must be"), (torch.zeros((4, 32), dtype=torch.float64), "dtype"), (torch.zeros((4, 24)), "multiple of 16"),
    (torch.zeros((0, 32)), "at least one"), (torch.zeros((4, 64))[:, ::2], "contiguous"), (torch.zeros(4 * 32 + 1)[1:].view(4, 32), "aligned"), (torch.zeros((4, 0)), "multiple")])
def test_bad_tables_raise(table, what):
    with pytest.raises(ValueError, match=what):
        Rope(table)


def test_host_side_checks_of_the_call(lib):  # noqa: F811
    fake = _FakeHandle(device=7, q_heads=4, kv_heads=2, D=64, max_seqs=8)
    memory = (ctypes.c_byte * 64)()
    at = ctypes.addressof(memory) + 32 - ctypes.addressof(memory) % 32
    pool, batch, rows = _CPool(k=at, v=at, dtype=1, num_pages=1, page_size=16), _CBatch(), _CRows(ptr=at, token_stride=64, head_stride=64)
    rope = _CRope(table=at, max_positions=4, rot_dim=64)
    h, p, b, r, t = (ctypes.byref(x) for x in (fake, pool, batch, rows, rope))
    assert lib.spec_attn_append_rotated(None, p, b, t, r, r, r, r, r, None) == sv.SV_ERR_ARG
    # without a GPU there is no current device at all
    assert lib.spec_attn_append_rotated(h, p, b, t, r, r, r, r, r, None) == (sv.SV_ERR_ARG if torch.cuda.is_available() else 4)
    assert sv.SV_E2M1 == 3 and _native.load() is lib


def test_reference_quantiser_by_brute_force():
    g = np.random.default_rng(0)
    x = torch.from_numpy(g.standard_normal((300, 64)).astype(np.float32) * np.exp(2 * g.standard_normal((300, 64))).astype(np.float32)).bfloat16().double().numpy()
    x[0], x[1, 5], x[2, 6] = 0, np.inf, np.nan
    codes, block, scale = _attn4.quantise4(x)
    assert (scale[1], scale[2], scale[0]) == (255, 255, 7) and (block[1:3] == 0x7f).all() and not block[0].any()
    back = _attn4.values4(codes, block, scale)
    assert np.isnan(back[1:3]).all() and not back[0].any()
    s = _attn.e4m3_value(block)
    for i in range(3, 300):
        unit = 2.0 ** (int(scale[i]) - 127)
        assert 1344 * unit < np.abs(x[i]).max() <= 2688 * unit
        for j in range(4):
            want = np.abs(x[i, 16 * j:16 * j + 16]).max() / 6 / unit
            assert abs(s[i, j] - want) == np.abs(_attn4._E4M3 - want).min()
        grid = np.concatenate([-_attn4.E2M1, _attn4.E2M1])[None] * np.repeat(s[i], 16)[:, None] * unit
        assert np.array_equal(np.abs(back[i] - x[i]), np.abs(grid - x[i][:, None]).min(-1))


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_turns_pairs(interleaved):
    g = np.random.default_rng(1)
    x = g.standard_normal((5, 2, 64)).astype(np.float32)
    table = _attn4.rope_table(40, 32)
    pos = np.array([0, 1, 7, 39, 39])
    y = _attn4.rotate(x, table, pos, interleaved)
    z = x[..., :32].reshape(5, 2, 16, 2) if interleaved else np.moveaxis(x[..., :32].reshape(5, 2, 2, 16), 2, 3)
    turn = np.exp(1j * pos[:, None] * 10000.0 ** -(np.arange(0, 32, 2) / 32))[:, None]
    z = (z[..., 0] + 1j * z[..., 1]) * turn
    want = np.stack([z.real, z.imag], -1).reshape(5, 2, 32) if interleaved else np.concatenate([z.real, z.imag], -1)
    assert np.allclose(y[..., :32], want, atol=2e-6) and np.array_equal(y[..., 32:], x[..., 32:]) and np.array_equal(y[0], x[0])


def test_the_quotient_of_the_quantiser_is_correctly_rounded():
    """x / s as q + (x - q s) r with q = fl(x r), r = fl(1 / s), fused: for every s of 4 significant bits."""
    import math
    fma = getattr(math, "fma", None)
    g = np.random.default_rng(2)
    for m in range(1, 16):
        s, r = np.float32(m), np.float32(1) / np.float32(m)
        # multiples of half-way points, their neighbours, and any x
        ties = np.outer(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), np.array([m])).astype(np.float32).ravel()
        x = np.concatenate([ties, np.nextafter(ties, np.float32(0)), np.nextafter(ties, np.float32(9e9)), g.uniform(1, 2, 2000).astype(np.float32)])
        q = x * r
        rem = (x.astype(np.float64) - q.astype(np.float64) * float(s)).astype(np.float32)      # exact in 64 bits
        assert np.array_equal(rem.astype(np.float64), x.astype(np.float64) - q.astype(np.float64) * float(s))
        out = np.array([np.float32(fma(float(b), float(r), float(a))) if fma else np.float32(np.longdouble(a) + np.longdouble(b) * np.longdouble(r))
                        for a, b in zip(q, rem)], np.float32)
        assert np.array_equal(out, x / s)
