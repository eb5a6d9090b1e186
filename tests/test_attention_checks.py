"""The cache and attention entry points without a GPU: declared symbols, the
library's host-side checks, the binding's tensor checks, and the reference
the GPU tests compare with."""
import ctypes
import os
import re
import shutil

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_68_gb300 as sv  # noqa: E402
from speculative_decoding_verification_68_gb300 import _native  # noqa: E402
from speculative_decoding_verification_68_gb300.attention import (KVPool, _CBatch, _CPool, _CRows, check_rows,  # noqa: E402
                                                                  check_sequences)
from tests import _attn  # noqa: E402

CPU = torch.device("cpu")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "spec_attn.h")


@pytest.fixture(scope="module")
def lib():
    if shutil.which(_native.nvcc()) is None and not os.path.exists(_native.nvcc()):
        pytest.skip("nvcc not available")
    _native.build()
    return _native.load()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(spec_attn_\w+)\s*\(", text)))
    assert "spec_attn_chunk" in names and "spec_attn_append" in names
    for name in names:
        assert hasattr(lib, name), name


def test_host_side_argument_checks(lib):
    h = ctypes.c_void_p()
    assert lib.spec_attn_init(None, 8, 8, 64, 1) == sv.SV_ERR_ARG
    assert lib.spec_attn_init(ctypes.byref(h), 0, 8, 64, 1) == sv.SV_ERR_ARG
    assert lib.spec_attn_init(ctypes.byref(h), 8, 8, 64, 0) == sv.SV_ERR_ARG
    assert lib.spec_attn_init(ctypes.byref(h), 9, 8, 64, 1) == 3       # groups of unequal size
    assert lib.spec_attn_init(ctypes.byref(h), 65, 1, 64, 1) == 3      # group above 64
    assert lib.spec_attn_init(ctypes.byref(h), 8, 8, 96, 1) == 3       # head dimension
    assert lib.spec_attn_init(ctypes.byref(h), 2048, 2048, 64, 1) == 3
    assert not h.value
    pool, batch, rows = _CPool(), _CBatch(), _CRows()
    p, b, r = ctypes.byref(pool), ctypes.byref(batch), ctypes.byref(rows)
    assert lib.spec_attn_append(None, p, b, r, r, None) == sv.SV_ERR_ARG
    assert lib.spec_attn_read(None, p, b, None, None, None) == sv.SV_ERR_ARG
    assert lib.spec_attn_chunk(None, p, b, r, 1, 1.0, None, None, None) == sv.SV_ERR_ARG
    assert lib.spec_attn_prompt(None, 1, 1, None, r, r, r, 1.0, None, None, None) == sv.SV_ERR_ARG
    assert lib.spec_attn_get_error(None) == sv.SV_ERR_ARG
    lib.spec_attn_destroy(None)


def rows(n=5, heads=4, d=64):
    return torch.zeros((n, heads, d), dtype=torch.bfloat16)


def test_rows_accept_slices_of_a_fused_projection():
    fused = torch.zeros((6, 12, 64), dtype=torch.bfloat16)
    assert check_rows(fused[:, 4:8], "k", 4, 64, CPU) == 6
    assert check_rows(torch.zeros((4, 6, 64), dtype=torch.bfloat16).transpose(0, 1), "k", 4, 64, CPU) == 6
    assert check_rows(rows(0), "k", 4, 64, CPU) == 0


@pytest.mark.parametrize("t, what", [
    (None, "required"),
    (rows().float(), "dtype"),
    (rows(heads=3), "shape"),
    (rows(d=128), "shape"),
    (rows()[0], "shape"),
    (torch.zeros((5, 4, 128), dtype=torch.bfloat16)[..., ::2], "contiguous"),
    (torch.zeros((5, 4, 68), dtype=torch.bfloat16)[..., :64], "aligned"),
    (torch.zeros(5 * 4 * 64 + 1, dtype=torch.bfloat16)[1:].view(5, 4, 64), "aligned"),
])
def test_bad_rows_raise(t, what):
    with pytest.raises(ValueError, match=what):
        check_rows(t, "k", 4, 64, CPU)


def test_row_counts_and_devices_must_agree():
    with pytest.raises(ValueError, match="shape"):
        check_rows(rows(5), "v", 4, 64, CPU, n_tokens=6)
    with pytest.raises(ValueError, match="expected cuda"):
        check_rows(rows(5), "v", 4, 64, torch.device("cuda", 0))


@pytest.mark.parametrize("cu, kv, table, what", [
    (torch.zeros(3, dtype=torch.int64), None, None, "dtype"),
    (torch.zeros((3, 1), dtype=torch.int32), None, None, "cu must be"),
    (torch.zeros(0, dtype=torch.int32), None, None, "cu must be"),
    (torch.zeros(12, dtype=torch.int32), None, None, "max_seqs"),
    (torch.zeros(3, dtype=torch.int32), None, None, "kv_len is required"),
    (torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), None, "shape"),
    (torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), None, "page_table must be"),
    (torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros((3, 4), dtype=torch.int32), "shape"),
    (torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros((2, 8), dtype=torch.int32)[:, ::2], "contiguous"),
])
def test_bad_metadata_raises(cu, kv, table, what):
    with pytest.raises(ValueError, match=what):
        check_sequences(cu, CPU, 10, kv, table)


def test_pool_checks():
    k = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    s = torch.zeros((3, 2, 16), dtype=torch.uint8)
    e = k.view(torch.uint8)[..., :64].contiguous().view(torch.float8_e4m3fn)
    assert KVPool(k, k.clone()).page_size == 16
    assert KVPool(e, e.clone(), s, s.clone()).quantised
    for args, what in (((k.float(), k.float()), "dtype"), ((k, k[:2]), "shape"), ((k[0], k[0]), "num_pages"),
                       ((k[:, :, :8].contiguous(),) * 2, "page_size"), ((k, k, s, s), "no scales"), ((e, e), "required"),
                       ((e, e, s.int(), s.int()), "dtype"), ((k.transpose(0, 1), k.transpose(0, 1)), "contiguous")):
        with pytest.raises(ValueError, match=what):
            KVPool(*args)


def test_reference_quantiser_matches_the_format():
    values = _attn.e4m3_value(np.arange(256, dtype=np.uint8))
    torch_values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(values, torch_values, equal_nan=True)
    x = torch.randn(64, 64).bfloat16().double().numpy()
    x[0], x[1, 0], x[2, 3], x[3] = 0, np.inf, np.nan, 448.0
    codes, scale = _attn.quantise(x)
    assert scale[0] == 7 and scale[1] == scale[2] == 255 and scale[3] == 127
    fine = scale != 255
    y = torch.from_numpy(x[fine] * 2.0 ** (127.0 - scale[fine])[:, None]).float()
    assert (y.abs().amax(-1)[1:] > 224).all() and (y.abs() <= 448).all()
    assert np.array_equal(y.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), codes[fine])


def test_reference_attention_is_a_softmax():
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((3, 4, 8)), g.standard_normal((5, 2, 8)), g.standard_normal((5, 2, 8))
    out, lse, _, _ = _attn.attention(q, k, v, 0.5, [0, 2, 5])
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()
    s = 0.5 * k[:, 1] @ q[2, 3]
    assert np.allclose(lse[2, 3], np.log(np.exp(s).sum()))
    assert np.allclose(out[2, 3], (np.exp(s) / np.exp(s).sum()) @ v[:, 1])


class _FakeHandle(ctypes.Structure):
    """A handle's first members; zeros behind them."""
    _fields_ = [("device", ctypes.c_int), ("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("D", ctypes.c_int),
                ("max_seqs", ctypes.c_int), ("rest", ctypes.c_byte * 256)]


def calls_of_another_devices_handle(lib):
    """Status of each call with a handle whose device is not the current one.  The batch has no
    sequences, so that nothing would be launched either way."""
    fake = _FakeHandle(device=7, q_heads=4, kv_heads=2, D=64, max_seqs=8)
    memory = (ctypes.c_byte * 64)()
    at = ctypes.addressof(memory) + 32 - ctypes.addressof(memory) % 32
    pool, batch, rows = _CPool(k=at, v=at, dtype=1, num_pages=1, page_size=16), _CBatch(), _CRows(ptr=at, token_stride=64, head_stride=64)
    h, p, b, r = (ctypes.byref(x) for x in (fake, pool, batch, rows))
    return [lib.spec_attn_append(h, p, b, r, r, None), lib.spec_attn_read(h, p, b, at, at, None),
            lib.spec_attn_chunk(h, p, b, r, 1, 1.0, at, None, None), lib.spec_attn_prompt(h, 0, 0, at, r, r, r, 1.0, at, None, None),
            lib.spec_attn_get_error(h)]


def test_a_handle_of_another_device_is_refused(lib):
    # without a GPU there is no current device at all: every call says so, and none succeeds
    want = sv.SV_ERR_ARG if torch.cuda.is_available() else 4            # SV_ERR_CUDA
    assert calls_of_another_devices_handle(lib) == [want] * 5
