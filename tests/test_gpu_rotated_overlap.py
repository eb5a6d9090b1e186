"""The C interface refuses rotated appends whose output rows overlap, before any launch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_verification_68_gb300.attention import _CBatch, _CRope, _CRows  # noqa: E402

pytestmark = pytest.mark.gpu
N, HQ, HKV, D = 3, 4, 2, 64


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    return sv


@pytest.fixture
def call(lib):
    """call(tokens=N, **tensors): the status, each of q, k, v, q_out, k_out given as (offset in elements, token stride,
    head stride) within one buffer, or None; and whether anything was written."""
    attn = lib.SpecAttention(HQ, HKV, D, 1)
    pool = attn.alloc_pool(1, 16)
    memory = torch.full((1 << 16,), 3.0, dtype=torch.bfloat16, device="cuda")
    turns = torch.zeros((16, D), device="cuda")                  # every rotated row becomes 0
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")

    def run(tokens=N, **tensors):
        memory.fill_(3.0), pool.k.zero_()
        places = dict(q=(0, HQ * D, D), k=(8192, HKV * D, D), v=(16384, HKV * D, D), q_out=(24576, HQ * D, D), k_out=(32768, HKV * D, D))
        places.update(tensors)
        rows = {name: None if p is None else _CRows(memory.data_ptr() + 2 * p[0], p[1], p[2]) for name, p in places.items()}
        cu, kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, tokens], [tokens]))
        batch = _CBatch(cu.data_ptr(), kv.data_ptr(), table.data_ptr(), 1, tokens, 1, 0)
        rope = _CRope(turns.data_ptr(), None, 16, D, 0)
        ref = {name: None if r is None else ctypes.byref(r) for name, r in rows.items()}
        rc = attn._lib.spec_attn_append_rotated(attn._h, pool._ref, ctypes.byref(batch), ctypes.byref(rope), ref["q"], ref["k"], ref["v"],
                                                ref["q_out"], ref["k_out"], torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert attn.get_error() == lib.SV_OK
        return rc, bool((memory != 3.0).any()) or bool(pool.k.any()) or bool((pool.v != 0).any())

    return run


QKV = dict(q=(0, 512, D), k=(256, 512, D), v=(384, 512, D))     # slices of a fused projection


@pytest.mark.parametrize("tokens, tensors", [
    (N, {}), (N, dict(k_out=None)), (N, dict(q=None, q_out=None)), (N, dict(q=None, q_out=None, k_out=None)),
    (N, dict(q_out=(0, HQ * D, D), k_out=(8192, HKV * D, D))), (N, {**QKV, "q_out": QKV["q"], "k_out": QKV["k"]}),
    (N, dict(q_out=(24576, D, N * D))), (N, dict(q_out=(24576, D + 8, N * D + 24))), (N, dict(q_out=(24576, 4 * D + 24, D + 8))),
    (1, dict(q_out=(24576, 0, D))), (1, dict(q_out=(0, 8, D), k_out=(8192, 0, D))), (N, dict(q=(0, 0, 0), k=(8192, 0, 0), v=(8192, 0, 0)))])
def test_rows_that_lie_apart_are_taken(lib, call, tokens, tensors):
    assert call(tokens, **tensors) == (lib.SV_OK, True)


@pytest.mark.parametrize("tokens, tensors", [
    (N, dict(q_out=(24576, 0, D))), (N, dict(q_out=(24576, HQ * D, 0))), (N, dict(k_out=(32768, 0, D))), (N, dict(k_out=(32768, HKV * D, 0))),
    (N, dict(q_out=(24576, D, D))), (N, dict(q_out=(24576, HQ * D - 8, D))), (N, dict(q_out=(24576, D, N * D - 8))), (N, dict(q_out=(24576, D - 8, 512))),
    (1, dict(q_out=(24576, 512, D - 8))), (1, dict(k_out=(32768, 512, 0))), (N, dict(k_out=(32768, (1 << 62) + 8, 1 << 62))),
    (N, dict(q_out=(0, 512, D))), (N, dict(q_out=(0, D, N * D))), (N, dict(k_out=(8192, 512, D))), (1, dict(q_out=(0, HQ * D, 2 * D))),
    (N, dict(q_out=(8192, HQ * D, D))), (N, dict(q_out=(16384, HQ * D, D))), (N, dict(k_out=(16384, HKV * D, D))), (N, dict(k_out=(0, HKV * D, D))),
    (N, dict(k_out=(24576, HKV * D, D))), (N, dict(v=(8192, HKV * D, D), k_out=(8192, HKV * D, D)))])
def test_rows_that_overlap_are_refused(lib, call, tokens, tensors):
    assert call(tokens, **tensors) == (lib.SV_ERR_ARG, False)
