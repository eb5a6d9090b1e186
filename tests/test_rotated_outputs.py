"""Outputs of a rotated append whose rows would overlap are refused: the strides' check, without a GPU."""
import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_verification_68_gb300.attention import SpecAttention, _CRows  # noqa: E402

D = 64


def check(n, heads, strides, size=8192):
    attn = SpecAttention.__new__(SpecAttention)
    attn.head_dim, attn.device, attn._h = D, torch.device("cpu"), None
    t = torch.zeros(size, dtype=torch.bfloat16).as_strided((n, heads, D), (*strides, 1))
    at = [t.storage_offset() + i * strides[0] + j * strides[1] for i in range(n) for j in range(heads)]
    c = _CRows()
    attn._out_rows(c, c, t, "output q", heads, n)
    return sorted(at)


@pytest.mark.parametrize("n, heads, strides", [
    (3, 4, (256, 64)), (3, 4, (64, 192)), (3, 4, (264, 64)), (3, 4, (768, 192)), (5, 2, (64, 320)), (1, 4, (0, 64)), (1, 4, (8, 72)),
    (4, 1, (64, 0)), (4, 1, (72, 8)), (1, 1, (0, 0)), (0, 4, (256, 64))])
def test_rows_that_lie_apart_are_taken(n, heads, strides):
    at = check(n, heads, strides)
    assert all(b - a >= D for a, b in zip(at, at[1:]))


@pytest.mark.parametrize("n, heads, strides", [
    (2, 4, (0, 64)), (3, 4, (256, 0)), (3, 4, (64, 64)), (3, 4, (128, 64)), (3, 4, (248, 64)), (3, 4, (64, 128)), (5, 2, (64, 312)),
    (2, 2, (56, 512)), (2, 2, (512, 56)), (1, 4, (512, 56)), (4, 1, (56, 512))])
def test_rows_that_overlap_are_refused(n, heads, strides):
    with pytest.raises(ValueError, match="overlap"):
        check(n, heads, strides)
