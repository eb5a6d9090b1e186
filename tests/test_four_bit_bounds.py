"""How far values of a 4-bit cache may be from what was appended, as the header states it: blocks from next to their
vector's largest element to where nothing is left of them, and vectors down to the smallest numbers of bf16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests._attn4 import BLOCK, FOUR, quantise4, values4  # noqa: E402


def vectors():
    """[n, 1, 64] bf16: a block with the vector's largest element, and three below it by up to 2^-24."""
    g = np.random.default_rng(3)
    n = 4000
    x = g.uniform(-1, 1, (n, 4, BLOCK))
    x[..., 0] = 1                                                       # a block's largest
    down = np.concatenate([np.zeros((n, 1)), g.uniform(-24, 0, (n, 3))], 1)
    size = g.uniform(-130, 120, (n, 1, 1)) * (g.random((n, 1, 1)) < 0.5)
    x = x * 2.0 ** (down[..., None] + size) * g.uniform(1, 2, (n, 1, 1))
    x[0], x[0, 0, 0], x[0, 1, 0] = 0, 1.0, 0.9 * 2.0 ** -18             # above 2^-19 of the largest: the least scale
    x[1], x[1, 0, 0], x[1, 1, 0] = 0, 1.0, 0.9 * 2.0 ** -19
    return torch.from_numpy(x.reshape(n, 1, 64)).bfloat16()


def assert_bounds(x, got):
    x, got = (y.reshape(-1, 4, BLOCK) for y in (x, got))
    top = np.abs(x).max((1, 2), keepdims=True)
    most = np.abs(x).max(2, keepdims=True)
    whole, gone = (most > 2.0 ** -13 * top) & (most > 2.0 ** -123), (most < 2.0 ** -19 * top) | (most < 2.0 ** -128)
    assert whole[:, 1:].sum() > 2000 and gone.sum() > 1000 and (~whole & ~gone).sum() > 1000
    off = np.abs(got - x)
    assert (off <= 0.18 * most)[np.broadcast_to(whole, off.shape)].all()
    assert (off <= 2.0 ** -4 * most)[whole & (np.abs(x) == most)].all()
    assert not got[np.broadcast_to(gone, got.shape)].any()
    # a largest of 1 gives 2^-11; 0.9 * 2^-7 of that would have a scale of 0.6 * 2^-9, has 2^-9, and is 3.6 of it: code 4
    assert got[0, 1, 0] == 4 * 2.0 ** -20 and not got[1, 1].any()


def test_bounds_of_the_definition():
    x = vectors().double().numpy()
    assert_bounds(x, values4(*quantise4(x)))


@pytest.mark.gpu
def test_bounds_of_the_cache():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    x = vectors()
    n = len(x)
    attn = sv.SpecAttention(1, 1, 64, 1)
    pool = attn.alloc_pool(-(-n // 128), 128, FOUR)
    cu, kv = (torch.tensor(y, dtype=torch.int32, device="cuda") for y in ([0, n], [n]))
    table = torch.arange(pool.num_pages, dtype=torch.int32, device="cuda")[None]
    attn.append(pool, x.cuda(), x.cuda(), cu, kv, table)
    back = attn.read(pool, cu, kv, table, n_tokens=n)
    assert attn.get_error() == sv.SV_OK
    want = torch.from_numpy(values4(*quantise4(x.double().numpy()))).bfloat16()      # exact but below bf16's normal range
    for name in ("k", "v"):
        assert torch.equal(back[name].cpu(), want), name
