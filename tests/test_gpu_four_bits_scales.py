"""Blocks that take each of the 126 scales, by append and by the append that rotates, each into a pool whose six parts
hold other bytes before: what a call leaves unwritten is seen."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import _attn  # noqa: E402
from tests._attn4 import FOUR, bytes_of, quantise4  # noqa: E402

pytestmark = pytest.mark.gpu
PARTS = ("k", "v", "k_scale", "v_scale", "k_block", "v_block")


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("shift", [0, -100, 100])
@pytest.mark.parametrize("d", [64, 128])
def test_every_scale_is_written(d, shift, rotated):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    blocks = d // 16 - 1                                                    # and one that makes the exponent `shift`
    n = 126 // blocks
    scales = _attn.e4m3_value(np.arange(1, 127, dtype=np.uint8)).reshape(n, blocks)
    g = np.random.default_rng(6)
    x = np.zeros((n, 1, d // 16, 16))
    x[:, 0, blocks] = 2688.0
    x[:, 0, :blocks] = scales[..., None] * g.uniform(-6, 6, (n, blocks, 16))
    x[:, 0, :blocks, 0] = 6 * scales
    x = torch.from_numpy(x.reshape(n, 1, d) * 2.0 ** shift).bfloat16()
    parts = quantise4(x.double().numpy())
    assert np.array_equal(parts[1][:, 0, :blocks].reshape(-1), np.arange(1, 127)) and (parts[2] == 127 + shift).all()
    attn = sv.SpecAttention(1, 1, d, 1)
    pool = attn.alloc_pool(2, 64, FOUR)
    for name in PARTS:
        getattr(pool, name).view(torch.uint8).fill_(0xAA)
    where = [torch.tensor(y, dtype=torch.int32, device="cuda") for y in ([0, n], [n], [[1, 0]])]
    if rotated:
        rope = sv.Rope(torch.cat([torch.ones((n, d // 2)), torch.zeros((n, d // 2))], 1).cuda())
        attn.append_rotated(pool, x.cuda(), x.cuda(), *where, rope)
    else:
        attn.append(pool, x.cuda(), x.cuda(), *where)
    assert attn.get_error() == sv.SV_OK
    got = bytes_of(pool)
    for part, y in zip(("", "_scale", "_block"), (parts[0], parts[2], parts[1])):
        for name in ("k", "v"):
            want = np.full(got[name + part].shape, 0xAA, np.uint8)
            for t in range(n):
                want[1 - t // 64, 0, t % 64] = y[t, 0]
            assert np.array_equal(got[name + part].numpy(), want), name + part
