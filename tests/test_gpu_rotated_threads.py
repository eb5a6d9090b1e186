"""Handles of two threads on streams of their own, sharing one table of angles, one
with positions of its own: each gets what it gets alone."""
import threading

import pytest

torch = pytest.importorskip("torch")
from tests._attn4 import FOUR, rope_table  # noqa: E402

pytestmark = pytest.mark.gpu


def test_two_threads_share_a_table():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    g = torch.Generator(device="cuda").manual_seed(0)
    n, hq, hkv, d = 40, 8, 2, 64
    rope = sv.Rope(rope_table(1000, d).cuda())
    cu, kv = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([n + 60], dtype=torch.int32, device="cuda")
    table = torch.arange(7, dtype=torch.int32, device="cuda")[None]
    q, k, v = (torch.randn((n, h, d), generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv))
    own = torch.randint(1000, (n,), generator=g, device="cuda", dtype=torch.int32)
    side = []
    for positions in (None, own):
        attn = sv.SpecAttention(hq, hkv, d, 1)
        pool = attn.alloc_pool(7, 16, FOUR)
        alone = attn.append_rotated(pool, k, v, cu, kv, table, rope, q=q, positions=positions)["q"]
        side.append((attn, pool, positions, alone, pool.k.view(torch.uint8).clone(), torch.cuda.Stream()))
    assert not torch.equal(side[0][3], side[1][3])
    torch.cuda.synchronize()
    wrong = []

    def work(attn, pool, positions, alone, codes, stream):
        out = {"q": torch.empty_like(q)}
        with torch.cuda.stream(stream):
            for _ in range(300):
                attn.append_rotated(pool, k, v, cu, kv, table, rope, q=q, positions=positions, out=out)
                if not torch.equal(out["q"], alone) or not torch.equal(pool.k.view(torch.uint8), codes):
                    wrong.append(positions is None)
                    return

    threads = [threading.Thread(target=work, args=s) for s in side]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and all(s[0].get_error() == sv.SV_OK for s in side)
