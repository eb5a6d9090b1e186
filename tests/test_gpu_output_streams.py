"""Outputs that a call on another stream than the current one allocates are of that stream's memory, and hold what
the call on the current stream gives."""
import pytest

torch = pytest.importorskip("torch")
from tests._attn4 import rope_table  # noqa: E402

pytestmark = pytest.mark.gpu


def stream_of(t):
    """The stream whose memory a tensor lies in, as the allocator has it."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def test_outputs_of_a_call_on_a_side_stream():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    n, hq, hkv, d = 70, 8, 2, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    attn = sv.SpecAttention(hq, hkv, d, 1)
    pool = attn.alloc_pool(5, 16)
    q, k, v = (torch.randn((n, h, d), generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv))
    cu, kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n]))
    where = (cu, kv, torch.arange(5, dtype=torch.int32, device="cuda")[None])
    rope = sv.Rope(rope_table(n, d).cuda())
    side = torch.cuda.Stream()
    for call in (lambda **kw: attn.append_rotated(pool, k, v, *where, rope, q=q, want_k=True, **kw), lambda **kw: attn.read(pool, *where, n_tokens=n, **kw),
                 lambda **kw: attn.attend(pool, q, *where, want_lse=True, **kw), lambda **kw: attn.prompt(q, k, v, cu, want_lse=True, **kw)):
        want = call()
        torch.cuda.synchronize()
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for name, t in want.items():
            assert stream_of(t) == torch.cuda.current_stream().cuda_stream and stream_of(got[name]) == side.cuda_stream
            assert torch.equal(got[name], t), name
        torch.cuda.synchronize()
    assert attn.get_error() == sv.SV_OK
