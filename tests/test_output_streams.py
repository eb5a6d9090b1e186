"""Outputs that a call allocates belong to the stream that it runs on, and are kept until the current stream is past
them too: the calls of SpecAttention without a GPU, over a library that records its arguments."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_verification_68_gb300 import _native, attention  # noqa: E402

BF16, HQ, HKV, D, N = torch.bfloat16, 4, 2, 64, 3
CURRENT, SIDE = (types.SimpleNamespace(cuda_stream=x) for x in (7, 11))


class Library:
    """Every entry point succeeds; `streams` are the last arguments."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            if name not in ("spec_attn_init", "spec_attn_destroy"):
                self.streams.append(args[-1])
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    """A handle on the CPU, and what happened: (stream, address) of each allocation, (address, stream) of each mark."""
    seen = types.SimpleNamespace(made=[], marked=[], lib=Library())
    on = [CURRENT]

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    empty = torch.empty

    def noted(*args, **kw):
        t = empty(*args, **kw)
        seen.made.append((on[-1].cuda_stream, t.data_ptr()))
        return t

    monkeypatch.setattr(_native, "load", lambda: seen.lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: on[-1])
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.marked.append((t.data_ptr(), s.cuda_stream)))
    attn = attention.SpecAttention(HQ, HKV, D, 1)
    attn.device, attn._current = torch.device("cpu"), lambda: on[-1].cuda_stream
    monkeypatch.setattr(torch, "empty", noted)
    return attn, seen


def calls(attn):
    pool = attention.KVPool(*(torch.zeros((1, HKV, 16, D), dtype=BF16) for _ in range(2)))
    q, k = torch.zeros((N, HQ, D), dtype=BF16), torch.zeros((N, HKV, D), dtype=BF16)
    where = (torch.tensor([0, N], dtype=torch.int32), torch.tensor([N], dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32))
    rope = attention.Rope(torch.zeros((16, D)))
    return {"attend": lambda **kw: attn.attend(pool, q, *where, want_lse=True, **kw),
            "prompt": lambda **kw: attn.prompt(q, k, k, where[0], want_lse=True, **kw),
            "read": lambda **kw: attn.read(pool, *where, n_tokens=N, **kw),
            "append_rotated": lambda **kw: attn.append_rotated(pool, k, k, *where, rope, q=q, want_k=True, **kw)}


@pytest.mark.parametrize("name", ["attend", "prompt", "read", "append_rotated"])
def test_outputs_belong_to_the_stream_of_the_call(world, name):
    attn, seen = world
    call = calls(attn)[name]
    for stream, runs_on in ((None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE)):
        seen.made.clear(), seen.marked.clear(), seen.lib.streams.clear()
        out = call(stream=stream)
        outputs = [t.data_ptr() for t in out.values()]
        assert len(outputs) == 2 and seen.lib.streams == [runs_on.cuda_stream]
        assert seen.made == [(runs_on.cuda_stream, x) for x in outputs]
        assert seen.marked == ([] if runs_on is CURRENT else [(x, CURRENT.cuda_stream) for x in outputs])
        seen.made.clear(), seen.marked.clear()
        assert call(stream=stream, out=out) is out and seen.made == seen.marked == []      # the caller's own: left alone
