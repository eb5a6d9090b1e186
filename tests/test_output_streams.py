"""Outputs that a call allocates belong to the stream that it runs on, and are kept until the current stream is past
them too: the calls of SpecAttention and SpecVerifier without a GPU, over a library that records its arguments."""
import contextlib
import ctypes
import types

import pytest

torch = pytest.importorskip("torch")
import speculative_decoding_verification_68_gb300 as sv  # noqa: E402
from speculative_decoding_verification_68_gb300 import _native, attention  # noqa: E402

BF16, HQ, HKV, D, N = torch.bfloat16, 4, 2, 64, 3
CURRENT, SIDE = (types.SimpleNamespace(cuda_stream=x) for x in (7, 11))


class Library:
    """Every entry point succeeds; `streams` are the last arguments."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            if not name.endswith(("_init", "_destroy")):
                self.streams.append(args[-1].value if isinstance(args[-1], ctypes.c_void_p) else args[-1])
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

    def noted(make):
        def call(*args, **kw):
            t = make(*args, **kw)
            seen.made.append((on[-1].cuda_stream, t.data_ptr()))
            return t
        return call

    monkeypatch.setattr(_native, "load", lambda: seen.lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: on[-1])
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.marked.append((t.data_ptr(), s.cuda_stream)))
    attn = attention.SpecAttention(HQ, HKV, D, 1)
    verifier = sv.SpecVerifier(2, 3, 8, torch.float32)
    attn.device = verifier.device = torch.device("cpu")
    attn._current = lambda: on[-1].cuda_stream
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, noted(getattr(torch, name)))
    return attn, verifier, seen


def calls(attn, verifier):
    pool = attention.KVPool(*(torch.zeros((1, HKV, 16, D), dtype=BF16) for _ in range(2)))
    q, k = torch.zeros((N, HQ, D), dtype=BF16), torch.zeros((N, HKV, D), dtype=BF16)
    where = (torch.tensor([0, N], dtype=torch.int32), torch.tensor([N], dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32))
    rope = attention.Rope(torch.zeros((16, D)))
    return {"attend": lambda **kw: attn.attend(pool, q, *where, want_lse=True, **kw),
            "prompt": lambda **kw: attn.prompt(q, k, k, where[0], want_lse=True, **kw),
            "read": lambda **kw: attn.read(pool, *where, n_tokens=N, **kw),
            "append_rotated": lambda **kw: attn.append_rotated(pool, k, k, *where, rope, q=q, want_k=True, **kw),
            **verifications(verifier)}


def verifications(v):
    target, draft, tokens = torch.zeros((2, 4, 8)), torch.zeros((2, 3, 8)), torch.zeros((2, 3), dtype=torch.int32)
    chains = (target, draft, tokens, torch.ones(2), torch.zeros((2, 4)))
    return {"verify": lambda **kw: v.verify(*chains, want_tv=True, want_entropy=True, **kw), "verify_lazy": lambda **kw: v.verify_lazy(*chains, **kw),
            "loss_grad": lambda **kw: v.loss_grad(target, draft, torch.ones(2), **kw), "verify_tv": lambda **kw: v.verify_tv(target, draft, torch.ones(2), **kw)}


COUNT = dict(attend=2, prompt=2, read=2, append_rotated=2, verify=7, verify_lazy=2, loss_grad=2, verify_tv=1)


@pytest.mark.parametrize("name", list(COUNT))
def test_outputs_belong_to_the_stream_of_the_call(world, name):
    attn, verifier, seen = world
    call = calls(attn, verifier)[name]
    for stream, runs_on in ((None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE)):
        seen.made.clear(), seen.marked.clear(), seen.lib.streams.clear()
        out = call(stream=stream)
        outputs = [t.data_ptr() for t in (out.values() if isinstance(out, dict) else (out,))]
        assert len(outputs) == COUNT[name] and seen.lib.streams == [runs_on.cuda_stream]
        assert seen.made == [(runs_on.cuda_stream, x) for x in outputs]
        assert seen.marked == ([] if runs_on is CURRENT else [(x, CURRENT.cuda_stream) for x in outputs])
        seen.made.clear(), seen.marked.clear()
        assert call(stream=stream, out=out) is out and seen.made == seen.marked == []      # the caller's own: left alone
