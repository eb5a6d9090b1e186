"""The serving example with positions that rotate queries and keys, over every type
of cache: greedy speculative decoding must emit the target's own greedy tokens."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_step.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    spec = importlib.util.spec_from_file_location("serving_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def recomputed(example, model, tokens):
    """Target logits of every position of one sequence, its rotation and attention in plain torch."""
    d, n = model.d, len(tokens)
    table = model.rope(n).table[:, None]
    c, s = table[..., :d // 2], table[..., d // 2:]

    def turn(x):
        a, b = x.float()[..., :d // 2], x.float()[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1).bfloat16()

    def attention(layer, q, k, v):
        group = model.hq // model.hkv
        q, k, v = turn(q).float(), turn(k).float().repeat_interleave(group, 1), v.float().repeat_interleave(group, 1)
        s = torch.einsum("nhd,lhd->hnl", q, k) * d ** -0.5
        s.masked_fill_(torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1), -float("inf"))
        return torch.einsum("hnl,lhd->nhd", torch.softmax(s, -1), v).bfloat16()

    return model.forward(torch.tensor(tokens, device="cuda"), attention).float()


def test_greedy_steps_emit_the_targets_tokens(example):
    model = example.Model(vocab=512, seed=3, theta=10000.0)
    prompts = [[1], list(range(40)), [7] * 129]
    server = example.Server(model, 3, 300, k=3)
    texts = [p + [t] for p, t in zip(prompts, server.prefill(prompts).tolist())]
    for _ in range(6):
        tokens, tau = server.step(torch.zeros(3, device="cuda"))
        for text, row, n in zip(texts, tokens.tolist(), tau.tolist()):
            assert 0 <= n <= 3 and row[n] >= 0 and all(t == -1 for t in row[n + 1:])
            text += row[:n + 1]
    assert server.attn.get_error() == 0 and server.verifier.get_error() == (0, 0)
    for prompt, text, length in zip(prompts, texts, server.kv_len.tolist()):
        assert length == len(text) - 1
        logits = recomputed(example, model, text)
        best = logits.max(-1).values
        for i in range(len(prompt), len(text)):
            # bf16 activations: two roundings (2^-8 each) of logits of a few units at each of two layers, as without rotation
            assert best[i - 1] - logits[i - 1, text[i]] <= 2.0 ** -5 * best[i - 1].abs()


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("rope", [[], ["--rope"]])
def test_sampled_steps_run(example, cache, rope, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["serving_step.py", "--steps", "3", "--cache", cache, *rope])
    example.main()
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 3 and all("accepted" in line for line in lines)
