"""Batches whose token tensors have rows that belong to no sequence: a program that
captured its calls for a fixed number of tokens pads them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests._attn import World, assert_attention  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    return sv


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("before, after", [(0, 1), (0, 40), (5, 0), (3, 200)])
def test_rows_of_no_sequence_are_left_alone_and_are_no_error(lib, before, after, dtype):
    w = World([8, 0, 3], [100, 4, 30], 8, 2, 64, 16, dtype, seed=20)
    attn = lib.SpecAttention(w.hq, w.hkv, w.d, len(w.new))
    tensors, cu, kv_len, table = w.to("cuda")
    pool = lib.KVPool(tensors["k"], tensors["v"], tensors["k_scale"], tensors["v_scale"])
    cu, n = cu + before, before + w.n + after
    rows = slice(before, before + w.n)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[rows] = False

    def padded(x):
        y = torch.full((n, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda")
        y[rows] = x.cuda()
        return y

    out = {"out": torch.full((n, w.hq, w.d), 7.0, dtype=BF16, device="cuda"), "lse": torch.full((n, w.hq), 7.0, device="cuda")}
    attn.attend(pool, padded(w.q), cu, kv_len, table, out=out)
    assert attn.get_error() == lib.SV_OK
    assert_attention(out["out"][rows], out["lse"][rows], w.expect_attention())
    assert (out["out"][rest] == 7).all() and (out["lse"][rest] == 7).all()

    back = {name: torch.full((n, w.hkv, w.d), 7.0, dtype=BF16, device="cuda") for name in ("k", "v")}
    attn.read(pool, cu, kv_len, table, n_tokens=n, out=back)
    assert attn.get_error() == lib.SV_OK
    for name, cached in (("k", w.kc), ("v", w.vc)):
        ref = np.concatenate([x[w.kv[b] - m:] for b, (x, m) in enumerate(zip(cached, w.new))])
        assert np.array_equal(back[name][rows].double().cpu().numpy(), ref)
        assert (back[name][rest] == 7).all()

    exact = [t.clone() for t in (pool.k.view(torch.uint8), pool.v.view(torch.uint8))]
    attn.append(pool, padded(w.k_new), padded(w.v_new), cu, kv_len, table)
    assert attn.get_error() == lib.SV_OK
    changed = sum((t != x).any(-1).any(1).sum().item() for t, x in zip((pool.k.view(torch.uint8), pool.v.view(torch.uint8)), exact))
    assert 0 < changed <= 2 * w.n                    # slots of the tokens, and no others

    for b, m in enumerate(w.new):
        w.kc[b], w.vc[b] = (x[w.cu[b]:w.cu[b + 1]].double().numpy() for x in (w.k_new, w.v_new))
        w.kv[b] = m
    out = {"out": torch.full((n, w.hq, w.d), 7.0, dtype=BF16, device="cuda"), "lse": torch.full((n, w.hq), 7.0, device="cuda")}
    attn.prompt(padded(w.q), padded(w.k_new), padded(w.v_new), cu, out=out)
    assert attn.get_error() == lib.SV_OK
    assert_attention(out["out"][rows], out["lse"][rows], w.expect_attention())
    assert (out["out"][rest] == 7).all() and (out["lse"][rest] == 7).all()


def test_wrong_row_ranges_are_still_reported(lib):
    w = World([8, 4], [10, 30], 8, 2, 64, 16, BF16, seed=21)
    attn = lib.SpecAttention(w.hq, w.hkv, w.d, 2)
    tensors, _, kv_len, table = w.to("cuda")
    pool = lib.KVPool(tensors["k"], tensors["v"])
    for bad in ([0, 9, 5], [-3, 8, 12], [0, 8, 99]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        attn.append(pool, w.k_new.cuda(), w.v_new.cuda(), cu, kv_len, table)
        assert attn.get_error() == lib.SV_ERR_DATA
        attn.read(pool, cu, kv_len, table, n_tokens=w.n)
        assert attn.get_error() == lib.SV_ERR_DATA
