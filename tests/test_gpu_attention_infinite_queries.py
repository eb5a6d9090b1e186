"""Query rows that are not finite, over every kind of cache and for prompts: what they give themselves, and that the
rows beside them give what they give without them."""
import pytest

torch = pytest.importorskip("torch")
from tests._attn4 import FOUR  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kv", [1, 5, 700])
@pytest.mark.parametrize("hq, n", [(2, 1), (16, 1), (4, 4), (40, 1), (8, 20)])
@pytest.mark.parametrize("dtype", [BF16, E4M3, FOUR, None])                    # None: a prompt
def test_rows_of_infinite_queries(dtype, hq, n, kv):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    d = 64
    attn = sv.SpecAttention(hq, 1, d, 1)
    n, kv = (max(n, 3), max(n, 3)) if dtype is None else (min(n, kv), kv)
    g = torch.Generator(device="cuda").manual_seed(0)
    k = torch.rand((kv, 1, d), generator=g, device="cuda").add(0.5).bfloat16()           # all above 0
    q, v = (torch.randn((m, h, d), generator=g, device="cuda").bfloat16() for m, h in ((n, hq), (kv, 1)))
    if dtype is not None:
        pool = attn.alloc_pool(44, 16, dtype)
        table = torch.arange(44, dtype=torch.int32, device="cuda")[None]
        attn.append(pool, k, v, ints(0, kv), ints(kv), table)

    def call(q):
        got = attn.prompt(q, k, v, ints(0, n), want_lse=True) if dtype is None else attn.attend(pool, q, ints(0, n), ints(kv), table, want_lse=True)
        assert attn.get_error() == sv.SV_OK
        return got["out"].flatten(0, 1), got["lse"].flatten()

    want, want_lse = call(q)
    rows = n * hq
    for value in (float("-inf"), float("inf"), float("nan")):
        odd = q.clone()
        odd.view(rows, d)[rows // 2, 3] = value
        out, lse = call(odd)
        mine = torch.arange(rows, device="cuda") == rows // 2
        assert torch.equal(out[~mine], want[~mine]) and torch.equal(lse[~mine], want_lse[~mine])
        if value == float("-inf"):                                          # every score is -inf
            assert (out[mine] == 0).all() and (lse[mine] == value).all()
        else:
            assert torch.isnan(out[mine]).all() and torch.isnan(lse[mine]).all()
