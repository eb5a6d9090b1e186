"""Batches of many rows and blocks, which the attention kernels with two tiles of rows a CTA
run: packed prompts and cached chunks of both head dimensions, against float64 on the GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_68_gb300 as sv
    sv.build()
    return sv


def takes_two_tiles(n_seqs, n_tokens, hq, hkv, keys):
    """The library's rule: more rows per sequence and head than a tile holds, and at least 12
    blocks of two tiles for every SM."""
    rows = -(-n_tokens * (hq // hkv) // n_seqs)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return rows > 128 and n_seqs * hkv * -(-rows // 256) * (keys // 128 + 1) >= 12 * sms


def reference(q, k, v, first):
    """One sequence: q [n, hq, D], k and v [L, hkv, D]; row i sees keys 0 .. first + i.  Output, log
    of the sum, and bounds of their errors.  Rounding to bf16 changes a number by at most u = 2^-8 of it.
    The weights p are rounded to bf16 before their product with the values: u sum p|v|.  The sum they are
    divided by is corrected by what that did to some of them: at most u of it, u |out|.  The output is
    rounded: u |out|.  Products of these and 32-bit arithmetic: well below 2^-12 sum p|v|.  The log of the
    sum moves by no more than a score: a 32-bit sum of D <= 128 exact products."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    out, lse, tol, tol_lse = (torch.empty(s, dtype=torch.float64, device=q.device) for s in ((n, hq, d), (n, hq)) * 2)
    last = first + torch.arange(n, device=q.device)
    over = torch.arange(k.shape[0], device=q.device)[None] > last[:, None]
    for h in range(hq):
        kk, vv, qq = k[:, h // group].double(), v[:, h // group].double(), q[:, h].double()
        s = (qq @ kk.T * d ** -0.5).masked_fill_(over, -INF)
        lse[:, h] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[:, h, None])
        out[:, h] = p @ vv
        tol[:, h] = 2.0 ** -7 * out[:, h].abs() + (2.0 ** -8 + 2.0 ** -12) * (p @ vv.abs())
        reach = (qq.abs() @ kk.abs().T).masked_fill_(over, 0).amax(-1) * d ** -0.5
        tol_lse[:, h] = 2.0 ** -16 * (1 + reach)
    return out, lse, tol, tol_lse


def assert_rows(got, rows, q, k, v, first, columns=slice(None)):
    out, lse, tol, tol_lse = reference(q[rows], k, v, first)
    x = got["out"][rows].double()
    assert ((x - out).abs() <= tol)[..., columns].all()
    assert ((got["lse"][rows].double() - lse).abs() <= tol_lse).all()


def tensors(seed, n, hq, hkv, d):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(heads):
        x = torch.randn((n, heads, d), generator=g, device="cuda")
        return (x * torch.exp(0.5 * torch.randn((n, heads, 1), generator=g, device="cuda"))).bfloat16()

    return make(hq), make(hkv), make(hkv)


def starts(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def paged(attn, k, v, lens, page):
    """A pool with a shuffled table that holds the packed k and v; its other slots are NaN."""
    need = [-(-n // page) for n in lens]
    pool = attn.alloc_pool(sum(need) + 2, page)
    pool.k.fill_(NAN), pool.v.fill_(NAN)
    order = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(1)).int()
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32)
    for b, c in enumerate(need):
        table[b, :c] = order[sum(need[:b]):sum(need[:b]) + c]
    table, kv_len = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    attn.append(pool, k, v, starts(lens), kv_len, table)
    return pool, kv_len, table


PROMPTS = [  # lengths, hq, hkv, d
    ([2900, 1, 3001, 1700], 32, 8, 128),
    ([2900, 1, 3001, 1700], 32, 8, 64),
    ([4099], 10, 2, 64),                             # 25 tokens a tile
    ([4099], 10, 2, 128),
    ([1, 5, 2900, 130, 0, 257, 3000], 64, 8, 128),   # items of one block beside long ones
    ([1, 5, 2900, 130, 0, 257, 3000], 32, 16, 64),
    ([650], 512, 8, 64),                             # 2 tokens a tile
    ([1900, 1900], 16, 16, 128),                     # one row a token
    ([2049, 1950], 16, 16, 64),
    ([60] * 200, 64, 8, 128),                        # every item of one block: weights in two parts
    ([60] * 200, 64, 8, 64),
]


@pytest.mark.parametrize("lengths, hq, hkv, d", PROMPTS)
def test_long_prompts(lib, lengths, hq, hkv, d):
    n = sum(lengths)
    assert takes_two_tiles(len(lengths), n, hq, hkv, n // len(lengths) // 2)
    q, k, v = tensors(30, n, hq, hkv, d)
    attn = lib.SpecAttention(hq, hkv, d, len(lengths))
    cu = starts(lengths)
    got = attn.prompt(q, k, v, cu, want_lse=True)
    again = attn.prompt(q, k, v, cu, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])
    at = cu.tolist()
    for b in {0, len(lengths) // 2, len(lengths) - 1} | {b for b, x in enumerate(lengths) if x > 200}:
        rows = slice(at[b], at[b + 1])
        assert_rows(got, rows, q, k[rows], v[rows], 0)


CHUNKS = [  # new, old, hq, hkv, d, page
    ([400, 512, 300], [6000, 2000, 4001], 32, 8, 128, 64),
    ([400, 512, 300], [6000, 2000, 4001], 32, 8, 64, 32),
    ([513, 1, 700], [0, 5000, 3000], 64, 8, 64, 16),
    ([513, 1, 700], [0, 5000, 3000], 64, 8, 128, 128),
    ([1000], [3000], 28, 4, 64, 16),                 # 18 tokens a tile
    ([257] * 12, [100 * b for b in range(12)], 16, 16, 64, 16),
]


@pytest.mark.parametrize("new, old, hq, hkv, d, page", CHUNKS)
def test_long_chunks(lib, new, old, hq, hkv, d, page):
    lens = [a + b for a, b in zip(new, old)]
    assert takes_two_tiles(len(new), sum(new), hq, hkv, sum(lens) // len(lens))
    _, k, v = tensors(31, sum(lens), 1, hkv, d)
    q, _, _ = tensors(32, sum(new), hq, 1, d)
    attn = lib.SpecAttention(hq, hkv, d, len(new))
    pool, kv_len, table = paged(attn, k, v, lens, page)
    cu, at = starts(new), starts(lens).tolist()
    got = attn.attend(pool, q, cu, kv_len, table, want_lse=True)
    again = attn.attend(pool, q, cu, kv_len, table, want_lse=True)
    assert attn.get_error() == lib.SV_OK
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])
    for b in range(len(new)):
        rows, keys = slice(cu[b].item(), cu[b + 1].item()), slice(at[b], at[b + 1])
        assert_rows(got, rows, q, k[keys], v[keys], old[b])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cached", [False, True])
def test_not_finite_values_of_later_tokens(lib, cached, d):
    """Every sequence has a NaN, an infinity and a negative one at three of its tokens: rows before a
    token do not see its column's value, rows from it on have it."""
    hq, hkv, lens, page = 32, 8, [2500, 131, 3100], 32
    n = sum(lens)
    assert takes_two_tiles(len(lens), n, hq, hkv, n // len(lens) // (1 if cached else 2))
    q, k, v = tensors(33, n, hq, hkv, d)
    at = starts(lens).tolist()
    clean = v.clone()
    bad = [[(m // 3, 5, NAN), (m // 2, 6, INF), (m - 1, d - 1, -INF), (m // 2 + 1, d // 2, INF)] for m in lens]
    for b, marks in enumerate(bad):
        for i, col, x in marks:
            v[at[b] + i, :, col] = x
    attn = lib.SpecAttention(hq, hkv, d, len(lens))
    cu = starts(lens)
    if cached:
        pool, kv_len, table = paged(attn, k, v, lens, page)
        calls = [lambda: attn.attend(pool, q, cu, kv_len, table, want_lse=True)] * 2
    else:
        calls = [lambda: attn.prompt(q, k, v, cu, want_lse=True)] * 2
    got, again = (f() for f in calls)
    assert attn.get_error() == lib.SV_OK
    assert torch.equal(got["out"].view(torch.int16), again["out"].view(torch.int16))
    for b, marks in enumerate(bad):
        rows = slice(at[b], at[b + 1])
        out = got["out"][rows].float()
        columns = torch.ones(d, dtype=torch.bool, device="cuda")
        for i, col, x in marks:
            columns[col] = False
            seen = out[i:, :, col]
            # where 32 bits hold the token's weight; as 0 it makes NaN of an infinity
            s = torch.einsum("nhd,hd->nh", q[rows][i:].double(), k[at[b] + i].double().repeat_interleave(hq // hkv, 0)) * d ** -0.5
            held = s - got["lse"][rows][i:].double() >= -126 * np.log(2.0)
            assert torch.isnan(seen).all() if x != x else (seen == x)[held].all() and ((seen == x) | torch.isnan(seen)).all()
            assert held.float().mean() > 0.999
            ref, _, tol, _ = reference(q[rows][:i], k[rows][:i], clean[rows][:i], 0)
            assert ((out[:i, :, col].double() - ref[..., col]).abs() <= tol[..., col]).all()
        assert_rows(got, rows, q, k[rows], clean[rows], 0, columns)


@pytest.mark.parametrize("cached", [False, True])
def test_keys_that_are_nan_reach_only_later_rows(lib, cached):
    hq, hkv, d, lens = 32, 8, 128, [2500, 131, 3100]
    q, k, v = tensors(34, sum(lens), hq, hkv, d)
    at = starts(lens).tolist()
    bad = k.clone()
    for b, m in enumerate(lens):
        bad[at[b] + m // 2, :, 3] = NAN
    attn = lib.SpecAttention(hq, hkv, d, len(lens))
    if cached:
        pool, kv_len, table = paged(attn, bad, v, lens, 16)
        got = attn.attend(pool, q, starts(lens), kv_len, table, want_lse=True)
    else:
        got = attn.prompt(q, bad, v, starts(lens), want_lse=True)
    assert attn.get_error() == lib.SV_OK
    for b, m in enumerate(lens):
        clean = slice(at[b], at[b] + m // 2)
        assert_rows(got, clean, q, k[clean], v[clean], 0)
        assert torch.isnan(got["out"][at[b] + m // 2:at[b + 1]]).all()


@pytest.mark.parametrize("new, old, hq, hkv, d", [
    ([113], [5983], 64, 8, 128),                     # one tile: few blocks
    ([113], [5983], 64, 8, 64),
    ([400, 512], [6000, 2000], 32, 8, 128),          # two tiles
    ([900, 1], [30, 0], 64, 8, 64),
])
def test_with_a_bound_of_the_lengths_the_tables_width_changes_nothing(lib, new, old, hq, hkv, d):
    """A server's table has room for its longest sequence; max_kv decides how a chunk runs."""
    page, lens = 64, [a + b for a, b in zip(new, old)]
    _, k, v = tensors(35, sum(lens), 1, hkv, d)
    q, _, _ = tensors(36, sum(new), hq, 1, d)
    attn = lib.SpecAttention(hq, hkv, d, len(new))
    pool, kv_len, table = paged(attn, k, v, lens, page)
    cu, at = starts(new), starts(lens).tolist()
    got = attn.attend(pool, q, cu, kv_len, table, want_lse=True, max_kv=max(lens))
    for width in (table.shape[1] + 1, 131072 // page, 1 << 20):
        wide = torch.full((len(new), width), -1, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        again = attn.attend(pool, q, cu, kv_len, wide, want_lse=True, max_kv=max(lens))
        assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])
    low = attn.attend(pool, q, cu, kv_len, table, want_lse=True, max_kv=1)     # a wrong bound costs time only
    assert attn.get_error() == lib.SV_OK
    for b in range(len(new)):
        rows, keys = slice(cu[b].item(), cu[b + 1].item()), slice(at[b], at[b + 1])
        assert_rows(got, rows, q, k[keys], v[keys], old[b])
        assert_rows(low, rows, q, k[keys], v[keys], old[b])
    with pytest.raises(ValueError, match="max_kv"):
        attn.attend(pool, q, cu, kv_len, table, max_kv=-1)
