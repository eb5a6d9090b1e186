"""The paged key-value cache and the attention of a verification step.

A thin binding over the ``spec_attn_*`` functions of ``libspec_verify.so``
(see ``include/spec_attn.h`` for the method, the layouts and what a sequence's
positions are).  Per layer, a verification step of k drafts is

    attn = SpecAttention(q_heads=64, kv_heads=8, head_dim=128, max_seqs=256)
    pool = attn.alloc_pool(num_pages, page_size=64, dtype=torch.float8_e4m3fn)
    attn.append(pool, k, v, cu, kv_len, page_table)
    out = attn.attend(pool, q, cu, kv_len, page_table)["out"]

and, once SpecVerifier has given the accepted lengths, a sequence drops its
rejected tokens by lowering its kv_len.  Where positions rotate queries and keys,

    rope = Rope(table, interleaved=False)
    q = attn.append_rotated(pool, k, v, cu, kv_len, page_table, rope, q=q)["q"]

does both on the way into the cache.

Calls run on the current stream, or on `stream` where it is given: the caller
orders it behind what makes the inputs, and what reads the outputs behind it.
Outputs are allocated where `out` is not given; rows of tokens that lie in no
sequence (behind cu[-1]) are not written, so in new tensors they hold anything.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native

SV_E4M3, SV_E2M1 = 2, 3
SCALE_BLOCK = 16            # elements of an e2m1 vector that share a scale
PAGE_SIZES = (16, 32, 64, 128)


class _CPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("k_block", ctypes.c_void_p), ("v_block", ctypes.c_void_p)]


class _CBatch(ctypes.Structure):
    _fields_ = [("cu", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("max_kv", ctypes.c_int32)]


class _CRope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("max_positions", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class _CRows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


def _same_device(t, device) -> bool:
    return t.device.type == device.type and (device.type != "cuda" or t.device.index == device.index)


def _check(t, name: str, dtype, shape: tuple, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not _same_device(t, device):
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def check_rows(t, name: str, heads: int, head_dim: int, device, n_tokens: int | None = None) -> int:
    """Checks a token tensor [n_tokens, heads, head_dim]; returns n_tokens.  It may
    be a slice of a larger tensor (a fused projection's output, for one) as long as
    its last dimension is contiguous and every vector is 16-byte aligned."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {torch.bfloat16}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim or (n_tokens is not None and shape[0] != n_tokens):
        raise ValueError(f"{name}: shape {tuple(shape)}, expected "
                         f"({'n_tokens' if n_tokens is None else n_tokens}, {heads}, {head_dim})")
    if shape[0]:
        if stride[2] != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        if stride[0] % 8 or stride[1] % 8 or t.data_ptr() % 16:
            raise ValueError(f"{name}: every vector must be 16-byte aligned (strides {tuple(stride)})")
    if not _same_device(t, device):
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return shape[0]


def check_sequences(cu, device, max_seqs: int, kv_len=None, page_table=None, paged: bool = True) -> int:
    """Checks the sequences' metadata (their values are checked on the device);
    returns the number of sequences."""
    if cu is None or cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu must be a [n_seqs + 1] tensor")
    n = cu.shape[0] - 1
    if n > max_seqs:
        raise ValueError(f"{n} sequences exceed the handle's max_seqs {max_seqs}")
    _check(cu, "cu", torch.int32, (n + 1,), device)
    if paged:
        _check(kv_len, "kv_len", torch.int32, (n,), device)
        if page_table is None or page_table.dim() != 2:
            raise ValueError("page_table must be a [n_seqs, max_pages] tensor")
        _check(page_table, "page_table", torch.int32, (n, page_table.shape[1]), device)
    return n


class KVPool:
    """Cache pages: k and v [num_pages, kv_heads, page_size, head_dim], bf16; or
    float8_e4m3fn with k_scale and v_scale [num_pages, kv_heads, page_size] uint8
    (a vector is code * 2^(byte - 127)); or float4_e2m1fn_x2 [..., head_dim / 2]
    with those and k_block and v_block [..., head_dim / 16] float8_e4m3fn (an
    element is code * its block's scale * 2^(byte - 127))."""

    def __init__(self, k, v, k_scale=None, v_scale=None, k_block=None, v_block=None):
        if k is None or k.dim() != 4:
            raise ValueError("k must be a [num_pages, kv_heads, page_size, head_dim] tensor")
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn, torch.float4_e2m1fn_x2):
            raise ValueError(f"unsupported cache dtype {k.dtype}")
        if k.shape[0] < 1 or k.shape[2] not in PAGE_SIZES:
            raise ValueError(f"page_size {k.shape[2]} with {k.shape[0]} pages: page_size must be one of {PAGE_SIZES}, "
                             "num_pages at least 1")
        for t, name in ((k, "k"), (v, "v")):
            _check(t, name, k.dtype, tuple(k.shape), k.device)
            if t.data_ptr() % 16:
                raise ValueError(f"{name} must be 16-byte aligned")
        four = k.dtype == torch.float4_e2m1fn_x2
        self.quantised = k.dtype != torch.bfloat16
        self.head_dim = k.shape[3] * (2 if four else 1)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if self.quantised:
                _check(t, name, torch.uint8, tuple(k.shape[:3]), k.device)
                if four and t.data_ptr() % 16:
                    raise ValueError(f"{name} must be 16-byte aligned")
            elif t is not None:
                raise ValueError(f"{name}: a bf16 pool has no scales")
        for t, name in ((k_block, "k_block"), (v_block, "v_block")):
            if four:
                _check(t, name, torch.float8_e4m3fn, (*k.shape[:3], self.head_dim // SCALE_BLOCK), k.device)
                if t.data_ptr() % 16:
                    raise ValueError(f"{name} must be 16-byte aligned")
            elif t is not None:
                raise ValueError(f"{name}: only a 4-bit pool has scales of blocks")
        self.k, self.v, self.k_scale, self.v_scale, self.k_block, self.v_block = k, v, k_scale, v_scale, k_block, v_block
        self.num_pages, self.kv_heads, self.page_size = k.shape[:3]
        self.device, self.dtype = k.device, k.dtype
        self._c = _CPool(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if self.quantised else None,
                         v_scale.data_ptr() if self.quantised else None, SV_E2M1 if four else SV_E4M3 if self.quantised else 1,
                         self.num_pages, self.page_size, k_block.data_ptr() if four else None, v_block.data_ptr() if four else None)
        self._ref = ctypes.byref(self._c)


class Rope:
    """How positions turn queries and keys: table [max_positions, rot_dim] float32
    holds the rot_dim / 2 cosines of a position, then its sines; the pairs that
    turn are neighbours (interleaved) or element i and i + rot_dim / 2."""

    def __init__(self, table, interleaved: bool = False):
        if table is None or table.dim() != 2:
            raise ValueError("table must be a [max_positions, rot_dim] tensor")
        self.max_positions, self.rot_dim = table.shape
        _check(table, "table", torch.float32, (self.max_positions, self.rot_dim), table.device)
        if not 1 <= self.max_positions < 1 << 31 or self.rot_dim < 16 or self.rot_dim % 16:
            raise ValueError(f"table: shape {tuple(table.shape)}, expected at least one position and a multiple of 16 columns")
        if table.data_ptr() % 16:
            raise ValueError("table must be 16-byte aligned")
        self.table, self.interleaved, self.device = table, bool(interleaved), table.device


class SpecAttention:
    """One library handle: attention of q_heads query heads over kv_heads key-value heads."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, max_seqs: int):
        from . import _check as check_status
        self._lib = _native.load()
        self.q_heads, self.kv_heads, self.head_dim, self.max_seqs = q_heads, kv_heads, head_dim, max_seqs
        h = ctypes.c_void_p()
        check_status(self._lib.spec_attn_init(ctypes.byref(h), q_heads, kv_heads, head_dim, max_seqs), "spec_attn_init")
        self._h = h
        index = torch.cuda.current_device()
        self.device = torch.device("cuda", index)     # the handle's GPU
        # the current stream's pointer; the public call builds a Stream object first
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._current = (lambda: raw(index)) if raw else (lambda: torch.cuda.current_stream(self.device).cuda_stream)
        # argument blocks of the calls, refilled by each (a handle is not thread-safe)
        self._batch_c, self._q_c, self._k_c, self._v_c = _CBatch(), _CRows(), _CRows(), _CRows()
        self._q_out_c, self._k_out_c, self._rope_c = _CRows(), _CRows(), _CRope()
        self._rope_ref = ctypes.byref(self._rope_c)
        self._batch_ref, self._q_ref, self._k_ref, self._v_ref, self._q_out_ref, self._k_out_ref = (
            ctypes.byref(x) for x in (self._batch_c, self._q_c, self._k_c, self._v_c, self._q_out_c, self._k_out_c))

    def close(self):
        if getattr(self, "_h", None):
            self._lib.spec_attn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _status(code: int, where: str):
        if code:
            from . import SpecVerifyError
            raise SpecVerifyError(code, where)

    def _stream(self, stream):
        return self._current() if stream is None else stream.cuda_stream

    def alloc_pool(self, num_pages: int, page_size: int = 64, dtype=torch.bfloat16) -> KVPool:
        """An empty pool for this handle's heads: bfloat16, float8_e4m3fn or float4_e2m1fn_x2."""
        shape = (num_pages, self.kv_heads, page_size, self.head_dim)
        if dtype not in (torch.float8_e4m3fn, torch.float4_e2m1fn_x2):
            return KVPool(*(torch.zeros(shape, dtype=dtype, device=self.device) for _ in range(2)))
        four = dtype == torch.float4_e2m1fn_x2
        codes = [torch.zeros((*shape[:3], shape[3] // 2 if four else shape[3]), dtype=torch.uint8, device=self.device).view(dtype) for _ in range(2)]
        scales = [torch.full(shape[:3], 127, dtype=torch.uint8, device=self.device) for _ in range(2)]
        blocks = [torch.zeros((*shape[:3], shape[3] // SCALE_BLOCK), dtype=torch.float8_e4m3fn, device=self.device) for _ in range(2)] if four else ()
        return KVPool(*codes, *scales, *blocks)

    # The checks below test everything in one expression and leave it to the
    # functions above, which say what is wrong, to raise.

    def _batch(self, pool, n_tokens, cu, kv_len, page_table, max_kv=0):
        device = self.device
        if pool.kv_heads != self.kv_heads or pool.head_dim != self.head_dim:
            raise ValueError(f"pool of {pool.kv_heads} heads of {pool.head_dim}, expected {self.kv_heads} of {self.head_dim}")
        if pool.device != device:
            raise ValueError(f"pool is on {pool.device}, expected {device}")
        i32 = torch.int32
        try:
            n, width = page_table.shape
            ok = (cu.shape == (n + 1,) and kv_len.shape == (n,) and n <= self.max_seqs
                  and cu.dtype is i32 and kv_len.dtype is i32 and page_table.dtype is i32
                  and cu.is_contiguous() and kv_len.is_contiguous() and page_table.is_contiguous()
                  and cu.device == device and kv_len.device == device and page_table.device == device)
        except (AttributeError, ValueError):
            ok = False
        if not ok:
            check_sequences(cu, device, self.max_seqs, kv_len, page_table)
        c = self._batch_c
        c.cu, c.kv_len, c.page_table = cu.data_ptr(), kv_len.data_ptr(), page_table.data_ptr()
        c.n_seqs, c.n_tokens, c.max_pages, c.max_kv = n, n_tokens, width, max_kv
        return self._batch_ref

    def _rows(self, c, t, name, heads, n_tokens=None):
        try:
            n, h, d = t.shape
            token, head, last = t.stride()
            ptr = t.data_ptr()
            ok = (h == heads and d == self.head_dim and (n_tokens is None or n == n_tokens) and t.dtype is torch.bfloat16
                  and t.device == self.device and (n == 0 or last == 1 and not (token | head | ptr >> 1) & 7))
        except (AttributeError, ValueError):
            ok = False
        if not ok:
            check_rows(t, name, heads, self.head_dim, self.device, n_tokens)
        c.ptr, c.token_stride, c.head_stride = ptr, token, head
        return n

    def _allocate(self, stream, make, *args) -> dict:
        """make's tensors, which a call on `stream` writes: memory of that stream, so that nothing still queued on the
        current one uses it; and where the two differ the tensors are marked as used by the current stream too, which
        may read them after waiting for the other, so that freeing them early is safe."""
        if stream is None or stream.cuda_stream == self._current():
            return make(*args)
        current = torch.cuda.current_stream(self.device)
        with torch.cuda.stream(stream):
            out = make(*args)
        for t in out.values():
            t.record_stream(current)
        return out

    def _new_outputs(self, n, want_lse):
        device = self.device
        out = {"out": torch.empty((n, self.q_heads, self.head_dim), dtype=torch.bfloat16, device=device)}
        if want_lse:
            out["lse"] = torch.empty((n, self.q_heads), dtype=torch.float32, device=device)
        return out

    def _outputs(self, n, want_lse, out, stream):
        if out is None:
            return self._allocate(stream, self._new_outputs, n, want_lse)
        _check(out.get("out"), "output out", torch.bfloat16, (n, self.q_heads, self.head_dim), self.device)
        if out["out"].data_ptr() % 32:
            raise ValueError("output out must be 32-byte aligned")
        if out.get("lse") is not None:
            _check(out["lse"], "output lse", torch.float32, (n, self.q_heads), self.device)
        elif want_lse:
            raise ValueError("output lse is required")
        return out

    def _scale(self, scale) -> float:
        if scale is None:
            return self.head_dim ** -0.5
        if not 0.0 < scale < 3e38:
            raise ValueError(f"scale must be positive and finite, not {scale}")
        return scale

    def append(self, pool: KVPool, k, v, cu, kv_len, page_table, stream=None) -> None:
        """spec_attn_append: writes k and v [n_tokens, kv_heads, head_dim], the last
        tokens of their sequences, into the pool (asynchronous)."""
        n = self._rows(self._k_c, k, "k", self.kv_heads)
        self._rows(self._v_c, v, "v", self.kv_heads, n)
        rc = self._lib.spec_attn_append(self._h, pool._ref, self._batch(pool, n, cu, kv_len, page_table), self._k_ref,
                                        self._v_ref, self._stream(stream))
        if rc:
            self._status(rc, "spec_attn_append")

    def append_rotated(self, pool: KVPool, k, v, cu, kv_len, page_table, rope: Rope, q=None, positions=None, want_k: bool = False,
                       out: dict | None = None, stream=None) -> dict:
        """spec_attn_append_rotated: as append, with the keys rotated by their
        positions on the way.  With q [n_tokens, q_heads, head_dim] the queries are
        rotated too, into "q" of the result, and with want_k the rotated keys are
        returned as "k" (for prompt).  positions: int32 [n_tokens], in place of the
        tokens' places in the cache.  out may hold "q" and "k", which may be q and k
        themselves (and no other tensor that overlaps them)."""
        n = self._rows(self._k_c, k, "k", self.kv_heads)
        self._rows(self._v_c, v, "v", self.kv_heads, n)
        batch = self._batch(pool, n, cu, kv_len, page_table)
        if rope.device != self.device:
            raise ValueError(f"rope is on {rope.device}, expected {self.device}")
        if rope.rot_dim > self.head_dim:
            raise ValueError(f"rope turns {rope.rot_dim} elements of {self.head_dim}")
        if positions is not None:
            _check(positions, "positions", torch.int32, (n,), self.device)
        c = self._rope_c                # the handle's own: handles of several threads may share a Rope
        c.table, c.positions = rope.table.data_ptr(), None if positions is None else positions.data_ptr()
        c.max_positions, c.rot_dim, c.interleaved = rope.max_positions, rope.rot_dim, rope.interleaved
        q_ref = q_out = k_out = None
        if q is not None:
            self._rows(self._q_c, q, "q", self.q_heads, n)
            q_ref = self._q_ref
        if out is None:
            out = self._allocate(stream, self._new_rotated, n, q is not None, want_k)
            q_out, k_out = self._q_out_ref if q is not None else None, self._k_out_ref if want_k else None
        else:
            if (q is None) != (out.get("q") is None):
                raise ValueError("q and output q go together")
            if q is not None:
                q_out = self._out_rows(self._q_out_c, self._q_out_ref, out["q"], "output q", self.q_heads, n)
            if out.get("k") is not None:
                k_out = self._out_rows(self._k_out_c, self._k_out_ref, out["k"], "output k", self.kv_heads, n)
            elif want_k:
                raise ValueError("output k is required")
        rc = self._lib.spec_attn_append_rotated(self._h, pool._ref, batch, self._rope_ref, q_ref, self._k_ref, self._v_ref, q_out, k_out,
                                                self._stream(stream))
        if rc:
            self._status(rc, "spec_attn_append_rotated")
        return out

    def _new_rotated(self, n, want_q, want_k):
        out = {}
        if want_q:
            out["q"] = self._new_rows(self._q_out_c, n, self.q_heads)
        if want_k:
            out["k"] = self._new_rows(self._k_out_c, n, self.kv_heads)
        return out

    def _new_rows(self, c, n, heads):
        d = self.head_dim
        t = torch.empty((n, heads, d), dtype=torch.bfloat16, device=self.device)
        c.ptr, c.token_stride, c.head_stride = t.data_ptr(), heads * d, d
        return t

    def _out_rows(self, c, ref, t, name, heads, n):
        self._rows(c, t, name, heads, n)
        # the rows of the closer stride lie apart, and the other stride steps over all of them
        (near, few), (far, many) = sorted(((c.token_stride if n > 1 else 0, n), (c.head_stride if heads > 1 else 0, heads)))
        if few > 1 and near < self.head_dim or many > 1 and far < (few - 1) * near + self.head_dim:
            raise ValueError(f"{name}: strides {tuple(t.stride())} let its rows overlap")
        return ref

    def read(self, pool: KVPool, cu, kv_len, page_table, n_tokens: int, out: dict | None = None, stream=None) -> dict:
        """spec_attn_read: positions kv_len[b] - n_b .. kv_len[b] - 1 of every sequence
        as bf16 tensors "k" and "v" [n_tokens, kv_heads, head_dim]; n_tokens is at
        least cu[-1] (a host number, so that nothing waits for the device)."""
        batch = self._batch(pool, n_tokens, cu, kv_len, page_table)
        shape = (n_tokens, self.kv_heads, self.head_dim)
        if out is None:
            out = self._allocate(stream, lambda: {name: torch.empty(shape, dtype=torch.bfloat16, device=self.device) for name in ("k", "v")})
        else:
            for name in ("k", "v"):
                _check(out.get(name), f"output {name}", torch.bfloat16, shape, self.device)
                if out[name].data_ptr() % 32:
                    raise ValueError(f"output {name} must be 32-byte aligned")
        rc = self._lib.spec_attn_read(self._h, pool._ref, batch, out["k"].data_ptr(), out["v"].data_ptr(), self._stream(stream))
        if rc:
            self._status(rc, "spec_attn_read")
        return out

    def attend(self, pool: KVPool, q, cu, kv_len, page_table, causal: bool = True, scale: float | None = None,
               want_lse: bool = False, out: dict | None = None, stream=None, max_kv: int = 0) -> dict:
        """spec_attn_chunk: attention of the new tokens q [n_tokens, q_heads, head_dim]
        over the pool, which holds their keys and values already.  Returns "out"
        (like q) and, if wanted, "lse" [n_tokens, q_heads].  scale defaults to
        head_dim ** -0.5; causal=False lets every new token see all kv_len entries.
        max_kv: a host-side bound of kv_len (0: unknown), which chooses the faster kernel
        for chunks where page_table is wider than the batch needs."""
        n = self._rows(self._q_c, q, "q", self.q_heads)
        if not 0 <= max_kv < 1 << 31:
            raise ValueError(f"max_kv must be 0 or a length, not {max_kv}")
        batch = self._batch(pool, n, cu, kv_len, page_table, max_kv)
        scale = self._scale(scale)
        out = self._outputs(n, want_lse, out, stream)
        lse = out.get("lse")
        rc = self._lib.spec_attn_chunk(self._h, pool._ref, batch, self._q_ref, int(causal), scale, out["out"].data_ptr(),
                                       None if lse is None else lse.data_ptr(), self._stream(stream))
        if rc:
            self._status(rc, "spec_attn_chunk")
        return out

    def prompt(self, q, k, v, cu, scale: float | None = None, want_lse: bool = False, out: dict | None = None,
               stream=None) -> dict:
        """spec_attn_prompt: causal attention over packed prompts, q [n_tokens, q_heads,
        head_dim], k and v [n_tokens, kv_heads, head_dim].  Returns as attend."""
        n = self._rows(self._q_c, q, "q", self.q_heads)
        self._rows(self._k_c, k, "k", self.kv_heads, n)
        self._rows(self._v_c, v, "v", self.kv_heads, n)
        try:
            n_seqs = cu.shape[0] - 1
            ok = (cu.dtype is torch.int32 and cu.dim() == 1 and 0 <= n_seqs <= self.max_seqs and cu.is_contiguous()
                  and cu.device == self.device)
        except (AttributeError, IndexError):
            ok = False
        if not ok:
            n_seqs = check_sequences(cu, self.device, self.max_seqs, paged=False)
        scale = self._scale(scale)
        out = self._outputs(n, want_lse, out, stream)
        lse = out.get("lse")
        rc = self._lib.spec_attn_prompt(self._h, n_seqs, n, cu.data_ptr(), self._q_ref, self._k_ref, self._v_ref, scale,
                                        out["out"].data_ptr(), None if lse is None else lse.data_ptr(), self._stream(stream))
        if rc:
            self._status(rc, "spec_attn_prompt")
        return out

    def get_error(self) -> int:
        """Synchronise; return the status the kernels flagged since the last call
        (SV_OK, SV_ERR_DATA for invalid metadata, SV_ERR_TIMEOUT) and clear it."""
        return self._lib.spec_attn_get_error(self._h)


__all__ = ["KVPool", "Rope", "SpecAttention", "SV_E2M1", "SV_E4M3", "check_rows", "check_sequences"]
