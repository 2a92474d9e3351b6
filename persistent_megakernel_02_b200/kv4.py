"""The 4-bit KV cache (``mk_kv4_*``): a paged pool of quantised K/V rows, written,
read back and attended over by the library's kernels.

The memory is the caller's: a uint8 pool, an int32 block table with each sequence's
pages of ``PAGE`` positions, and int32 lengths on the device, so a captured graph can
be replayed while sequences grow.  Calls are asynchronous on ``stream`` (default: the
current torch stream of the pool's device), check every tensor's type, shape, layout and device
first and raise :class:`MkError` before anything is launched.  What only the device
can see (lengths or page ids out of bounds) is recorded in the cache's status word,
which :meth:`Kv4Cache.check` reads.

The package's other stages (``matvec_engine``, ``greedy_head_noalloc``, a handle's steps) run on
the default stream unless they are given one: inside ``torch.cuda.stream(s)`` give them ``s``.
``Megakernel.park`` and ``resume`` without a stream keep the order of both.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import MkError, MkKv4Batch, MkKv4CacheStruct, MkKv4Rows, _check, lib

# the raw forms of torch.cuda.current_device and current_stream, where this torch has them
# (the public ones cost about 2 us of a call of 5)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)

PAGE = 64
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _bad(what, why):
    raise MkError(1, f"{what}: {why}")


def page_bytes(head_dim: int) -> int:
    """Bytes of one page (PAGE positions, K and V) of one kv head."""
    n = lib().mk_kv4_page_bytes(head_dim)
    if n == 0:
        raise MkError(2, "mk_kv4_page_bytes: head_dim must be 64 or 128")
    return n


class Kv4Batch:
    """The sequences of a call: row ``cu[i] .. cu[i + 1] - 1`` of its tensors are the last
    positions of sequence ``i``, which is ``kv_lens[i]`` long with them (see
    :meth:`Kv4Cache.batch`)."""

    def __init__(self, cache, block_table, cu, kv_lens, n_rows, max_new, max_len):
        for name, t, dims in (("block_table", block_table, 2), ("cu", cu, 1), ("kv_lens", kv_lens, 1)):
            if t is None or t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous():
                _bad("Kv4Batch", f"{name} must be a contiguous int32 tensor with {dims} dimension(s)")
            if t.device != cache.device:
                _bad("Kv4Batch", f"{name} must be on {cache.device}")
        n = int(kv_lens.shape[0])
        if n < 1 or int(cu.shape[0]) != n + 1:
            _bad("Kv4Batch", "cu must have one element more than kv_lens, and kv_lens at least one")
        if int(block_table.shape[0]) < n or int(block_table.shape[1]) < 1:
            _bad("Kv4Batch", "block_table must have a row for every sequence and at least one page")
        max_pages = int(block_table.shape[1])
        if n_rows < 0 or max_new < 0 or not 0 <= max_len <= PAGE * max_pages or max(n_rows, max_len) >= 2**31:
            _bad("Kv4Batch", f"bounds: 0 <= n_rows, 0 <= max_new, 0 <= max_len <= {PAGE} * {max_pages}")
        self.n_rows, self.device = int(n_rows), cache.device
        self._keep = (block_table, cu, kv_lens)
        self._workspace_bytes = {}  # by cache shape, heads and type: caches of other shapes may share a batch
        self._struct = MkKv4Batch(block_table.data_ptr(), cu.data_ptr(), kv_lens.data_ptr(), n, max_pages,
                                  int(n_rows), min(int(max_new), int(n_rows)), int(max_len))


class Kv4Cache:
    """A 4-bit KV cache over a caller-owned pool: uint8 CUDA tensor
    ``[n_layers, n_pages, n_kv_heads, page_bytes(head_dim)]``, contiguous.

    ``block_table`` (int32 ``[n_seqs, max_pages]``) is the default of :meth:`batch`.
    The values it stands for are within half a step of the rows written: a 15-step grid
    over the range of every 32 neighbouring values.
    """

    def __init__(self, pool, block_table=None, head_dim: int = 128):
        if pool.dtype != torch.uint8 or pool.dim() != 4 or not pool.is_contiguous() or not pool.is_cuda:
            _bad("Kv4Cache", "pool must be a contiguous uint8 CUDA tensor [n_layers, n_pages, n_kv_heads, page_bytes]")
        if int(pool.shape[3]) != page_bytes(head_dim) or pool.numel() == 0:
            _bad("Kv4Cache", f"pages of {head_dim}-value heads are {page_bytes(head_dim)} bytes, and none may be missing")
        self.pool, self.block_table, self.head_dim = pool, block_table, int(head_dim)
        self.device = pool.device
        self.n_layers, self.n_pages, self.n_kv_heads = (int(x) for x in pool.shape[:3])
        self._status = torch.zeros(1, dtype=torch.int32, device=pool.device)
        with torch.cuda.device(pool.device):
            if not torch.cuda.is_current_stream_capturing():  # calls on any stream come behind the zero
                torch.cuda.current_stream().synchronize()
        self._struct = MkKv4CacheStruct(pool.data_ptr(), self._status.data_ptr(), self.n_layers, self.n_pages,
                                        self.n_kv_heads, self.head_dim)
        self._index = pool.device.index
        self._shape = (self.n_kv_heads, self.head_dim)
        self._scale = 1.0 / math.sqrt(head_dim)
        so = lib()
        self._append, self._read, self._attention = so.mk_kv4_append, so.mk_kv4_read, so.mk_kv4_attention

    @classmethod
    def empty(cls, n_layers, n_pages, n_kv_heads, head_dim, block_table=None, device="cuda"):
        """A cache with a pool of its own."""
        pool = torch.empty((n_layers, n_pages, n_kv_heads, page_bytes(head_dim)), dtype=torch.uint8, device=device)
        return cls(pool, block_table, head_dim)

    def batch(self, cu, kv_lens, n_rows, max_new, max_len, block_table=None) -> Kv4Batch:
        """Describe the sequences of the calls to come.  ``cu`` (int32 ``[n + 1]``) and
        ``kv_lens`` (int32 ``[n]``) may change on the device between calls, within the
        bounds given here: ``n_rows`` rows of the tensors, spans of at most ``max_new``
        rows, lengths of at most ``max_len``."""
        return Kv4Batch(self, self.block_table if block_table is None else block_table, cu, kv_lens, n_rows,
                        max_new, max_len)

    def _launch(self, what, stream, batch=None):
        if _current_device() != self._index:
            _bad(what, f"the cache is not on the current CUDA device ({torch.cuda.current_device()})")
        if batch is not None and batch.device != self.device:
            _bad(what, f"the batch must be on {self.device}")
        if stream is None:
            return _current_stream(self._index)
        return getattr(stream, "cuda_stream", stream)

    def _torch_stream(self, raw):
        # (ExternalStream takes the default stream's 0 for none and makes a new stream)
        return torch.cuda.ExternalStream(raw, self.device) if raw else torch.cuda.default_stream(self.device)

    def _rows(self, what, name, t, heads, batch, dtype):
        if (t.shape == (batch.n_rows, heads, self.head_dim) and t.dtype is dtype and dtype in _DTYPES
                and t.get_device() == self._index):
            rs, hs, es = t.stride()
            if es == 1:
                return MkKv4Rows(t.data_ptr(), rs, hs)
        if t.shape != (batch.n_rows, heads, self.head_dim):
            _bad(what, f"{name} must have shape ({batch.n_rows}, {heads}, {self.head_dim}), got {tuple(t.shape)}")
        if t.dtype is not dtype or dtype not in _DTYPES:
            _bad(what, f"{name} must be bfloat16, float16 or float32, the same type for every tensor; got {t.dtype}")
        if t.get_device() != self._index:
            _bad(what, f"{name} must be on {self.device}")
        _bad(what, f"the last dimension of {name} must be contiguous")

    def _kv(self, fn, what, layer, k, v, batch, stream):
        dtype = k.dtype
        kr = self._rows(what, "k", k, self.n_kv_heads, batch, dtype)
        vr = self._rows(what, "v", v, self.n_kv_heads, batch, dtype)
        st = fn(self._struct, layer, batch._struct, kr, vr, _DTYPES[dtype], self._launch(what, stream, batch))
        if st:
            raise MkError(st, what)

    def append(self, layer, k, v, batch, stream=None):
        """Quantise rows ``k`` and ``v`` ([n_rows, n_kv_heads, head_dim], any row and head
        strides) into their positions."""
        self._kv(self._append, "mk_kv4_append", layer, k, v, batch, stream)

    def read(self, layer, k, v, batch, stream=None):
        """Write the values the cache holds for the batch's rows into ``k`` and ``v``, which
        must not share memory."""
        self._kv(self._read, "mk_kv4_read", layer, k, v, batch, stream)

    def attend(self, layer, q, out, batch, scale=None, workspace=None, stream=None):
        """Causal attention of query rows ``q`` [n_rows, n_heads, head_dim] over the cache,
        each row seeing the positions up to its own; ``out`` like ``q``, or ``q`` itself.  Many bf16 rows lose
        accuracy over keys with channels beyond 100, fp16 ones do not (figures in mk.h).  ``scale`` defaults to
        1 / sqrt(head_dim).  ``workspace``: a uint8 CUDA tensor of ``workspace_bytes`` for calls
        that must not allocate; otherwise one is allocated on the launch stream."""
        what = "mk_kv4_attention"
        dtype = q.dtype
        heads = q.shape[1] if q.dim() == 3 else 0
        qr = self._rows(what, "q", q, heads, batch, dtype)
        orow = self._rows(what, "out", out, heads, batch, dtype)
        raw = self._launch(what, stream, batch)
        need = batch._workspace_bytes.get((self._shape, heads, dtype))
        if need is None:
            need = self.workspace_bytes(batch, heads, dtype)
        ptr = None
        if need:
            if workspace is None:
                if stream is None:
                    workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
                else:
                    with torch.cuda.stream(self._torch_stream(raw)):
                        workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            elif workspace.dtype != torch.uint8 or workspace.get_device() != self._index or not workspace.is_contiguous():
                _bad(what, f"workspace must be a contiguous uint8 tensor on {self.device}")
            need, ptr = workspace.numel(), workspace.data_ptr()
        st = self._attention(self._struct, layer, batch._struct, qr, orow, heads, _DTYPES[dtype],
                             self._scale if scale is None else scale, ptr, need, raw)
        if st:
            raise MkError(st, what)

    def workspace_bytes(self, batch, n_heads, dtype) -> int:
        """Workspace of :meth:`attend` for this batch (0 where it needs none)."""
        got = batch._workspace_bytes.get((self._shape, n_heads, dtype))
        if got is None:
            n = ctypes.c_int64()
            _check(lib().mk_kv4_attention_workspace(self._struct, batch._struct, n_heads, _DTYPES.get(dtype, -1),
                                                    ctypes.byref(n)), "mk_kv4_attention_workspace")
            got = batch._workspace_bytes[(self._shape, n_heads, dtype)] = n.value
        return got

    def check(self, stream=None):
        """Wait for ``stream`` and raise MkError if a call met numbers outside its batch's
        bounds or a page id outside the pool since the last check.  One that another stream's call
        meets meanwhile is reported by this check or the next one."""
        raw = self._launch("Kv4Cache.check", stream)
        with torch.cuda.stream(self._torch_stream(raw)):
            taken = torch.empty(1, dtype=torch.int32, device=self.device)
            _check(lib().mk_kv4_take_status(self._struct, taken.data_ptr(), raw), "mk_kv4_take_status")
            bits = int(taken.item())
        if bits & 4:
            raise MkError(5, "Kv4Cache: a bounded wait ran out")
        if bits:
            why = [w for b, w in ((1, "batch numbers out of bounds"), (2, "a page id out of range")) if bits & b]
            raise MkError(6, "Kv4Cache: " + " and ".join(why))
