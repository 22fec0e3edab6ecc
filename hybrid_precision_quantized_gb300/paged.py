"""A pool of quantised pages for many sequences (include/hyq.h, "Paged cache").

PyTorch only allocates memory and provides the stream; every step runs in
libhyq's kernels.  One step of a model with ``n_layers`` layers:

    cache.reserve(seqs, n_new)                        # lengths, pages, copies on write
    for layer in range(n_layers):
        cache.append(layer, k, v, seqs=seqs, ...)     # this step's rows
        cache.attention(layer, q, out, seqs=seqs)     # or select + attention_blocks

``fork`` lets sequences share what they have in common, ``truncate`` shortens
or frees them, ``compact`` moves the pages in use to the front of the pool.
Nothing synchronises; errors that only the GPU can see collect in
``cache.err()`` (hyq_read_device_error).
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib as L
from ._lib import HyqConfig, HyqPages

_DTYPES = {"pool": torch.uint8, "bounds": torch.uint8, "table": torch.int32, "lens": torch.int32,
           "refs": torch.int32, "err": torch.int32}


class PagedCache:
    """The buffers of a pool and the calls on it.

    cfg        : heads and code widths (make_config; batch and capacity are not used)
    n_pages    : pages of 64 positions, each for every layer
    n_seqs     : rows of the table (a call takes 1024 of them at most; more are given in several calls)
    max_blocks : pages a sequence may have
    buffers    : tensors to use instead of new ones, by name (pool, bounds, table, lens, refs, err), contiguous, of
                 the C layout's types and sizes; those not given are allocated (and, without any, reset)

    The workspaces belong to the object and grow with the largest call: calls of one kind that may overlap on the
    GPU (other streams, graphs replayed at once) need a PagedCache of their own over the same buffers.  Call each kind once at its
    largest size before capturing it into a CUDA graph, and keep to that size while the graph lives.
    """

    def __init__(self, cfg: HyqConfig, n_pages: int, n_seqs: int, max_blocks: int, n_layers: int = 1, device="cuda",
                 buffers: dict | None = None):
        self.cfg = cfg
        self.n_pages, self.n_seqs, self.max_blocks, self.n_layers = n_pages, n_seqs, max_blocks, n_layers
        self.c = HyqPages(n_layers=n_layers, n_pages=n_pages, n_seqs=n_seqs, max_blocks=max_blocks)
        sizes = dict(zip(L.PAGES_FIELDS, L.hyq_pages_sizes(cfg, self.c)))
        block = L.qblock_bytes(cfg.bits_k, cfg.bits_v)
        shapes = {"pool": (n_layers, n_pages, cfg.num_kv_heads, block),
                  "bounds": (n_layers, n_pages, cfg.num_kv_heads, L.BOUND_BYTES), "table": (n_seqs, max_blocks),
                  "lens": (n_seqs,), "refs": (n_pages,), "err": (1,)}
        given = buffers or {}
        if set(given) - set(shapes):
            raise ValueError(f"unknown buffers: {sorted(set(given) - set(shapes))}")
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.buf = {}
        for name, shape in shapes.items():
            t = given.get(name)
            if t is None:
                n = sizes[name] // _DTYPES[name].itemsize
                make = torch.empty if name in ("pool", "bounds") else torch.zeros
                t = make(n, dtype=_DTYPES[name], device=dev)
                t = t[: int(torch.Size(shape).numel())].view(shape)
            elif t.dtype != _DTYPES[name] or tuple(t.shape) != shape or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"{name}: expected a contiguous {_DTYPES[name]} tensor of shape {shape} on {dev}")
            self.buf[name] = t
            setattr(self.c, name, t.data_ptr())
        self._ws, self._kept = {}, []
        self._streams = {}      # that calls were queued on, by handle
        self._lib, self._index = L.load(), dev.index
        self._cfg, self._pages = ctypes.byref(cfg), ctypes.byref(self.c)

    # typed views -----------------------------------------------------------
    def pool(self) -> torch.Tensor:
        """uint8 [n_layers, n_pages, HKV, block bytes]"""
        return self.buf["pool"]

    def bounds(self) -> torch.Tensor:
        """uint8 [n_layers, n_pages, HKV, 272]"""
        return self.buf["bounds"]

    def table(self) -> torch.Tensor:
        return self.buf["table"]

    def lens(self) -> torch.Tensor:
        return self.buf["lens"]

    def refs(self) -> torch.Tensor:
        return self.buf["refs"]

    def err(self) -> torch.Tensor:
        return self.buf["err"]

    # argument checks ---------------------------------------------------------
    # A decode step makes these calls for every layer, a few microseconds apart:
    # the common forms (contiguous tensors, the cache's device being the
    # current one) are tested first and cost well under a microsecond each.
    def _run(self, name, args, stream, *tensors):
        """Call the C entry point on the given stream, or the current one of the cache's device.  A given stream is noted on
        the call's tensors, and every stream once on the cache's own: memory that is dropped is not reused before the
        call has read it."""
        fn = getattr(self._lib, name)
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(self._index)
        else:
            raw = stream.cuda_stream
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        if raw not in self._streams:
            self._streams[raw] = stream = stream if stream is not None else torch.cuda.current_stream(self.device)
            for t in (*self.buf.values(), *self._kept):
                t.record_stream(stream)
        if torch.cuda.current_device() == self._index:
            st = fn(self._cfg, self._pages, *args, raw)
        else:
            with torch.cuda.device(self.device):
                st = fn(self._cfg, self._pages, *args, raw)
        if st:
            raise L.HyqError(name, st)

    def _ints(self, t, name, n=None):
        """Entries of an int32 index tensor (None: n)."""
        if t is None:
            return n
        if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.device != self.device:
            raise ValueError(f"{name}: expected a contiguous int32 vector on {self.device}")
        m = t.shape[0]
        if n is not None and m != n:
            raise ValueError(f"{name}: expected {n} entries, got {m}")
        return m

    def _heads(self, t, name, heads):
        """Elements between consecutive tokens of a bf16 [..., heads, 128] tensor whose tokens are evenly spaced and whose
        heads are dense."""
        shape = t.shape
        if t.dtype != torch.bfloat16 or shape[-1] != 128 or shape[-2] != heads or t.device != self.device:
            raise ValueError(f"{name}: expected a bf16 [..., {heads}, 128] tensor on {self.device}")
        if t.is_contiguous():
            return heads * 128
        strides = t.stride()
        if strides[-1] != 1 or (heads > 1 and strides[-2] != 128):
            raise ValueError(f"{name}: the heads of a token must be dense")
        ld = None
        for i in range(t.dim() - 3, -1, -1):
            if shape[i] == 1:
                continue
            if ld is None:
                ld, step = strides[i], strides[i] * shape[i]
            elif strides[i] != step:
                raise ValueError(f"{name}: the tokens must be evenly spaced")
            else:
                step *= shape[i]
        return heads * 128 if ld is None else ld

    def _dense(self, t, name, dtype, shape):
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != self.device:
            raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {self.device}")
        return t.data_ptr()

    def workspace(self, op: int, batch: int, n_q: int = 1, stream=None) -> torch.Tensor:
        """The zero-filled workspace of an operation for calls of batch * n_q tokens, kept and grown as needed.  One that
        has been outgrown stays allocated: work queued earlier, or a captured graph, may still use it.  A larger one takes
        at least twice the tokens of the last, so that there are few of them however the calls grow."""
        w = self._ws.get(op)
        tokens = batch * n_q
        if w is None or w[0] < tokens:
            n = L.hyq_pages_workspace_size(self.cfg, self.c, op, max(batch, 1), n_q)
            if n == 0:
                raise ValueError(f"no call of this kind takes {batch} sequences with {n_q} tokens")
            if w is not None:       # the size depends on the product alone
                b = min(max(tokens, 2 * w[0]), L.PAGED_MAX_BATCH)
                q = min(-(-max(tokens, 2 * w[0]) // b), L.PAGED_MAX_Q)
                n, tokens = L.hyq_pages_workspace_size(self.cfg, self.c, op, b, q), b * q
            with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(self.device)):
                t = torch.zeros(n, dtype=torch.uint8, device=self.device)
            self._kept.append(t)
            for s in self._streams.values():
                t.record_stream(s)
            w = self._ws[op] = (tokens, t)
        return w[1]

    # tables ------------------------------------------------------------------
    def reset(self, stream=None):
        """Empty pool."""
        self._run("hyq_pages_reset", (), stream)

    def reserve(self, seqs=None, n_new=None, stream=None):
        """Room for n_new[i] (default 1) more positions of sequence seqs[i] (default: sequence i; all of them without
        n_new, in a cache of up to 1024)."""
        n = self._ints(n_new, "n_new", self._ints(seqs, "seqs"))
        ws = self.workspace(L.OP_PAGES_RESERVE, 1, stream=stream)
        self._run("hyq_pages_reserve", (L.ptr(seqs), self.n_seqs if n is None else n, L.ptr(n_new), ws.data_ptr(),
                                        ws.nbytes), stream, seqs, n_new)

    def fork(self, src, dst, stream=None):
        """Let the empty sequences dst begin as copies of src, sharing their pages."""
        n = self._ints(dst, "dst", self._ints(src, "src"))
        self._run("hyq_pages_fork", (src.data_ptr(), dst.data_ptr(), n), stream, src, dst)

    def truncate(self, seqs=None, new_lens=None, stream=None):
        """Shorten the sequences (default: sequence i; all of them without new_lens, however many) to new_lens (default 0:
        free them)."""
        n = self._ints(new_lens, "new_lens", self._ints(seqs, "seqs"))
        self._run("hyq_pages_truncate", (L.ptr(seqs), L.ptr(new_lens), self.n_seqs if n is None else n), stream, seqs,
                  new_lens)

    def compact(self, table_out=None, refs_out=None, stream=None):
        """Move the pages in use to the front of the pool; the new table and refs go to the given tensors, or in place."""
        table = refs = None
        if table_out is not None:
            table = self._dense(table_out, "table_out", torch.int32, (self.n_seqs, self.max_blocks))
        if refs_out is not None:
            refs = self._dense(refs_out, "refs_out", torch.int32, (self.n_pages,))
        ws = self.workspace(L.OP_PAGES_COMPACT, 1, stream=stream)
        self._run("hyq_pages_compact", (table, refs, ws.data_ptr(), ws.nbytes), stream, table_out, refs_out)

    # one layer -----------------------------------------------------------------
    def append(self, layer: int, k, v, seqs=None, cu_rows=None, k_hat=None, v_hat=None, stream=None):
        """Quantise rows k, v [rows, HKV, 128] into the last positions of their sequences: one row per sequence, or rows
        cu_rows[i] .. cu_rows[i + 1] for sequence seqs[i].  k_hat, v_hat: bf16 tensors for the rows as they are held."""
        hkv = self.cfg.num_kv_heads
        if k.dim() != 3 or v.shape != k.shape:
            raise ValueError("k and v: expected [rows, HKV, 128] each")
        rows = k.shape[0]
        ld = self._heads(k, "k", hkv)
        if self._heads(v, "v", hkv) != ld:
            raise ValueError("k and v must share the spacing of their rows")
        if cu_rows is None:
            n = self._ints(seqs, "seqs", rows)
        else:
            n = self._ints(cu_rows, "cu_rows") - 1
            self._ints(seqs, "seqs", n)
        kh = vh = None
        if k_hat is not None:
            kh = self._dense(k_hat, "k_hat", torch.bfloat16, k.shape)
        if v_hat is not None:
            vh = self._dense(v_hat, "v_hat", torch.bfloat16, k.shape)
        self._run("hyq_paged_append", (layer, L.ptr(seqs), n, L.ptr(cu_rows), rows, k.data_ptr(), v.data_ptr(), ld, kh,
                                       vh), stream, seqs, cu_rows, k, v, k_hat, v_hat)

    def _query(self, q, seqs):
        """(batch, n_q, elements between tokens) of q."""
        if q.dim() != 4:
            raise ValueError("q: expected [sequences, tokens, HQ, 128]")
        b, n_q = q.shape[0], q.shape[1]
        self._ints(seqs, "seqs", b)
        return b, n_q, self._heads(q, "q", self.cfg.num_q_heads)

    def attention(self, layer: int, q, out, seqs=None, stream=None):
        """Causal attention of the last n_q tokens of every sequence: q, out bf16 [sequences, n_q, HQ, 128]."""
        b, n_q, ldq = self._query(q, seqs)
        o = self._dense(out, "out", torch.bfloat16, q.shape)
        ws = self.workspace(L.OP_PAGED_ATTENTION, b, n_q, stream)
        self._run("hyq_paged_attention", (layer, L.ptr(seqs), b, n_q, q.data_ptr(), ldq, o, ws.data_ptr(), ws.nbytes),
                  stream, seqs, q, out)

    def select(self, layer: int, q, sel, seqs=None, n_first: int = 1, n_last: int = 1, stream=None):
        """The blocks worth reading for every token and KV head: sel int32 [sequences, n_q, HKV, k]."""
        b, n_q, ldq = self._query(q, seqs)
        k = sel.shape[-1]
        p = self._dense(sel, "sel", torch.int32, (b, n_q, self.cfg.num_kv_heads, k))
        ws = self.workspace(L.OP_PAGED_SELECT, b, n_q, stream)
        self._run("hyq_paged_select", (layer, L.ptr(seqs), b, n_q, q.data_ptr(), ldq, k, n_first, n_last, p,
                                       ws.data_ptr(), ws.nbytes), stream, seqs, q, sel)

    def attention_blocks(self, layer: int, q, sel, out, seqs=None, stream=None):
        """attention over the blocks that sel lists for each token and KV head."""
        b, n_q, ldq = self._query(q, seqs)
        o = self._dense(out, "out", torch.bfloat16, q.shape)
        k = sel.shape[-1]
        p = self._dense(sel, "sel", torch.int32, (b, n_q, self.cfg.num_kv_heads, k))
        ws = self.workspace(L.OP_PAGED_ATTENTION, b, n_q, stream)
        self._run("hyq_paged_attention_blocks", (layer, L.ptr(seqs), b, n_q, q.data_ptr(), ldq, p, k, o, ws.data_ptr(),
                                                 ws.nbytes), stream, seqs, q, sel, out)
