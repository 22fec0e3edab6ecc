"""The paged cache without a GPU: sizes, argument checks of the C entry points
(before any launch) and of PagedCache."""
import ctypes
import os

import pytest
import torch

import hybrid_precision_quantized_gb300 as hyq
from hybrid_precision_quantized_gb300 import _lib as L


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return hyq.load()


def cfg(**kw):
    base = dict(batch=1, num_q_heads=8, num_kv_heads=2, capacity=64)
    base.update(kw)
    return hyq.make_config(**base)


def pages(**kw):
    base = dict(n_layers=2, n_pages=10, n_seqs=3, max_blocks=5)
    base.update(kw)
    return L.HyqPages(**base)


def test_sizes(lib):
    s = hyq.hyq_pages_sizes(cfg(), pages())
    assert s == [2 * 10 * 2 * 10240, -(-2 * 10 * 2 * 272 // 256) * 256, 256, 256, 256, 256]
    assert hyq.hyq_pages_sizes(cfg(bits_k=8, bits_v=8), pages())[0] == 2 * 10 * 2 * 18432
    big = pages(n_pages=1 << 20, n_layers=64)
    assert hyq.hyq_pages_sizes(cfg(), big)[0] == 64 * (1 << 20) * 2 * 10240
    for bad in (dict(n_layers=0), dict(n_pages=0), dict(n_pages=(1 << 20) + 1), dict(n_seqs=0), dict(max_blocks=0),
                dict(max_blocks=(1 << 22) + 1), dict(n_seqs=-1)):
        with pytest.raises(hyq.HyqError):
            hyq.hyq_pages_sizes(cfg(), pages(**bad))
    with pytest.raises(hyq.HyqError):
        hyq.hyq_pages_sizes(cfg(head_dim=64), pages())


def test_workspace_sizes(lib):
    c, p = cfg(), pages()
    for op in (L.OP_PAGED_ATTENTION, L.OP_PAGED_SELECT):
        sizes = [hyq.hyq_pages_workspace_size(c, p, op, b, n) for b, n in ((1, 1), (100, 1), (100, 4), (1024, 64))]
        assert 0 < sizes[0] <= sizes[1] < sizes[2] < sizes[3]
        for b, n in ((0, 1), (1025, 1), (1, 0), (1, 65)):
            assert hyq.hyq_pages_workspace_size(c, p, op, b, n) == 0
    for op in (L.OP_PAGES_RESERVE, L.OP_PAGES_COMPACT):
        assert hyq.hyq_pages_workspace_size(c, p, op, 1) > 0
    assert hyq.hyq_pages_workspace_size(c, p, 99, 1) == 0
    assert hyq.hyq_pages_workspace_size(c, p, L.OP_DECODE, 1) == 0


# Fake device addresses are only ever passed where no GPU exists.
@pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation runs only without a GPU")
def test_entry_points_refuse_before_launch(lib):
    c, none = ctypes.byref(cfg()), None
    p = pages(**{n: 4096 * (i + 1) for i, n in enumerate(L.PAGES_FIELDS)})
    g = ctypes.byref(p)
    W = 1 << 40
    INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
    for name in L.PAGES_FIELDS:      # every buffer is needed, 256-byte aligned
        for bad in (None, 4096 + 128):
            q = pages(**{n: 4096 * (i + 1) for i, n in enumerate(L.PAGES_FIELDS)})
            setattr(q, name, bad)
            assert lib.hyq_pages_reset(c, ctypes.byref(q), none) == INVALID
            assert lib.hyq_paged_attention(c, ctypes.byref(q), 0, none, 1, 1, 256, 1024, 256, 256, W, none) == INVALID
    assert lib.hyq_pages_reset(none, g, none) == INVALID and lib.hyq_pages_reset(c, none, none) == INVALID
    # attention: layer, batch, table rows, n_q, spacing, alignment, workspace
    att = lib.hyq_paged_attention
    assert att(c, g, 2, none, 1, 1, 256, 1024, 256, 256, W, none) == INVALID
    assert att(c, g, -1, none, 1, 1, 256, 1024, 256, 256, W, none) == INVALID
    assert att(c, g, 0, none, -1, 1, 256, 1024, 256, 256, W, none) == INVALID
    assert att(c, g, 0, none, 4, 1, 256, 1024, 256, 256, W, none) == INVALID         # 3 table rows
    assert att(c, g, 0, 256, 1025, 1, 256, 1024, 256, 256, W, none) == UNSUPPORTED
    assert att(c, g, 0, 258, 1, 1, 256, 1024, 256, 256, W, none) == INVALID
    assert att(c, g, 0, none, 0, 1, none, 0, none, none, 0, none) == 0               # nothing to do
    assert att(c, g, 0, none, 1, 0, 256, 1024, 256, 256, W, none) == INVALID
    assert att(c, g, 0, none, 1, 65, 256, 1024, 256, 256, W, none) == UNSUPPORTED
    assert att(c, g, 0, none, 1, 1, 256, 1016, 256, 256, W, none) == INVALID
    assert att(c, g, 0, none, 1, 1, 256, 1028, 256, 256, W, none) == INVALID
    assert att(c, g, 0, none, 1, 1, 264, 1024, 256, 256, W, none) == INVALID
    assert att(c, g, 0, none, 1, 1, none, 1024, 256, 256, W, none) == INVALID
    assert att(c, g, 0, none, 1, 1, 256, 1024, none, 256, W, none) == INVALID
    assert att(c, g, 0, none, 1, 1, 256, 1024, 256, none, W, none) == WORKSPACE
    assert att(c, g, 0, none, 1, 1, 256, 1024, 256, 128, W, none) == WORKSPACE
    assert att(c, g, 0, none, 1, 1, 256, 1024, 256, 256, 1000, none) == WORKSPACE
    blk = lib.hyq_paged_attention_blocks
    assert blk(c, g, 0, none, 1, 1, 256, 1024, none, 3, 256, 256, W, none) == INVALID
    assert blk(c, g, 0, none, 1, 1, 256, 1024, 256, 0, 256, 256, W, none) == INVALID
    assert blk(c, g, 0, none, 1, 1, 256, 1024, 256, 3, 256, 256, 10, none) == WORKSPACE
    sel = lib.hyq_paged_select
    for k, a, b in ((0, 0, 0), (2, 2, 1), (2, -1, 0), (2, 0, -1), (2, 2 ** 31 - 1, 2 ** 31 - 1)):
        assert sel(c, g, 0, none, 1, 1, 256, 1024, k, a, b, 256, 256, W, none) == INVALID
    assert sel(c, g, 0, none, 1, 1, 256, 1024, 2, 1, 1, none, 256, W, none) == INVALID
    assert sel(c, g, 0, none, 1, 1, 256, 1024, 2, 1, 1, 256, 256, 10, none) == WORKSPACE
    app = lib.hyq_paged_append
    assert app(c, g, 0, none, 2, none, 3, 256, 256, 256, none, none, none) == INVALID   # one row each: 2 rows
    assert app(c, g, 0, none, 2, 256, -1, 256, 256, 256, none, none, none) == INVALID
    assert app(c, g, 0, none, 2, 256, 0, none, none, 0, none, none, none) == 0
    assert app(c, g, 0, none, 2, 256, 5, none, 256, 256, none, none, none) == INVALID
    assert app(c, g, 0, none, 2, 256, 5, 256, 256, 248, none, none, none) == INVALID
    assert app(c, g, 0, none, 2, 256, 5, 256, 256, 260, none, none, none) == INVALID
    assert app(c, g, 0, none, 2, 256, 5, 256, 256, 256, 256, none, none) == INVALID     # both hats or none
    assert app(c, g, 0, none, 4, none, 4, 256, 256, 256, none, none, none) == INVALID
    assert lib.hyq_pages_reserve(c, g, none, 4, none, 256, W, none) == INVALID
    assert lib.hyq_pages_reserve(c, g, none, 3, none, none, W, none) == WORKSPACE
    assert lib.hyq_pages_reserve(c, g, none, 0, none, none, 0, none) == 0
    assert lib.hyq_pages_reserve(c, g, 256, 2000, none, 256, W, none) == UNSUPPORTED
    assert lib.hyq_pages_fork(c, g, none, 256, 1, none) == INVALID
    assert lib.hyq_pages_fork(c, g, 256, none, 1, none) == INVALID
    assert lib.hyq_pages_fork(c, g, none, none, 0, none) == 0
    assert lib.hyq_pages_truncate(c, g, none, none, 4, none) == INVALID
    assert lib.hyq_pages_truncate(c, g, none, 257, 3, none) == INVALID
    assert lib.hyq_pages_compact(c, g, 257, none, 256, W, none) == INVALID
    assert lib.hyq_pages_compact(c, g, none, none, 256, 10, none) == WORKSPACE


def test_paged_cache_checks_its_arguments(lib):
    c = hyq.PagedCache(cfg(), 10, 3, 5, n_layers=2, device="cpu")
    assert c.pool().shape == (2, 10, 2, 10240) and c.bounds().shape == (2, 10, 2, 272)
    assert c.table().shape == (3, 5) and not c.refs().any() and not c.lens().any()
    bf = torch.bfloat16
    q, out = torch.zeros(2, 1, 8, 128, dtype=bf), torch.zeros(2, 1, 8, 128, dtype=bf)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    for bad in (q.float(), q[:, 0], q[:, :, :4], q.transpose(2, 3), torch.zeros(2, 1, 16, 128, dtype=bf)[:, :, ::2],
                torch.zeros(2, 3, 9, 128, dtype=bf)[:, :2, :8]):
        with pytest.raises(ValueError):
            c.attention(0, bad, out)
    for bad in (out.float(), out[:1], torch.zeros(2, 1, 128, 8, dtype=bf).transpose(2, 3)):
        with pytest.raises(ValueError):
            c.attention(0, q, bad)
    for bad in (torch.zeros(2, dtype=torch.int64), i32(0), i32(0, 1, 2, 3)[::2]):
        with pytest.raises(ValueError):
            c.attention(0, q, out, seqs=bad)
    k = torch.zeros(4, 2, 128, dtype=bf)
    for kk, vv, kw in ((k, k[:3], {}), (k.float(), k.float(), {}), (k, torch.zeros(4, 3, 128, dtype=bf)[:, :2], {}),
                       (k, k, dict(seqs=i32(0, 1))), (k, k, dict(cu_rows=i32(0, 1, 4), seqs=i32(0))),
                       (k, k, dict(cu_rows=torch.zeros(3))), (k, k, dict(k_hat=k.float(), v_hat=k)), (k[0], k[0], {})):
        with pytest.raises(ValueError):
            c.append(0, kk, vv, **kw)
    with pytest.raises(ValueError):
        c.select(0, q, torch.zeros(2, 1, 3, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        c.attention_blocks(0, q, torch.zeros(2, 1, 2, 4), out)
    with pytest.raises(ValueError):
        c.fork(i32(0, 1), i32(2))
    with pytest.raises(ValueError):
        c.reserve(i32(0, 1), i32(1))
    with pytest.raises(ValueError):
        c.compact(torch.zeros(3, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        hyq.PagedCache(cfg(), 10, 3, 5, device="cpu", buffers={"table": torch.zeros(3, 4, dtype=torch.int32)})
    with pytest.raises(ValueError):
        hyq.PagedCache(cfg(), 10, 3, 5, device="cpu", buffers={"tables": torch.zeros(3, 5, dtype=torch.int32)})


def test_paged_cache_takes_given_buffers(lib):
    table = torch.ones(3, 5, dtype=torch.int32)
    c = hyq.PagedCache(cfg(), 10, 3, 5, device="cpu", buffers={"table": table})
    assert c.table() is table and c.c.table == table.data_ptr()


def test_paged_cache_notes_every_stream_on_its_own_memory(lib, monkeypatch):
    """The pool, the tables and the workspaces are not reused, once the cache is dropped, before the streams that its calls
    were queued on have read them."""
    from types import SimpleNamespace
    seen = set()
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.add((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: SimpleNamespace(cuda_stream=5))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 5, raising=False)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: __import__("contextlib").nullcontext())
    c = hyq.PagedCache(cfg(), 10, 3, 5, device="cpu")
    c._lib = SimpleNamespace(**{n: lambda *a: 0 for n in ("hyq_pages_reset", "hyq_pages_reserve", "hyq_paged_attention")})
    q = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16)
    side = SimpleNamespace(cuda_stream=7)
    c.reset(stream=side)
    assert {(t.data_ptr(), 7) for t in c.buf.values()} <= seen
    c.reserve(stream=side)
    c.attention(0, q, torch.empty_like(q))              # the current stream
    c.attention(0, q, torch.empty_like(q), stream=side)
    own = [t.data_ptr() for t in (*c.buf.values(), *c._kept)]
    assert len(own) == 8 and {(p, s) for p in own for s in (5, 7)} <= seen
