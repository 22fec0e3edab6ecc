"""Shared prefixes, cross attention, accumulated weights and eviction without a GPU: workspace sizes and argument checks of
the C entry points (before any launch) and of PagedCache."""
import ctypes

import pytest
import torch

import hybrid_precision_quantized_gb300 as hyq
from hybrid_precision_quantized_gb300 import _lib as L
from tests.test_paged_host import cfg, lib, pages  # noqa: F401

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
W = 1 << 60


def test_workspace_sizes(lib):  # noqa: F811
    c, p = cfg(), pages()
    size = lambda op, b, n=1: hyq.hyq_pages_workspace_size(c, p, op, b, n)  # noqa: E731
    a = [size(L.OP_PAGED_SHARED, b, n) for b, n in ((1, 1), (100, 1), (100, 4), (1024, 64))]
    assert 0 < a[0] < a[1] < a[2] < a[3]
    assert size(L.OP_PAGED_SHARED, 100, 4) == size(L.OP_PAGED_SHARED, 400, 1)   # their product alone counts
    for b, n in ((0, 1), (1025, 1), (1, 0), (1, 65)):
        assert size(L.OP_PAGED_SHARED, b, n) == 0
    assert 0 < size(L.OP_PAGED_CROSS, 1) <= size(L.OP_PAGED_CROSS, 1024)
    assert size(L.OP_PAGED_CROSS, 5, 0) == size(L.OP_PAGED_CROSS, 5, 1000)
    assert size(L.OP_PAGED_CROSS, 1025) == 0 and size(L.OP_PAGES_EVICT, 0) == 0 and size(L.OP_PAGES_EVICT, 1025) == 0
    # a mask and a count per page, head, sequence and layer, and the rows
    assert size(L.OP_PAGES_EVICT, 3) >= 3 * 5 * 2 * 2 * 12
    big = hyq.hyq_pages_workspace_size(c, pages(n_layers=64, max_blocks=1 << 22), L.OP_PAGES_EVICT, 1024)
    assert big >= 64 * (1 << 22) * 1024 * 2 * 12


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation runs only without a GPU")
def test_entry_points_refuse_before_launch(lib):  # noqa: F811
    c, none = ctypes.byref(cfg()), None
    p = pages(**{n: 4096 * (i + 1) for i, n in enumerate(L.PAGES_FIELDS)})
    g = ctypes.byref(p)
    # (layer, seqs, batch, n_q, q, ldq, out, lse, ws, bytes)
    lse = lambda layer=0, seqs=none, b=1, n=1, q=256, ld=1024, o=256, e=256, ws=256, by=W: lib.hyq_paged_attention_lse(  # noqa: E731
        c, g, layer, seqs, b, n, q, ld, o, e, ws, by, none)
    for kw in (dict(layer=2), dict(b=4), dict(n=0), dict(q=none), dict(q=264), dict(ld=1016), dict(ld=1028), dict(o=none),
               dict(o=264), dict(e=258), dict(seqs=258)):
        assert lse(**kw) == INVALID, kw
    assert lse(n=65) == UNSUPPORTED and lse(b=1025, seqs=256) == UNSUPPORTED
    assert lse(ws=none) == WORKSPACE and lse(ws=128) == WORKSPACE and lse(by=100) == WORKSPACE and lse(b=0, q=none, o=none) == 0
    sh = lambda layer=0, seqs=none, b=1, n=1, cu=256, ns=256, ng=1, q=256, ld=1024, o=256, ws=256, by=W: lib.hyq_paged_attention_shared(  # noqa: E731
        c, g, layer, seqs, b, n, cu, ns, ng, q, ld, o, ws, by, none)
    for kw in (dict(layer=-1), dict(b=4), dict(b=-1), dict(n=0), dict(ng=-1), dict(cu=none), dict(ns=none), dict(cu=258),
               dict(ns=257), dict(q=none), dict(ld=1020), dict(o=none)):
        assert sh(**kw) == INVALID, kw
    assert sh(ng=1025) == UNSUPPORTED and sh(n=65) == UNSUPPORTED and sh(b=0, q=none, o=none) == 0
    need = hyq.hyq_pages_workspace_size(cfg(), p, L.OP_PAGED_SHARED, 1, 1)
    assert sh(by=need - 1) == WORKSPACE and sh(ws=none) == WORKSPACE
    cr = lambda layer=0, seqs=none, b=1, cu=256, t=5, q=256, ld=1024, o=256, ws=256, by=W: lib.hyq_paged_cross_attention(  # noqa: E731
        c, g, layer, seqs, b, cu, t, q, ld, o, ws, by, none)
    for kw in (dict(layer=2), dict(b=4), dict(t=-1), dict(cu=none), dict(cu=257), dict(q=none), dict(q=8), dict(ld=1000),
               dict(ld=1025), dict(o=none), dict(seqs=257)):
        assert cr(**kw) == INVALID, kw
    assert cr(b=0, q=none) == 0 and cr(t=0, q=none) == 0 and cr(cu=none, t=1, q=none) == INVALID
    assert cr(t=1 << 28) == UNSUPPORTED and cr(seqs=256, b=1025) == UNSUPPORTED
    need = hyq.hyq_pages_workspace_size(cfg(), p, L.OP_PAGED_CROSS, 1)
    assert cr(by=need - 1) == WORKSPACE and cr(ws=64) == WORKSPACE
    ac = lambda layer=0, seqs=none, b=1, n=1, q=256, ld=1024, e=256, new=none, m=256: lib.hyq_paged_accumulate(  # noqa: E731
        c, g, layer, seqs, b, n, q, ld, e, new, m, none)
    for kw in (dict(layer=2), dict(b=4), dict(n=0), dict(q=none), dict(ld=8), dict(e=none), dict(e=255), dict(new=258),
               dict(m=none), dict(m=264)):
        assert ac(**kw) == INVALID, kw
    assert ac(n=65) == UNSUPPORTED and ac(b=0, q=none, m=none) == 0
    ev = lambda seqs=none, b=1, keep=256, f=0, la=0, m=256, ws=256, by=W: lib.hyq_pages_evict(  # noqa: E731
        c, g, seqs, b, keep, f, la, m, ws, by, none)
    for kw in (dict(b=4), dict(keep=none), dict(keep=258), dict(f=-1), dict(la=-1), dict(f=2 ** 31 - 1, la=1), dict(m=none),
               dict(m=8), dict(seqs=1)):
        assert ev(**kw) == INVALID, kw
    need = hyq.hyq_pages_workspace_size(cfg(), p, L.OP_PAGES_EVICT, 1)
    assert ev(by=need - 1) == WORKSPACE and ev(ws=none) == WORKSPACE and ev(b=0, keep=none, m=none) == 0
    assert ev(seqs=256, b=1025) == UNSUPPORTED
    for name in L.PAGES_FIELDS:      # every buffer is needed
        bad = pages(**{n: 4096 * (i + 1) for i, n in enumerate(L.PAGES_FIELDS)})
        setattr(bad, name, None)
        b = ctypes.byref(bad)
        assert lib.hyq_paged_attention_shared(c, b, 0, none, 1, 1, 256, 256, 1, 256, 1024, 256, 256, W, none) == INVALID
        assert lib.hyq_paged_cross_attention(c, b, 0, none, 1, 256, 5, 256, 1024, 256, 256, W, none) == INVALID
        assert lib.hyq_paged_accumulate(c, b, 0, none, 1, 1, 256, 1024, 256, none, 256, none) == INVALID
        assert lib.hyq_pages_evict(c, b, none, 1, 256, 0, 0, 256, 256, W, none) == INVALID


def test_paged_cache_checks_its_arguments(lib):  # noqa: F811
    c = hyq.PagedCache(cfg(), 10, 3, 5, n_layers=2, device="cpu")
    bf, f32 = torch.bfloat16, torch.float32
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    q, out, lse = torch.zeros(2, 1, 8, 128, dtype=bf), torch.zeros(2, 1, 8, 128, dtype=bf), torch.zeros(2, 1, 8)
    for bad in (lse.double(), lse[:1], torch.zeros(2, 1, 16)[..., ::2]):
        with pytest.raises(ValueError):
            c.attention(0, q, out, lse=bad)
    for kw in (dict(cu_groups=i32(0, 1), n_shared=i32(0, 0)), dict(cu_groups=i32(0, 2).long(), n_shared=i32(0)),
               dict(cu_groups=i32(0, 2), n_shared=torch.zeros(1)), dict(cu_groups=i32(0, 2), n_shared=i32(0), seqs=i32(0))):
        with pytest.raises(ValueError):
            c.attention_shared(0, q, out, **kw)
    with pytest.raises(ValueError):
        c.attention_shared(0, q[:, 0], out, i32(0, 2), i32(0))
    with pytest.raises(ValueError):
        c.attention_shared(0, q, out[:1], i32(0, 2), i32(0))
    t = torch.zeros(5, 8, 128, dtype=bf)
    for qq, oo, kw in ((t[None], t, {}), (t, t[:4], {}), (t.float(), t, {}), (t, t.float(), {}), (t, t, dict(seqs=i32(0, 1))),
                       (t, t, dict(cu_q=i32(0, 5).long())), (t, t, dict(cu_q=i32(0, 2, 5), seqs=i32(0))),
                       (t[:, :4], t[:, :4], {})):
        with pytest.raises(ValueError):
            c.cross_attention(0, qq, oo, **kw)
    assert c.mass_shape == (2, 10, 2, 64)
    mass = torch.zeros(c.mass_shape)
    for ee, mm, kw in ((lse.to(bf), mass, {}), (lse, mass[0], {}), (lse, mass.double(), {}), (lse, mass, dict(n_new=i32(1))),
                       (lse, torch.zeros(2, 10, 64, 2, dtype=f32).transpose(2, 3), {})):
        with pytest.raises(ValueError):
            c.accumulate(0, q, ee, mm, **kw)
    for mm, kk, kw in ((mass[:1], i32(0), {}), (mass, torch.zeros(1), {}), (mass, i32(1, 2), dict(seqs=i32(0)))):
        with pytest.raises(ValueError):
            c.evict(mm, kk, **kw)
