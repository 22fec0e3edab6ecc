"""Calls on the paged cache that its documentation allows, beside those of
test_gpu_paged.py."""
import numpy as np
import pytest
import torch

from hybrid_precision_quantized_gb300 import HyqError, hyq_read_device_error, unpack_qblocks
from hybrid_precision_quantized_gb300 import _lib as L
from oracle.quant import quantize
from tests.gpu_util import mixed_rows
from tests.test_gpu_paged import check_bounds, check_rows, grow, ints, make, np64, queries

pytestmark = pytest.mark.gpu


def test_choice_reports_queries_that_are_not_finite_whatever_k_is(hyq):
    """Also where every block is taken; a token that sees nothing is not looked at."""
    cache = make(2, 2, 16, 3, 16)
    grow(cache, [0, 1], [64 * 10, 5], 1)
    for seqs, bad, err in (([0], 0, L.DEVERR_SCORE), ([1], 0, L.DEVERR_SCORE), ([2, 0], 0, 0), ([2, 1], 0, 0),
                           ([0, 1, 2], 1, L.DEVERR_SCORE)):
        for k in (3, 10, 40):
            q = queries(6, len(seqs), 1, 2)
            want, sel = (torch.full((len(seqs), 1, 2, k), 50, dtype=torch.int32, device="cuda") for _ in range(2))
            cache.select(0, q, want, seqs=ints(seqs), n_first=0, n_last=0)
            assert hyq_read_device_error(cache.err()) == 0
            q[bad, 0, 1, 7] = float("nan")
            cache.select(0, q, sel, seqs=ints(seqs), n_first=0, n_last=0)
            assert hyq_read_device_error(cache.err()) == err, (seqs, k)
            cache.err().zero_()
            assert torch.equal(sel[:, :, 0], want[:, :, 0])
            if k >= 10 or err == 0:
                assert torch.equal(sel, want)


def test_append_with_a_bad_pair_between_two_good_ones(hyq):
    """A pair of cu_rows that descends is left out and reported; the others are written whole, though they share rows and
    so reach more pages than as many distinct rows could."""
    for HKV, n in ((2, 640), (8, 1000)):
        cache = make(HKV, HKV, 64, 3, 20)
        cache.reserve(ints([0, 1, 2]), ints([n, 0, n + 7]))
        before = cache.pool().clone()
        k, v = (mixed_rows(s, (HKV, n, 128)).transpose(0, 1).contiguous() for s in (1, 2))
        kh, vh = (torch.full((n, HKV, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cache.append(0, k.cuda(), v.cuda(), seqs=ints([0, 1, 2]), cu_rows=ints([0, n, 0, n]), k_hat=kh, v_hat=vh)
        assert hyq_read_device_error(cache.err()) == L.DEVERR_INDEX
        assert kh.isfinite().all() and vh.isfinite().all()
        for h in range(HKV):
            check_rows(cache, 0, h, np64(k[:, h]), np64(v[:, h]))
            check_bounds(cache, 0, h, np64(k[:, h]))
        # sequence 2 begins with seven rows that no call wrote
        pages = cache.table()[2, : -(-(n + 7) // 64)].long()
        for h in range(HKV):
            kc, vc, ks, kz, vs, vz = unpack_qblocks(cache.pool()[0, pages, h].cpu().numpy(), n + 7, 4, 4)
            for got, want in zip((kc, ks, kz, vc, vs, vz), (*quantize(np64(k[:, h]), 4), *quantize(np64(v[:, h]), 4))):
                got = got[7:]
                if want.dtype == np.float16:
                    got, want = got.view(np.uint16), want.view(np.uint16)
                assert np.array_equal(got, want)
        untouched = [p for p in range(64) if p not in set(pages.tolist()) | set(cache.table()[0, : -(-n // 64)].tolist())]
        assert torch.equal(cache.pool()[0, untouched], before[0, untouched])


def test_workspaces_stay_few_as_calls_grow(hyq):
    """One sequence more each time: what is kept stays within a few times the largest call's need."""
    n = 300
    cache = make(2, 2, 320, n, 200)
    grow(cache, list(range(n)), [5 + i % 50 for i in range(n)], 1)
    q = queries(1, n, 1, 2)
    want, out = torch.empty_like(q), torch.empty_like(q)
    other = make(2, 2, 320, n, 200)
    grow(other, list(range(n)), [5 + i % 50 for i in range(n)], 1)
    other.attention(0, q, want)
    sel = torch.empty(n, 1, 2, 3, dtype=torch.int32, device="cuda")
    for b in range(1, n + 1):
        cache.attention(0, q[:b], out[:b])
        cache.select(0, q[:b], sel[:b])
        assert torch.equal(out[:b], want[:b])
    kept = sum(t.nbytes for t in cache._kept)
    need = [L.hyq_pages_workspace_size(cache.cfg, cache.c, op, n) for op in (L.OP_PAGED_ATTENTION, L.OP_PAGED_SELECT)]
    assert len(cache._kept) <= 1 + 2 * 10 and kept <= 10 * sum(need)     # 1, 2, 4 .. 512, and the reserve's
    for b, n_q in ((1024, 1), (1024, 33), (700, 64), (1024, 64)):        # up to the largest call there is
        assert cache.workspace(L.OP_PAGED_ATTENTION, b, n_q).nbytes >= \
            L.hyq_pages_workspace_size(cache.cfg, cache.c, L.OP_PAGED_ATTENTION, b, n_q)
    for b, n_q in ((1025, 64), (1024, 65)):
        with pytest.raises(ValueError):
            cache.workspace(L.OP_PAGED_ATTENTION, b, n_q)
    assert hyq_read_device_error(cache.err()) == 0


def test_a_cache_may_be_dropped_while_its_calls_are_queued(hyq):
    """Its memory is not reused before they have run, whichever stream they are on and however it was named."""
    for named in (True, False):
        cache = make(4, 2, 40, 2, 32)
        grow(cache, [0, 1], [1500, 700], 3)
        q = queries(1, 2, 1, 4)
        want, out = torch.empty_like(q), torch.zeros_like(q)
        cache.attention(0, q, want)
        sizes = [t.nbytes for t in (*cache.buf.values(), *cache._kept)]
        side = torch.cuda.Stream()
        big = torch.randn(4096, 4096, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(30):
                big = big @ big * 1e-3
            if not named:
                cache.attention(0, q, out)
        if named:
            cache.attention(0, q, out, stream=side)
        del cache
        junk = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del junk, big


def test_tables_of_more_rows_than_a_call_takes(hyq):
    """3000 sequences: reserved in parts, refused as a whole, shortened and freed as a whole."""
    n = 3000
    cache = make(2, 1, 2 * n, n, 2)
    for at in range(0, n, 1000):
        cache.reserve(ints(list(range(at, at + 1000))), ints([100] * 1000))
    with pytest.raises(HyqError) as e:
        cache.reserve()
    assert e.value.status == 2
    assert (cache.lens() == 100).all() and int(cache.refs().sum()) == 2 * n
    lens = torch.arange(n, dtype=torch.int32, device="cuda") % 100
    cache.truncate(None, lens)
    assert torch.equal(cache.lens(), lens) and int(cache.refs().sum()) == int(((lens + 63) // 64).sum())
    with pytest.raises(HyqError):
        cache.truncate(ints(list(range(1025))))
    cache.truncate()
    assert not cache.lens().any() and not cache.refs().any()
    assert hyq_read_device_error(cache.err()) == 0


def test_the_plain_bindings_make_the_same_calls(hyq):
    """A step through hyq_pages_* and hyq_paged_* on raw sizes gives what PagedCache gives."""
    HQ, HKV, n, nb = 4, 2, 3, 6
    caches = [make(HQ, HKV, 24, n + 1, nb) for _ in range(2)]
    rows = [mixed_rows(s, (HKV, 300, 128)).transpose(0, 1).contiguous().cuda() for s in (1, 2)]
    one = [mixed_rows(s, (HKV, 2, 128)).transpose(0, 1).contiguous().cuda() for s in (3, 4)]
    q, seqs, cu, counts = queries(5, 2, 1, HQ), ints([0, 1]), ints([0, 200, 300]), ints([200, 100])
    results = []
    for plain, c in zip((False, True), caches):
        hats = [torch.zeros_like(rows[0]) for _ in range(2)]
        out, sparse = torch.zeros_like(q), torch.zeros_like(q)
        sel = torch.zeros(2, 1, HKV, 2, dtype=torch.int32, device="cuda")
        if plain:
            cfg, p = c.cfg, c.c
            ws = {op: torch.zeros(L.hyq_pages_workspace_size(cfg, p, op, 2), dtype=torch.uint8, device="cuda")
                  for op in (L.OP_PAGED_ATTENTION, L.OP_PAGED_SELECT, L.OP_PAGES_RESERVE, L.OP_PAGES_COMPACT)}
            ld = HKV * 128
            L.hyq_pages_reset(cfg, p)
            L.hyq_pages_reserve(cfg, p, seqs, 2, counts, ws[L.OP_PAGES_RESERVE])
            L.hyq_paged_append(cfg, p, 0, seqs, 2, cu, 300, *rows, ld, *hats)
            L.hyq_pages_fork(cfg, p, seqs, ints([2, 3]), 2)
            L.hyq_pages_truncate(cfg, p, ints([0, 3]), ints([70, 0]), 2)
            L.hyq_pages_reserve(cfg, p, ints([2, 0]), 2, None, ws[L.OP_PAGES_RESERVE])
            L.hyq_paged_append(cfg, p, 0, ints([2, 0]), 2, None, 2, *one, ld)
            L.hyq_pages_compact(cfg, p, None, None, ws[L.OP_PAGES_COMPACT])
            L.hyq_paged_attention(cfg, p, 0, ints([2, 1]), 2, 1, q, HQ * 128, out, ws[L.OP_PAGED_ATTENTION])
            L.hyq_paged_select(cfg, p, 0, ints([2, 1]), 2, 1, q, HQ * 128, 2, 1, 1, sel, ws[L.OP_PAGED_SELECT])
            L.hyq_paged_attention_blocks(cfg, p, 0, ints([2, 1]), 2, 1, q, HQ * 128, sel, 2, sparse,
                                         ws[L.OP_PAGED_ATTENTION])
        else:
            c.reserve(seqs, counts)
            c.append(0, *rows, seqs=seqs, cu_rows=cu, k_hat=hats[0], v_hat=hats[1])
            c.fork(seqs, ints([2, 3]))
            c.truncate(ints([0, 3]), ints([70, 0]))
            c.reserve(ints([2, 0]))
            c.append(0, *one, seqs=ints([2, 0]))
            c.compact()
            c.attention(0, q, out, seqs=ints([2, 1]))
            c.select(0, q, sel, seqs=ints([2, 1]))
            c.attention_blocks(0, q, sel, sparse, seqs=ints([2, 1]))
        assert hyq_read_device_error(c.err()) == 0
        results.append([*hats, out, sel, sparse, c.lens(), c.refs(), c.pool(), c.bounds()])
    assert results[0][5].tolist() == [71, 100, 201, 0] and results[0][2].any() and results[0][4].any()
    assert all(torch.equal(a, b) for a, b in zip(*results))
