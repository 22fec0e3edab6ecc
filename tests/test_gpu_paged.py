"""GPU parity of the paged cache: quantised rows, bounds and page tables exact,
attention within a bound counted from its roundings, block choice exact."""
import numpy as np
import pytest
import torch

from hybrid_precision_quantized_gb300 import (HyqError, PagedCache, hyq_read_device_error, make_config,
                                              unpack_qblocks)
from hybrid_precision_quantized_gb300 import _lib as L
from oracle import paged as P
from oracle.quant import QuantRangeError, quantize
from tests.gpu_util import mixed_rows, tie_rows

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def np64(t):
    return t.detach().double().cpu().numpy()


def make(HQ, HKV, n_pages, n_seqs, max_blocks, n_layers=1, bits=(4, 4), fill=0xFF):
    """A cache whose pool and bounds start as garbage (0xFF: NaN metadata)."""
    cfg = make_config(1, HQ, HKV, capacity=64, bits_k=bits[0], bits_v=bits[1])
    c = PagedCache(cfg, n_pages, n_seqs, max_blocks, n_layers)
    c.pool().fill_(fill)
    c.bounds().fill_(fill)
    c.reset()
    return c


def pages_of(cache, seq):
    n = int(cache.lens()[seq])
    return cache.table()[seq, : -(-n // 64)].tolist(), n


def check_rows(cache, seq, h, k, v, layer=0):
    """Sequence ``seq`` holds exactly the rows k, v [n, 128] of head h."""
    pages, n = pages_of(cache, seq)
    assert n == len(k)
    bk, bv = cache.cfg.bits_k, cache.cfg.bits_v
    blocks = cache.pool()[layer, pages, h].cpu().numpy()
    kc, vc, ks, kz, vs, vz = unpack_qblocks(blocks, n, bk, bv)
    for got, want in zip((kc, ks, kz, vc, vs, vz), (*quantize(k, bk), *quantize(v, bv))):
        if want.dtype == np.float16:
            got, want = got.view(np.uint16), want.view(np.uint16)
        assert np.array_equal(got, want)


def check_bounds(cache, seq, h, k, layer=0):
    pages, n = pages_of(cache, seq)
    for i, p in enumerate(pages):
        rec = cache.bounds()[layer, p, h].cpu().numpy()
        lo, hi, e = P.bounds(k[64 * i:64 * i + 64])
        assert rec[256:260].view(np.int32)[0] == e
        assert np.array_equal(rec[:128].view(np.int8), lo) and np.array_equal(rec[128:256].view(np.int8), hi)


def grow(cache, seqs, counts, seed, layer=0, one=False, rows=None, hats=False, strided=False, reserve=True):
    """Append ``counts`` random rows to the sequences; returns (k, v) [rows, HKV, 128] and the hats."""
    hkv, n = cache.cfg.num_kv_heads, sum(counts)
    if rows is None:
        k, v = (mixed_rows(seed + i, (hkv, n, 128)).transpose(0, 1).contiguous() if n else
                torch.zeros(0, hkv, 128, dtype=torch.bfloat16) for i in range(2))
    else:
        k, v = rows
    if reserve:
        cache.reserve(ints(seqs), ints(counts))
    if strided:     # rows inside a wider projection output
        wide = torch.full((n, 3 * hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :hkv], wide[:, hkv:2 * hkv] = k.cuda(), v.cuda()
        kd, vd = wide[:, :hkv], wide[:, hkv:2 * hkv]
    else:
        kd, vd = k.cuda(), v.cuda()
    kh = vh = None
    if hats:
        kh, vh = (torch.full((n, hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu = None if one else ints(np.concatenate([[0], np.cumsum(counts)]).tolist())
    cache.append(layer, kd, vd, seqs=ints(seqs), cu_rows=cu, k_hat=kh, v_hat=vh)
    return k, v, kh, vh


class History:
    """What each sequence was given, row by row."""

    def __init__(self, n_seqs, hkv):
        self.k = [np.zeros((0, hkv, 128)) for _ in range(n_seqs)]
        self.v = [np.zeros((0, hkv, 128)) for _ in range(n_seqs)]

    def add(self, seqs, counts, k, v):
        at = 0
        for s, n in zip(seqs, counts):
            self.k[s] = np.concatenate([self.k[s], np64(k[at:at + n])])
            self.v[s] = np.concatenate([self.v[s], np64(v[at:at + n])])
            at += n


def check_attention(cache, hist, q, out, seqs, sel=None, layer=0):
    """out [B, n_q, HQ, 128] against the oracle over the history of each sequence."""
    hkv, hq = cache.cfg.num_kv_heads, cache.cfg.num_q_heads
    g = hq // hkv
    qn, on = np64(q), np64(out)
    assert np.isfinite(on).all()
    worst = 0.0
    for b, s in enumerate(seqs):
        n = len(hist.k[s])
        for h in range(hkv):
            if n:
                kd, kp, _ = P.dequantised(hist.k[s][:, h], cache.cfg.bits_k)
                vd, vp, vc = P.dequantised(hist.v[s][:, h], cache.cfg.bits_v)
            for i in range(q.shape[1]):
                lim = n - q.shape[1] + 1 + i
                vis = np.arange(n) < lim
                if sel is not None:
                    vis &= np.isin(np.arange(n) // 64, sel[b][i][h])
                for r in range(h * g, h * g + g):
                    if not vis.any():
                        assert not on[b, i, r].any()
                        continue
                    want = P.attend(qn[b, i, r], kd, vd, vis)
                    tol = P.attend_error(qn[b, i, r], kd, kp, vp, vc, vis, want)
                    err = np.abs(on[b, i, r] - want)
                    worst = max(worst, float((err / tol).max()))
                    assert (err <= tol).all(), (b, s, i, r, n, float((err / tol).max()))
    return worst


def queries(seed, b, n_q, hq):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(b, n_q, hq, 128, generator=gen) * 1.5).to(torch.bfloat16).cuda()


# --- rows ------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [(4, 4), (8, 8), (4, 8), (8, 4)])
@pytest.mark.parametrize("counts", [[1], [1, 5, 0, 16], [64, 63, 65], [130, 7, 1, 0, 257], [15, 17]])
def test_append_is_the_quantiser_and_keeps_other_rows(hyq, bits, counts):
    HKV, seqs = 3, [4, 1, 3, 0, 2][:len(counts)]
    cache = make(6, HKV, 32, 5, 13, bits=bits)     # 3 * 257 rows: 13 pages
    hist = History(5, HKV)
    for step in range(3):     # the second and third call begin inside pages
        k, v, kh, vh = grow(cache, seqs, counts, 10 * step + 1, hats=step != 1, strided=step == 2)
        hist.add(seqs, counts, k, v)
        if kh is not None:
            for x, hat, bits_x in ((k, kh, bits[0]), (v, vh, bits[1])):
                c, s, z = quantize(np64(x), bits_x)
                val = c.astype(np.float32).reshape(-1, HKV, 4, 32) * s.astype(np.float32)[..., None] + \
                    z.astype(np.float32)[..., None]
                assert torch.equal(hat.cpu(), torch.from_numpy(val.reshape(-1, HKV, 128)).to(torch.bfloat16))
        used = {p for s in range(5) for p in pages_of(cache, s)[0]}
        for s in range(5):
            for h in range(HKV):
                check_rows(cache, s, h, hist.k[s][:, h], hist.v[s][:, h])
                check_bounds(cache, s, h, hist.k[s][:, h])
        spare = [p for p in range(32) if p not in used]
        assert (cache.pool()[0, spare] == 0xFF).all() and (cache.bounds()[0, spare] == 0xFF).all()
    # rows that no call wrote keep their bits
    for s in range(5):
        pages, n = pages_of(cache, s)
        if n % 64:
            kc, vc, ks, *_ = unpack_qblocks(cache.pool()[0, pages, 1].cpu().numpy(), 64 * len(pages), *bits)
            assert (kc[n:] == (1 << bits[0]) - 1).all() and (vc[n:] == (1 << bits[1]) - 1).all()
            assert (ks[n:].view(np.uint16) == 0xFFFF).all()
    assert hyq_read_device_error(cache.err()) == 0


@pytest.mark.parametrize("bits", [(4, 4), (8, 8), (4, 8), (8, 4)])
def test_append_one_row_each_equals_ragged_append(hyq, bits):
    HKV, n = 2, 70
    rows = [tie_rows(s, (n, HKV, 128), bits[i]) for i, s in enumerate((5, 6))]
    a, b = make(4, HKV, 8, 3, 4, bits=bits), make(4, HKV, 8, 3, 4, bits=bits)
    for i in range(n):
        x = [r[i:i + 1].expand(2, -1, -1).contiguous() for r in rows]
        grow(a, [2, 0], [1, 1], 0, one=True, rows=x)
    y = [torch.cat([r, r]) for r in rows]
    grow(b, [2, 0], [n, n], 0, rows=y)
    for s in (0, 2):
        pa, pb = pages_of(a, s)[0], pages_of(b, s)[0]
        assert torch.equal(a.pool()[0, pa], b.pool()[0, pb]) and torch.equal(a.bounds()[0, pa], b.bounds()[0, pb])
        check_rows(a, s, 1, np64(rows[0][:, 1]), np64(rows[1][:, 1]))
        check_bounds(a, s, 1, np64(rows[0][:, 1]))
    assert hyq_read_device_error(a.err()) == 0


@pytest.mark.parametrize("one", [False, True])
def test_append_rows_that_fp16_cannot_hold(hyq, one):
    cache = make(2, 1, 4, 1, 2)
    k, v = mixed_rows(1, (1, 1, 128)), mixed_rows(2, (1, 1, 128))
    k[0, 0, 40], v[0, 0, 100], v[0, 0, 5] = -70000.0, float("nan"), float("inf")
    grow(cache, [0], [1], 0, one=one, rows=(k, v))
    assert hyq_read_device_error(cache.err()) == L.DEVERR_QUANT_RANGE
    k[0, 0, 32:64], v[0, 0, 96:], v[0, 0, :32] = 0, 0, 0
    check_rows(cache, 0, 0, np64(k[:, 0]), np64(v[:, 0]))
    check_bounds(cache, 0, 0, np64(k[:, 0]))
    with pytest.raises(QuantRangeError):
        quantize(np.full((1, 128), np.nan))


def test_append_leaves_out_what_does_not_fit(hyq):
    cache = make(2, 1, 6, 4, 2)
    grow(cache, [0, 1, 2], [10, 20, 30], 3)
    before = cache.pool().clone()
    k = torch.zeros(12, 1, 128, dtype=torch.bfloat16, device="cuda")
    # sequence 0 holds 10 rows, not 12; there is no sequence 9; rows 5 .. 13 of 12
    for seqs, cu in (([0], [0, 12]), ([9], [0, 3]), ([1], [5, 13]), ([1], [4, 2]), ([3], [0, 1]), ([-1], [0, 1])):
        cache.append(0, k, k, seqs=ints(seqs), cu_rows=ints(cu))
        assert hyq_read_device_error(cache.err()) == L.DEVERR_INDEX
        cache.err().zero_()
    assert torch.equal(cache.pool(), before)
    cache.table()[1, 0] = 77     # outside the pool
    cache.append(0, k[:3], k[:3], seqs=ints([1]), cu_rows=ints([0, 3]))
    assert hyq_read_device_error(cache.err()) == L.DEVERR_INDEX and torch.equal(cache.pool(), before)
    cache.err().zero_()
    cache.append(0, k[:0], k[:0], seqs=ints([1]), cu_rows=ints([0, 0]))
    assert hyq_read_device_error(cache.err()) == 0


# --- attention --------------------------------------------------------------------------------------------------------

LENS = [0, 1, 15, 16, 17, 63, 64, 65, 129, 300]


@pytest.mark.parametrize("HQ,HKV,bits,n_q", [(4, 4, (4, 4), 1), (8, 2, (4, 4), 1), (8, 1, (4, 4), 1), (10, 2, (4, 4), 3),
                                             (14, 2, (4, 4), 2), (8, 2, (8, 8), 1), (8, 2, (4, 8), 5),
                                             (8, 2, (8, 4), 4), (3, 1, (4, 4), 16), (16, 2, (8, 8), 2)])
def test_attention_over_ragged_lengths(hyq, HQ, HKV, bits, n_q):
    cache = make(HQ, HKV, 30, len(LENS), 6, bits=bits)
    hist = History(len(LENS), HKV)
    seqs = list(range(len(LENS)))
    k, v, _, _ = grow(cache, seqs, LENS, HQ + n_q)
    hist.add(seqs, LENS, k, v)
    order = [7, 3, 9, 0, 1, 8, 2, 5, 6, 4, 9, 9]          # any order, and again
    q = queries(HQ, len(order), n_q, HQ)
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out, seqs=ints(order))
    assert hyq_read_device_error(cache.err()) == 0
    print(f"error / bound: {check_attention(cache, hist, q, out, order):.3f}")
    # again, with the rows of a wider projection output; the same bits
    wide = torch.full((len(order), n_q, HQ + 3, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 2:HQ + 2] = q
    again = torch.full_like(q, float("nan"))
    cache.attention(0, wide[:, :, 2:HQ + 2], again, seqs=ints(order))
    assert torch.equal(out, again)


@pytest.mark.parametrize("B,HQ,HKV,n,n_q", [(1, 8, 2, 20011, 1), (1, 1, 1, 30000, 1), (3, 8, 2, 5000, 3), (1, 4, 1, 16384, 1)])
def test_long_sequences_are_shared_out_and_joined(hyq, B, HQ, HKV, n, n_q):
    """Split over many blocks, whose partials are joined: against the oracle, and the same bits every time."""
    nb = -(-n // 64)
    cache = make(HQ, HKV, B * nb, B, nb)
    k = torch.randn(n * B, HKV, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    v = torch.randn(n * B, HKV, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    grow(cache, list(range(B)), [n] * B, 0, rows=(k, v))
    hist = History(B, HKV)
    hist.add(range(B), [n] * B, k, v)
    q = queries(3, B, n_q, HQ)
    outs = []
    for _ in range(3):
        out = torch.full_like(q, float("nan"))
        cache.attention(0, q, out)
        outs.append(out)
    print(f"error / bound: {check_attention(cache, hist, q, outs[0], range(B)):.3f}")
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_attention_of_many_sequences(hyq):
    """1024 sequences (the largest call), most of them empty or a few rows long."""
    lens = [(7 * i) % 23 if i % 3 else 0 for i in range(1024)]
    lens[1000] = 500
    cache = make(4, 2, 1100, 1024, 8)
    k, v, _, _ = grow(cache, list(range(1024)), lens, 5)
    hist = History(1024, 2)
    hist.add(range(1024), lens, k, v)
    q = queries(6, 1024, 1, 4)
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    check_attention(cache, hist, q, out, range(1024))


def test_attention_of_extreme_values(hyq):
    """Peaked logits (one row takes all), equal logits, zero queries, large values, tiny values."""
    cache = make(2, 1, 16, 5, 4)
    n = 150
    gen = torch.Generator().manual_seed(8)
    base = torch.randn(n, 1, 128, generator=gen)
    ks = [base * 200, torch.ones(n, 1, 128), base, base * 1e-5, base]
    ks[0][40] *= 3
    vs = [base * 1000, base, base * 30000 / base.abs().max(), base * 1e-6, base]
    hist = History(5, 1)
    for s in range(5):
        k, v = ks[s].to(torch.bfloat16), vs[s].to(torch.bfloat16)
        grow(cache, [s], [n], 0, rows=(k, v))
        hist.add([s], [n], k, v)
    q = queries(9, 5, 1, 2)
    q[4] = 0
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    assert hyq_read_device_error(cache.err()) == 0
    check_attention(cache, hist, q, out, range(5))


def test_attention_reports_bad_sequences_and_pages(hyq):
    cache = make(4, 2, 8, 3, 4)
    k, v, _, _ = grow(cache, [0, 1], [100, 100], 1)
    hist = History(3, 2)
    hist.add([0, 1], [100, 100], k, v)
    q = queries(1, 4, 1, 4)
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out, seqs=ints([0, 7, -2, 2]))
    assert hyq_read_device_error(cache.err()) == L.DEVERR_INDEX
    check_attention(cache, hist, q[:1], out[:1], [0])
    assert not out[1:].any()
    cache.err().zero_()
    cache.table()[1, 1] = 8
    cache.attention(0, q[:2], out[:2], seqs=ints([1, 0]))
    assert hyq_read_device_error(cache.err()) == L.DEVERR_INDEX
    check_attention(cache, hist, q[1:2], out[1:2], [0])     # the other sequence is as it should be


def test_pool_past_32_bits(hyq):
    """Pages and records past 4 GiB of the pool."""
    n_pages = (5 << 30) // (8 * 10240)
    cfg = make_config(1, 8, 8, capacity=64)
    cache = PagedCache(cfg, n_pages, 2, 8)
    cache.reset()
    cache.refs()[: n_pages - 5] = 1      # only the last pages are free
    k, v, _, _ = grow(cache, [1], [200], 4)
    assert pages_of(cache, 1)[0] == list(range(n_pages - 5, n_pages - 1))
    hist = History(2, 8)
    hist.add([1], [200], k, v)
    check_rows(cache, 1, 7, hist.k[1][:, 7], hist.v[1][:, 7])
    q = queries(2, 1, 1, 8)
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out, seqs=ints([1]))
    check_attention(cache, hist, q, out, [1])
    sel = torch.full((1, 1, 8, 2), 99, dtype=torch.int32, device="cuda")
    cache.select(0, q, sel, seqs=ints([1]))
    check_choice(cache, q, sel, [1], 1, 1)


# --- block choice -----------------------------------------------------------------------------------------------------

def check_choice(cache, q, sel, seqs, n_first, n_last, layer=0):
    g = cache.cfg.num_q_heads // cache.cfg.num_kv_heads
    qn, got, bounds = np64(q), sel.cpu().numpy(), cache.bounds()[layer].cpu().numpy()
    k, n_q = sel.shape[-1], q.shape[1]
    for b, s in enumerate(seqs):
        pages, n = pages_of(cache, s)
        rec = bounds[pages]
        for i in range(n_q):
            nb = -(-max(0, n - n_q + 1 + i) // 64)
            for h in range(cache.cfg.num_kv_heads):
                codes = P.query_codes(qn[b, i, h * g:h * g + g])
                scores = [P.block_score(codes, r[:128].view(np.int8).astype(np.int64),
                                        r[128:256].view(np.int8).astype(np.int64),
                                        int(r[256:260].view(np.int32)[0])) for r in rec[:nb, h]]
                want = P.choose_blocks(scores, k, n_first, n_last)
                assert got[b, i, h].tolist() == want + [-1] * (k - len(want)), (b, i, h)


@pytest.mark.parametrize("HQ,HKV,n_q,k,first,last", [(8, 2, 1, 4, 1, 1), (8, 1, 2, 7, 0, 0), (5, 1, 3, 6, 2, 4),
                                                     (2, 2, 1, 1, 0, 0), (8, 8, 1, 40, 1, 2), (6, 2, 4, 5, 5, 0)])
def test_choice_and_sparse_attention(hyq, HQ, HKV, n_q, k, first, last):
    lens = [0, 1, 64, 65, 700, 2300, 1024, 3]
    cache = make(HQ, HKV, 80, len(lens), 36)
    hist = History(len(lens), HKV)
    kk, vv, _, _ = grow(cache, list(range(len(lens))), lens, 11)
    hist.add(range(len(lens)), lens, kk, vv)
    order = [5, 2, 0, 4, 7, 1, 6, 3]
    q = queries(12, len(order), n_q, HQ)
    sel = torch.full((len(order), n_q, HKV, k), 1234, dtype=torch.int32, device="cuda")
    for _ in range(2):
        cache.select(0, q, sel, seqs=ints(order), n_first=first, n_last=last)
    check_choice(cache, q, sel, order, first, last)
    out = torch.full_like(q, float("nan"))
    cache.attention_blocks(0, q, sel, out, seqs=ints(order))
    assert hyq_read_device_error(cache.err()) == 0
    check_attention(cache, hist, q, out, order, sel=sel.cpu().tolist())


def test_choice_among_ties_takes_the_lower_blocks(hyq):
    cache = make(4, 1, 40, 1, 40)
    page = mixed_rows(3, (1, 64, 128)).transpose(0, 1)
    grow(cache, [0], [64 * 30], 0, rows=(page.repeat(30, 1, 1), page.repeat(30, 1, 1)))
    q = queries(4, 1, 1, 4)
    for k, first, last in ((5, 0, 0), (6, 1, 2), (29, 0, 1), (3, 0, 3), (30, 1, 1)):
        sel = torch.full((1, 1, 1, k), 77, dtype=torch.int32, device="cuda")
        cache.select(0, q, sel, n_first=first, n_last=last)
        assert sel.flatten().tolist() == list(range(k - last)) + list(range(30 - last, 30))


@pytest.mark.parametrize("nb", [8192, 8193, 20000])
def test_choice_among_many_blocks(hyq, nb):
    """Past what one block's shared memory holds, with few distinct scores (many ties)."""
    cache = make(2, 1, nb, 1, nb)
    cache.table()[0] = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    cache.lens()[0] = 64 * nb - 5
    rec = torch.zeros(nb, 272, dtype=torch.uint8)
    gen = torch.Generator().manual_seed(2)
    lo = torch.randint(-2, 2, (nb, 1), generator=gen)
    rec[:, :256] = lo.to(torch.int8).view(torch.uint8)
    rec[:, 128:129] = (lo + torch.randint(0, 4, (nb, 1), generator=gen)).to(torch.int8).view(torch.uint8)
    cache.bounds()[0, :, 0] = rec.cuda()
    q = queries(5, 1, 1, 2)
    for k in (1, 100, nb - 1):
        sel = torch.full((1, 1, 1, k), -9, dtype=torch.int32, device="cuda")
        cache.select(0, q, sel, n_first=1 if k > 1 else 0, n_last=0)
        check_choice(cache, q, sel, [0], 1 if k > 1 else 0, 0)


def test_choice_reports_queries_that_are_not_finite(hyq):
    cache = make(2, 2, 16, 1, 16)
    grow(cache, [0], [64 * 10], 1)
    q = queries(6, 1, 1, 2)
    sel = torch.full((1, 1, 2, 3), 50, dtype=torch.int32, device="cuda")
    ok = sel.clone()
    cache.select(0, q, ok, n_first=0, n_last=0)
    q[0, 0, 1, 7] = float("inf")
    cache.select(0, q, sel, n_first=0, n_last=0)
    assert hyq_read_device_error(cache.err()) == L.DEVERR_SCORE
    assert sel[0, 0, 1].tolist() == [0, 1, 2] and torch.equal(sel[0, 0, 0], ok[0, 0, 0])


def test_sparse_attention_over_given_lists(hyq):
    cache = make(4, 2, 16, 2, 8)
    k, v, _, _ = grow(cache, [0, 1], [450, 100], 2)
    hist = History(2, 2)
    hist.add([0, 1], [450, 100], k, v)
    q = queries(7, 2, 1, 4)
    sel = [[[[0, 3, 7], [7, -1, -1]]], [[[-1, -1, -1], [0, 1, -1]]]]      # one token and head reads nothing
    out = torch.full_like(q, float("nan"))
    cache.attention_blocks(0, q, torch.tensor(sel, dtype=torch.int32, device="cuda"), out)
    assert hyq_read_device_error(cache.err()) == 0
    check_attention(cache, hist, q, out, [0, 1], sel=sel)
    for bad in ([0, 0, 1], [3, 2, -1], [0, -1, 2], [0, 1, 8], [1, 2, 1 << 30]):
        x = torch.tensor(sel, dtype=torch.int32, device="cuda")
        x[0, 0, 0] = ints(bad)
        cache.attention_blocks(0, q, x, out)
        assert hyq_read_device_error(cache.err()) == L.DEVERR_INDEX, bad
        cache.err().zero_()
        check_attention(cache, hist, q[1:], out[1:], [1], sel=sel[1:])


# --- tables ------------------------------------------------------------------------------------------------------------

def check_tables(cache, t):
    assert cache.lens().tolist() == t.lens and cache.refs().tolist() == t.refs()
    table = cache.table().tolist()
    for s, row in enumerate(t.pages):
        assert table[s][:len(row)] == row, s


@pytest.mark.parametrize("seed", range(6))
def test_tables_follow_the_rules(hyq, seed):
    """Random calls, the invalid among them, against the plain tables; the copies of a reserve by content."""
    rng = np.random.default_rng(seed)
    n_pages, n_seqs, blocks, layers = 40, 10, 7, 2
    cache, t = make(2, 2, n_pages, n_seqs, blocks, n_layers=layers), P.Tables(n_pages, n_seqs, blocks)
    cache.pool().copy_(torch.randint(0, 256, cache.pool().shape, dtype=torch.uint8))
    cache.bounds().copy_(torch.randint(0, 256, cache.bounds().shape, dtype=torch.uint8))
    for step in range(60):
        what = rng.choice(["reserve", "reserve", "fork", "truncate", "compact"])
        pool, bounds = cache.pool().clone(), cache.bounds().clone()
        seqs = rng.integers(-1 if rng.random() < 0.05 else 0, n_seqs, rng.integers(1, 6)).tolist()
        if rng.random() < 0.8:
            seqs = list(dict.fromkeys(seqs))
        if what == "reserve":
            n = rng.integers(0, 150, len(seqs)).tolist()
            copies = t.reserve(seqs, n)
            cache.reserve(ints(seqs), ints(n))
            for a, b, tiles in copies or []:
                want = pool[:, b].clone()
                want[..., :2560 * tiles] = pool[:, a, :, :2560 * tiles]
                pool[:, b], bounds[:, b] = want, bounds[:, a]
            bad = copies is None
        elif what == "fork":
            dst = rng.integers(0, n_seqs, len(seqs)).tolist()
            bad = bool(t.fork(seqs, dst))
            cache.fork(ints(seqs), ints(dst))
        elif what == "truncate":
            n = [int(rng.integers(0, max(1, t.lens[s] + (2 if rng.random() < 0.1 else 0)))) if rng.random() < 0.7 else 0
                 for s in seqs]
            bad = bool(t.truncate(seqs, n))
            cache.truncate(ints(seqs), ints(n))
        else:
            for a, b in t.compact():
                pool[:, b], bounds[:, b] = pool[:, a].clone(), bounds[:, a].clone()
            cache.compact()
            bad = False
        assert (hyq_read_device_error(cache.err()) != 0) == bad, (step, what)
        cache.err().zero_()
        check_tables(cache, t)
        assert torch.equal(cache.pool(), pool) and torch.equal(cache.bounds(), bounds), (step, what)


def test_reserve_is_all_or_nothing(hyq):
    cache, t = make(2, 1, 10, 5, 4), P.Tables(10, 5, 4)
    for seqs, n, err in (([0, 1], [64, 100], 0), ([2, 3], [256, 256], L.DEVERR_PAGES), ([0, 2], [1, 257], L.DEVERR_PAGES),
                         ([0, 0], [1, 1], L.DEVERR_INDEX), ([0, 5], [1, 1], L.DEVERR_INDEX), ([0, 1], [1, -1], L.DEVERR_INDEX),
                         ([2, 3, 0], [256, 192, 0], 0), ([4], [1], L.DEVERR_PAGES), ([1], [28], 0), ([4], [0], 0)):
        assert (t.reserve(seqs, n) is None) == (err != 0)
        cache.reserve(ints(seqs), ints(n))
        assert hyq_read_device_error(cache.err()) == err
        cache.err().zero_()
        check_tables(cache, t)
    cache.truncate()                       # all of them
    assert not cache.refs().any() and not cache.lens().any()


def test_reserve_from_a_large_pool(hyq):
    """More pages than one pass of the scan looks at, free ones scattered, and a call that takes most of them."""
    n = 70000
    cfg = make_config(1, 1, 1, capacity=64)
    cache = PagedCache(cfg, n, 1024, 300)
    cache.reset()
    refs = torch.randint(0, 2, (n,), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    cache.refs().copy_(refs)
    free = torch.nonzero(refs == 0).flatten().tolist()
    rng = np.random.default_rng(2)
    counts = rng.integers(0, 64 * 60, 1024).tolist()
    cache.reserve(None, ints(counts))
    assert hyq_read_device_error(cache.err()) == 0
    at, table = 0, cache.table().cpu()
    for s, c in enumerate(counts):
        nb = -(-c // 64)
        assert table[s, :nb].tolist() == free[at:at + nb]
        at += nb
    assert at > 16384 and cache.refs().sum().item() == int(refs.sum()) + at
    lens = cache.lens().clone()
    cache.reserve(None, ints([64 * 100] * 1024))       # far more than there are
    assert hyq_read_device_error(cache.err()) == L.DEVERR_PAGES and torch.equal(cache.lens(), lens)


def test_compact_into_other_tables_keeps_the_old_ones_valid(hyq):
    cache = make(4, 2, 50, 6, 8)
    hist = History(6, 2)
    for s in range(6):
        k, v, _, _ = grow(cache, [s], [150 + 40 * s], s)
        hist.add([s], [150 + 40 * s], k, v)
    cache.truncate(ints([0, 2, 3]))
    q = queries(1, 3, 1, 4)
    live = [1, 4, 5]
    old_table, old_refs = cache.table().clone(), cache.refs().clone()
    to, refs = torch.full_like(old_table, -5), torch.full_like(old_refs, -5)
    cache.compact(to, refs)
    assert torch.equal(cache.table(), old_table) and torch.equal(cache.refs(), old_refs)
    n = int((old_refs > 0).sum())
    assert refs.tolist() == [1] * n + [0] * (50 - n)
    outs = []
    for table in (old_table, to):
        cache.table().copy_(table)
        out = torch.full_like(q, float("nan"))
        cache.attention(0, q, out, seqs=ints(live))
        check_attention(cache, hist, q, out, live)
        outs.append(out)
    assert torch.equal(*outs) and hyq_read_device_error(cache.err()) == 0


# --- together ----------------------------------------------------------------------------------------------------------

def test_serving_with_forks_drafts_and_compaction(hyq):
    """Prompts, shared prefixes, single tokens, drafted tokens some of which are taken back, freed and compacted sequences, two layers:
    attention and block choice always see exactly the rows that each sequence was given."""
    rng = np.random.default_rng(5)
    HQ, HKV, layers, n_seqs = 8, 2, 2, 8
    cache = make(HQ, HKV, 60, n_seqs, 10, n_layers=layers)
    hist = [History(n_seqs, HKV) for _ in range(layers)]

    def step(seqs, counts, one=False):
        cache.reserve(ints(seqs), None if one else ints(counts))
        for l in range(layers):
            k, v, _, _ = grow(cache, seqs, counts, int(rng.integers(1 << 30)), layer=l, one=one, reserve=False)
            hist[l].add(seqs, counts, k, v)

    def look(seqs, n_q):
        for l in range(layers):
            q = queries(int(rng.integers(1 << 30)), len(seqs), n_q, HQ)
            out = torch.full_like(q, float("nan"))
            cache.attention(l, q, out, seqs=ints(seqs))
            check_attention(cache, hist[l], q, out, seqs, layer=l)
            sel = torch.empty(len(seqs), n_q, HKV, 3, dtype=torch.int32, device="cuda")
            cache.select(l, q, sel, seqs=ints(seqs))
            cache.attention_blocks(l, q, sel, out, seqs=ints(seqs))
            check_attention(cache, hist[l], q, out, seqs, sel=sel.cpu().tolist(), layer=l)

    step([0, 1], [200, 70])
    cache.fork(ints([0, 0, 1, 0]), ints([2, 3, 4, 5]))
    for l in range(layers):
        for s, d in ((0, 2), (0, 3), (1, 4), (0, 5)):
            hist[l].k[d], hist[l].v[d] = hist[l].k[s], hist[l].v[s]
    for _ in range(3):
        step([3, 0, 2, 4, 1], [1] * 5, one=True)
        look([3, 0, 2, 4, 1, 5], 1)
    step([2, 3, 5], [4, 4, 4])
    look([2, 3, 5], 4)
    cut = [len(hist[0].k[2]) - 3, len(hist[0].k[3]), len(hist[0].k[5]) - 1]
    cache.truncate(ints([2, 3, 5]), ints(cut))
    for l in range(layers):
        for s, n in zip((2, 3, 5), cut):
            hist[l].k[s], hist[l].v[s] = hist[l].k[s][:n], hist[l].v[s][:n]
    step([2, 5], [2, 90])
    cache.truncate(ints([0, 4]))
    for l in range(layers):
        for s in (0, 4):
            hist[l].k[s], hist[l].v[s] = hist[l].k[s][:0], hist[l].v[s][:0]
    cache.compact()
    step([1, 2, 3, 5, 0], [1, 1, 1, 1, 30])
    look([1, 2, 3, 5, 0], 1)
    assert hyq_read_device_error(cache.err()) == 0


def test_a_captured_step_follows_the_growing_lengths(hyq):
    """One decode step of all sequences (reserve, append, attention, choice, sparse attention) captured once and
    replayed, on a stream of its own, equals the same steps made one by one."""
    HQ, HKV, n = 8, 2, 5
    caches, hist = [make(HQ, HKV, 40, n, 8) for _ in range(2)], History(n, HKV)
    lens = [60, 0, 127, 300, 5]
    rows = [mixed_rows(s, (HKV, sum(lens), 128)).transpose(0, 1).contiguous() for s in (1, 2)]
    for c in caches:
        grow(c, list(range(n)), lens, 0, rows=rows)
    hist.add(range(n), lens, *rows)
    static = {x: torch.zeros(n, HKV, 128, dtype=torch.bfloat16, device="cuda") for x in "kv"}
    q, out, sparse = (torch.zeros(n, 1, HQ, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    sel = torch.zeros(n, 1, HKV, 2, dtype=torch.int32, device="cuda")

    def step(c):
        c.reserve()
        c.append(0, static["k"], static["v"])
        c.attention(0, q, out)
        c.select(0, q, sel, n_first=0)
        c.attention_blocks(0, q, sel, sparse)

    cache = caches[0]
    for op in (L.OP_PAGED_ATTENTION, L.OP_PAGED_SELECT, L.OP_PAGES_RESERVE):
        cache.workspace(op, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(cache)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(8):
        k, v = (mixed_rows(20 + 2 * i + j, (n, HKV, 128)) for j in range(2))
        static["k"].copy_(k)
        static["v"].copy_(v)
        q.copy_(queries(i, n, 1, HQ))
        hist.add(range(n), [1] * n, k, v)
        graph.replay()
        got = [x.clone() for x in (out, sel, sparse)]
        check_attention(cache, hist, q, got[0], range(n))
        check_attention(cache, hist, q, got[2], range(n), sel=got[1].cpu().tolist())
        step(caches[1])
        assert all(torch.equal(a, b) for a, b in zip(got, (out, sel, sparse)))
    for c in caches:
        assert hyq_read_device_error(c.err()) == 0


def test_workspaces_serve_calls_of_any_smaller_size_in_turn(hyq):
    cache = make(8, 2, 200, 6, 40)
    lens = [2000, 10, 700, 0, 64, 130]
    k, v, _, _ = grow(cache, list(range(6)), lens, 3)
    hist = History(6, 2)
    hist.add(range(6), lens, k, v)
    for seqs, n_q in (([0, 1, 2, 3, 4, 5], 3), ([0], 1), ([2, 5], 2), ([0, 1, 2, 3, 4, 5], 3), ([1], 1)):
        q = queries(n_q, len(seqs), n_q, 8)
        out = torch.full_like(q, float("nan"))
        cache.attention(0, q, out, seqs=ints(seqs))
        check_attention(cache, hist, q, out, seqs)
        sel = torch.full((len(seqs), n_q, 2, 5), -7, dtype=torch.int32, device="cuda")
        cache.select(0, q, sel, seqs=ints(seqs))
        check_choice(cache, q, sel, seqs, 1, 1)


def test_refused_calls_raise_and_change_nothing(hyq):
    cache = make(4, 2, 8, 3, 4)
    grow(cache, [0], [10], 1)
    q = queries(1, 1, 1, 4)
    out = torch.full_like(q, 7.0)
    with pytest.raises(HyqError) as e:
        cache.attention(1, q, out, seqs=ints([0]))          # no such layer
    assert e.value.status == 1
    with pytest.raises(HyqError):
        cache.attention(0, queries(1, 4, 1, 4), torch.empty(4, 1, 4, 128, dtype=torch.bfloat16, device="cuda"))
    sel = torch.full((1, 1, 2, 2), 9, dtype=torch.int32, device="cuda")
    with pytest.raises(HyqError):
        cache.select(0, q, sel, seqs=ints([0]), n_first=2, n_last=1)
    with pytest.raises(ValueError):
        cache.attention(0, q.float(), out, seqs=ints([0]))
    with pytest.raises(ValueError):
        cache.attention(0, q, out, seqs=torch.zeros(1, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (sel == 9).all() and hyq_read_device_error(cache.err()) == 0


def test_calls_on_several_streams_at_once(hyq):
    """Appends into two layers, then attention and choice on both, from two streams at once (a PagedCache of its own
    over the same buffers for each, as their workspaces need), equal the same calls made in turn."""
    HQ, HKV, lens = 8, 2, [900, 64, 333]
    base = make(HQ, HKV, 40, 3, 16, n_layers=2)
    base.reserve(None, ints(lens))
    rows = [mixed_rows(s, (HKV, sum(lens), 128)).transpose(0, 1).contiguous().cuda() for s in range(4)]
    cu = ints(np.concatenate([[0], np.cumsum(lens)]).tolist())
    q = [queries(s, 3, 1, HQ) for s in (1, 2)]
    views = [PagedCache(base.cfg, 40, 3, 16, 2, buffers=base.buf) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for together in (False, True):
        base.pool().fill_(0xFF)
        base.bounds().fill_(0xFF)
        outs = [[torch.full_like(q[0], float("nan")), torch.zeros(3, 1, HKV, 4, dtype=torch.int32, device="cuda")]
                for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(3):
            for l in range(2):
                v, s = views[l], streams[l] if together else None
                v.append(l, rows[2 * l], rows[2 * l + 1], cu_rows=cu, stream=s)
                v.attention(l, q[l], outs[l][0], stream=s)
                v.select(l, q[l], outs[l][1], stream=s)
        torch.cuda.synchronize()
        results.append([base.pool()[:, base.table()[0, :14].long()].clone(), base.bounds()[:, base.table()[0, :14].long()].clone()]
                       + [x.clone() for o in outs for x in o])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    hist = History(3, HKV)
    hist.add(range(3), lens, rows[2], rows[3])
    check_attention(base, hist, q[1], results[1][4], range(3), layer=1)
    assert hyq_read_device_error(base.err()) == 0


def test_a_call_on_a_stream_of_its_own_follows_that_stream(hyq):
    """Work queued on the given stream before the call (here the rows' and queries' copies behind a long kernel) is seen by it,
    with the default stream idle."""
    cache = make(4, 2, 8, 2, 4)
    k, v = (mixed_rows(s, (2, 150, 128)).transpose(0, 1).contiguous() for s in (3, 4))
    hist = History(2, 2)
    hist.add([1], [150], k, v)
    kd, vd = (torch.zeros(150, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, out = (torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ks, vs, qs = k.cuda(), v.cuda(), queries(5, 1, 1, 4)
    big = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = big @ big * 1e-3
        kd.copy_(ks)
        vd.copy_(vs)
        q.copy_(qs)
    cache.reserve(ints([1]), ints([150]), stream=side)
    cache.append(0, kd, vd, seqs=ints([1]), cu_rows=ints([0, 150]), stream=side)
    cache.attention(0, q, out, seqs=ints([1]), stream=side)
    side.synchronize()
    check_attention(cache, hist, qs, out, [1])


@pytest.mark.parametrize("HKV", [1, 2, 4, 5, 8, 12])
def test_append_for_any_number_of_heads(hyq, HKV):
    counts, seqs = [70, 0, 200, 3, 64, 1], [5, 4, 3, 2, 1, 0]
    cache, hist = make(HKV, HKV, 24, 6, 8), History(6, HKV)
    for step in range(2):
        k, v, _, _ = grow(cache, seqs, counts, 7 * step + HKV)
        hist.add(seqs, counts, k, v)
    for s in range(6):
        for h in range(HKV):
            check_rows(cache, s, h, hist.k[s][:, h], hist.v[s][:, h])
            check_bounds(cache, s, h, hist.k[s][:, h])
    assert hyq_read_device_error(cache.err()) == 0


@pytest.mark.parametrize("one", [False, True])
def test_append_to_the_most_sequences(hyq, one):
    """1024 sequences in one call, a row each or none to two."""
    n = 1024
    cache, hist = make(2, 2, 1100, n, 3), History(n, 2)
    for step in range(2):
        counts = [1] * n if one else [(i + step) % 3 for i in range(n)]
        k, v, _, _ = grow(cache, list(range(n))[::-1], counts, step, one=one)
        hist.add(list(range(n))[::-1], counts, k, v)
    for s in (0, 1, 2, 511, 1022, 1023):
        if len(hist.k[s]):
            check_rows(cache, s, 1, hist.k[s][:, 1], hist.v[s][:, 1])
            check_bounds(cache, s, 1, hist.k[s][:, 1])
    q = queries(3, n, 1, 2)
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    check_attention(cache, hist, q, out, range(n))


@pytest.mark.parametrize("HQ,HKV,n_q", [(8, 1, 64), (5, 1, 13), (64, 8, 3)])
def test_many_query_tokens(hyq, HQ, HKV, n_q):
    """Up to the largest number of tokens: several passes of four query tiles, rows that end inside a tile."""
    lens = [40, 700, 64, n_q, n_q - 1]
    cache, hist = make(HQ, HKV, 24, 5, 12), History(5, HKV)
    k, v, _, _ = grow(cache, list(range(5)), lens, 2)
    hist.add(range(5), lens, k, v)
    q = queries(9, 5, n_q, HQ)
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    check_attention(cache, hist, q, out, range(5))


def test_queries_that_are_not_finite_stay_in_their_rows(hyq):
    """A NaN or infinite query gives NaN in its own output row; all others are as without it."""
    cache = make(8, 2, 8, 2, 4)
    grow(cache, [0, 1], [200, 100], 3)
    q = queries(4, 2, 2, 8)
    outs = []
    for bad in (False, True):
        if bad:
            q[0, 1, 3, 5], q[1, 0, 6, 100] = float("nan"), float("inf")
        out = torch.zeros_like(q)
        cache.attention(0, q, out)
        outs.append(out)
    hit = torch.zeros(2, 2, 8, dtype=torch.bool, device="cuda")
    hit[0, 1, 3] = hit[1, 0, 6] = True
    assert outs[1][hit].isnan().any(1).all()
    assert torch.equal(outs[0][~hit], outs[1][~hit])


def test_calls_captured_between_other_nodes(hyq):
    """A captured step whose calls follow copies, fills and joined branches of another stream (and are followed by such)
    replays to what the same calls give one by one."""
    cache = make(8, 2, 24, 3, 8)
    lens = [200, 64, 31]
    k, v, _, _ = grow(cache, [0, 1, 2], lens, 4)
    hist = History(3, 2)
    hist.add(range(3), lens, k, v)
    qs, q = queries(5, 3, 1, 8), torch.zeros(3, 1, 8, 128, dtype=torch.bfloat16, device="cuda")
    out, copy = (torch.zeros_like(q) for _ in range(2))
    other = PagedCache(cache.cfg, 24, 3, 8, buffers=cache.buf)
    out2, sel = torch.zeros_like(q), torch.zeros(3, 1, 2, 2, dtype=torch.int32, device="cuda")
    for c in (cache, other):
        for op in (L.OP_PAGED_ATTENTION, L.OP_PAGED_SELECT):
            c.workspace(op, 3)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        q.copy_(qs)
        out.fill_(float("nan"))
        cache.attention(0, q, out)              # after a fill
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other.select(0, q, sel)             # begins a branch
            other.attention_blocks(0, q, sel, out2)
        copy.copy_(out)
        cache.attention(0, q, out)              # after a kernel of another library, beside the branch
        torch.cuda.current_stream().wait_stream(side)
        cache.attention(0, q, out)              # after a join
        cache.truncate(ints([]))                # nothing
    for _ in range(3):
        q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_attention(cache, hist, qs, out, range(3))
        check_attention(cache, hist, qs, out2, range(3), sel=sel.cpu().tolist())
        assert torch.equal(copy, out)
    assert hyq_read_device_error(cache.err()) == 0


@pytest.mark.parametrize("bits", [(4, 4), (8, 8), (4, 8), (8, 4)])
def test_pages_hold_the_bytes_of_the_stream(hyq, bits):
    """The same rows appended to the fixed-batch stream and to pages give the same bytes: rows of many scales, offsets
    much larger than their range (codes that need the clamp), coarse grids with planted midpoints, few distinct values."""
    from hybrid_precision_quantized_gb300 import HybridLayer, hyq_quantize_append
    HKV, n = 4, 64 * 24
    gen = torch.Generator().manual_seed(bits[0] * 16 + bits[1])
    parts = []
    for scale in (1e-4, 0.03, 1.0, 20.0, 3000.0):
        x = torch.randn(2, HKV, 192, 128, generator=gen) * scale
        parts.append(x)
        parts.append(x * 0.01 + scale * 3 * torch.randn(2, HKV, 192, 4, 1, generator=gen).expand(-1, -1, -1, -1, 32).flatten(-2))
    rows = torch.cat(parts, 2)[:, :, : n - 192].to(torch.bfloat16)
    ties = torch.stack([tie_rows(7 + i, (HKV, 192, 128), bits[i]) for i in range(2)])
    k, v = torch.cat([rows, ties], 2).cuda()
    assert k.shape[1] == n
    layer = HybridLayer(make_config(1, HKV, HKV, capacity=n, window=0, bits_k=bits[0], bits_v=bits[1]))
    layer.reset()
    hyq_quantize_append(layer.cfg, k[None].contiguous(), v[None].contiguous(), n, layer.c)
    cache = make(HKV, HKV, n // 64, 1, n // 64, bits=bits)
    cache.reserve(ints([0]), ints([n]))
    cache.append(0, k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous(), cu_rows=ints([0, n]))
    assert hyq_read_device_error(layer.err()) == 0 and hyq_read_device_error(cache.err()) == 0
    pages = cache.pool()[0, cache.table()[0].long()]          # [blocks, HKV, bytes]
    assert torch.equal(pages.transpose(0, 1), layer.qblocks()[0])


# --- many query rows a KV head: from 25 to 32 on (wide codes; 4-bit: 57 to 64) fours of query tiles are taken together ----

WIDE = [(8, 1, (8, 8), 4), (5, 1, (4, 8), 5), (14, 2, (8, 4), 4), (16, 2, (8, 8), 8), (6, 3, (8, 4), 14), (8, 1, (4, 4), 4),
        (5, 1, (4, 4), 5), (8, 2, (4, 4), 4), (4, 1, (8, 8), 3), (8, 2, (4, 8), 4), (10, 2, (8, 4), 9), (8, 1, (4, 4), 6),
        (8, 1, (4, 4), 8), (7, 1, (4, 4), 9)]


@pytest.mark.parametrize("HQ,HKV,bits,n_q", WIDE)
def test_many_query_rows_over_ragged_lengths(hyq, HQ, HKV, bits, n_q):
    cache = make(HQ, HKV, 30, len(LENS), 6, bits=bits)
    hist = History(len(LENS), HKV)
    k, v, _, _ = grow(cache, list(range(len(LENS))), LENS, HQ + n_q)
    hist.add(range(len(LENS)), LENS, k, v)
    order = [7, 3, 9, 0, 1, 8, 2, 5, 6, 4, 9, 9]
    q = queries(HQ, len(order), n_q, HQ)
    outs = []
    for _ in range(2):
        out = torch.full_like(q, float("nan"))
        cache.attention(0, q, out, seqs=ints(order))
        outs.append(out)
    assert hyq_read_device_error(cache.err()) == 0
    print(f"error / bound: {check_attention(cache, hist, q, outs[0], order):.3f}")
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("B,HQ,HKV,bits,n,n_q", [(1, 8, 1, (8, 8), 20011, 4), (2, 7, 1, (8, 4), 9000, 4), (1, 5, 1, (4, 8), 7777, 6),
                                                    (1, 8, 1, (4, 4), 12345, 4), (1, 4, 1, (4, 4), 20011, 4),
                                                    (1, 3, 1, (8, 8), 15000, 5), (2, 6, 1, (4, 8), 5000, 7),
                                                    (1, 8, 1, (4, 4), 9000, 8)])
def test_many_query_rows_joined(hyq, B, HQ, HKV, bits, n, n_q):
    """Split over many blocks, whose partials (15 to 64 rows) are joined; the same bits every time."""
    nb = -(-n // 64)
    cache = make(HQ, HKV, B * nb, B, nb, bits=bits)
    k = torch.randn(n * B, HKV, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    v = torch.randn(n * B, HKV, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    grow(cache, list(range(B)), [n] * B, 0, rows=(k, v))
    hist = History(B, HKV)
    hist.add(range(B), [n] * B, k, v)
    q = queries(3, B, n_q, HQ)
    outs = []
    for _ in range(3):
        out = torch.full_like(q, float("nan"))
        cache.attention(0, q, out)
        outs.append(out)
    print(f"error / bound: {check_attention(cache, hist, q, outs[0], range(B)):.3f}")
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("bits,HQ,n_q", [((8, 8), 8, 4), ((4, 4), 8, 8), ((8, 8), 4, 4), ((4, 4), 4, 4)])
def test_many_query_rows_of_extreme_values(hyq, bits, HQ, n_q):
    """Peaked logits late in the sequence (the maximum moves), equal ones, zero queries, large and tiny values."""
    cache = make(HQ, 1, 25, 5, 5, bits=bits)     # 290 rows: five pages each
    n = 290
    base = torch.randn(n, 1, 128, generator=torch.Generator().manual_seed(8))
    ks = [base * 200, torch.ones(n, 1, 128), base, base * 1e-5, base]
    ks[0][240] *= 3
    vs = [base * 1000, base, base * 30000 / base.abs().max(), base * 1e-6, base]
    hist = History(5, 1)
    for s in range(5):
        k, v = ks[s].to(torch.bfloat16), vs[s].to(torch.bfloat16)
        grow(cache, [s], [n], 0, rows=(k, v))
        hist.add([s], [n], k, v)
    q = queries(9, 5, n_q, HQ)
    q[4] = 0
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    check_attention(cache, hist, q, out, range(5))


@pytest.mark.parametrize("bits,HQ,n_q", [((8, 8), 8, 4), ((4, 4), 8, 8), ((8, 8), 4, 4), ((4, 4), 4, 4)])
def test_many_query_rows_that_are_not_finite(hyq, bits, HQ, n_q):
    """A NaN or infinite query gives NaN in its own output row; all others are as without it."""
    cache = make(HQ, 1, 8, 2, 4, bits=bits)
    grow(cache, [0, 1], [200, 100], 3)
    q = queries(4, 2, n_q, HQ)
    outs = []
    for bad in (False, True):
        if bad:
            q[0, 1, 3, 5], q[1, 3, 2, 100] = float("nan"), float("inf")
        out = torch.zeros_like(q)
        cache.attention(0, q, out)
        outs.append(out)
    same = torch.ones(2, n_q, HQ, dtype=torch.bool, device="cuda")
    same[0, 1, 3] = same[1, 3, 2] = False
    assert torch.equal(outs[0][same], outs[1][same])
    assert outs[1][~same].isnan().any(1).all()


@pytest.mark.parametrize("bits,HQ,n_q", [((8, 8), 8, 4), ((4, 4), 8, 8), ((8, 8), 4, 4), ((4, 4), 4, 4)])
def test_many_query_rows_skip_pages_outside_the_pool(hyq, bits, HQ, n_q):
    """A table entry outside the pool counts as nothing to see and is reported; the other sequences are as before."""
    cache, hist = make(HQ, 1, 12, 2, 6, bits=bits), History(2, 1)
    k, v, _, _ = grow(cache, [0, 1], [300, 300], 3)
    hist.add([0, 1], [300, 300], k, v)
    q = queries(4, 2, n_q, HQ)
    cache.table()[0, 1], cache.table()[0, 3] = -5, 12
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    assert hyq_read_device_error(cache.err()) == L.DEVERR_INDEX
    sel = [[[np.array([0, 2, 4])]] * n_q, [[np.arange(5)]] * n_q]
    check_attention(cache, hist, q, out, [0, 1], sel=sel)


@pytest.mark.parametrize("bits,n_q", [((8, 8), 4), ((4, 4), 8)])
def test_many_query_rows_of_many_sequences(hyq, bits, n_q):
    """1024 sequences, most of them shorter than the tokens asked for or empty: rows that see nothing are zeros."""
    lens = [(5 * i) % 11 if i % 4 == 0 else 0 for i in range(1024)]
    lens[5], lens[700], lens[1023] = 130, 70, 65
    cache = make(8, 1, 300, 1024, 3, bits=bits)
    k, v, _, _ = grow(cache, list(range(1024)), lens, 5)
    hist = History(1024, 1)
    hist.add(range(1024), lens, k, v)
    q = queries(6, 1024, n_q, 8)
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    assert hyq_read_device_error(cache.err()) == 0
    check_attention(cache, hist, q, out, range(1024))
