"""Attention over the paged cache where its arithmetic is at its limits: values
of any size under few large probabilities, queries that are not finite."""
import numpy as np
import pytest
import torch

from hybrid_precision_quantized_gb300 import hyq_read_device_error
from oracle import paged as P
from oracle.quant import quantize
from tests.test_gpu_paged import History, check_attention, grow, ints, make, np64, queries

pytestmark = pytest.mark.gpu


# --- queries that are not finite ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("bits,HQ,n_q", [((4, 4), 8, 1), ((8, 8), 8, 1), ((8, 4), 8, 2), ((8, 8), 8, 4), ((4, 4), 8, 8)])
def test_short_sequences_keep_what_is_not_finite(hyq, bits, HQ, n_q):
    """A NaN or infinite query gives NaN in its own output row however short the sequence is, and zeros where it sees
    nothing; all other rows are as without it."""
    lens = [1, 10, 15, 16, 17, 31, 32, 33, 100]
    n = len(lens)
    cache, hist = make(HQ, 1, 16, n, 2, bits=bits), History(n, 1)
    k, v, _, _ = grow(cache, list(range(n)), lens, 3)
    hist.add(range(n), lens, k, v)
    q = queries(4, n, n_q, HQ)
    clean = torch.zeros_like(q)
    cache.attention(0, q, clean)
    check_attention(cache, hist, q, clean, range(n))
    for bad in (float("nan"), float("inf"), -float("inf")):
        x, out = q.clone(), torch.zeros_like(q)
        x[:, :, 3, 77] = bad
        cache.attention(0, x, out)
        for b in range(n):
            for i in range(n_q):
                if lens[b] - n_q + 1 + i > 0:
                    assert out[b, i, 3].isnan().all(), (b, i, bad)
                else:
                    assert not out[b, i].any(), (b, i, bad)
        rest = [h for h in range(HQ) if h != 3]
        assert torch.equal(out[:, :, rest], clean[:, :, rest])
    assert hyq_read_device_error(cache.err()) == 0


# --- values of any size ----------------------------------------------------------------------------------------------------

def sinks(bits, HQ, n_q, std, n_seqs, n=32768, every=None, nats=12.0, small=0.01):
    """n_seqs sequences that share one cache of n positions (so that each is worked on by one or two blocks), some of
    whose positions (one, or every so many) stand ``nats`` above the rest and have small values."""
    gen = torch.Generator().manual_seed(int(1e6 * std) + bits[1])
    u = torch.randn(128, generator=gen)
    k, v = 0.25 * torch.randn(n, 1, 128, generator=gen), std * torch.randn(n, 1, 128, generator=gen)
    at = [5003] if every is None else list(range(17, n - 100, every))
    k[at] += u * (nats * 128 ** 0.5 / float(u @ u))
    v[at] *= small
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    cache = make(HQ, 1, n // 64 + 1, n_seqs, n // 64, bits=bits)
    grow(cache, [0], [n], 0, rows=(k, v))
    cache.fork(ints([0] * (n_seqs - 1)), ints(list(range(1, n_seqs))))
    q = (u + 0.05 * torch.randn(1, n_q, HQ, 128, generator=gen)).to(torch.bfloat16).expand(n_seqs, -1, -1, -1).contiguous()
    kd, _, _ = P.dequantised(np64(k[:, 0]), bits[0])
    vd, _, _ = P.dequantised(np64(v[:, 0]), bits[1])
    want = np.zeros((n_q, HQ, 128))
    for i in range(n_q):
        vis = np.arange(n) < n - n_q + 1 + i
        for h in range(HQ):
            want[i, h] = P.attend(np64(q[0, i, h]), kd, vd, vis)
    return cache, q.cuda(), want


# Largest root mean square of the error against the output's own.  An output is a sum of terms p v with independent
# errors: p and p s are rounded to fp16 (uniform within 2^-11 of their size, 2^-11 / sqrt(3) = 0.0003 as root mean
# square; a term's parts |c s| and |z| are together at most 5 times |v| as root mean squares of normal rows: 0.0015
# each, 0.002 for both), and the sum to BF16 (uniform within 2^-8, 0.0023 for a significand of 1, 0.0016 on
# average): 0.0026 in all.  Logits are off by at most 2^-18 of their products' sizes, below 0.0003 here.
RMS = 0.004
SINKS = [((4, 4), s) for s in (1e4, 100.0, 1.0, 0.1, 0.05, 0.02, 0.005, 1e-3, 1e-4)] + \
        [((8, 8), s) for s in (1e4, 100.0, 1.0, 0.3, 0.1, 0.05, 0.02, 0.005, 1e-3)]


def off(got, want):
    got = np64(got)
    assert np.isfinite(got).all()
    return float(np.sqrt(((got - want) ** 2).mean() / (want ** 2).mean()))


@pytest.mark.parametrize("bits,std", SINKS)
@pytest.mark.parametrize("every,nats", [(None, 12.0), (1000, 10.0)])
def test_values_of_any_size_under_few_large_probabilities(hyq, bits, std, every, nats):
    cache, q, want = sinks(bits, 4, 1, std, 320, every=every, nats=nats)
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    worst = [off(out, want)]
    sel = torch.arange(512, dtype=torch.int32, device="cuda").expand(320, 1, 1, -1).contiguous()
    cache.attention_blocks(0, q, sel, out)
    worst.append(off(out, want))
    print(f"bits {bits} std {std}: {worst[0]:.5f} {worst[1]:.5f}")
    assert max(worst) < RMS
    assert hyq_read_device_error(cache.err()) == 0


@pytest.mark.parametrize("bits,HQ,n_q", [((8, 8), 8, 4), ((4, 8), 8, 4), ((8, 4), 8, 4), ((4, 4), 8, 8)])
@pytest.mark.parametrize("std", [1.0, 0.05, 0.005])
def test_values_of_any_size_for_many_query_rows(hyq, bits, HQ, n_q, std):
    cache, q, want = sinks(bits, HQ, n_q, std, 160, every=1000, nats=10.0)
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    print(f"bits {bits} std {std}: {off(out, want):.5f}")
    assert off(out, want) < RMS


@pytest.mark.parametrize("bits,HQ,n_q", [((4, 4), 4, 1), ((8, 8), 4, 1), ((4, 8), 4, 1), ((8, 8), 8, 4), ((4, 4), 8, 8)])
@pytest.mark.parametrize("rising", [True, False])
def test_values_whose_size_changes_along_the_sequence(hyq, bits, HQ, n_q, rising):
    """Standard deviations from 0.001 to 1000, the probabilities in inverse ratio: all rows count alike, so the factors that
    keep products in range move while there is something to lose."""
    n, n_seqs = 8192, 320 if n_q == 1 else 160
    gen = torch.Generator().manual_seed(7)
    u = torch.randn(128, generator=gen)
    x = torch.linspace(-6.9, 6.9, n)                    # log of the size
    x = x if rising else x.flip(0)
    k = 0.1 * torch.randn(n, 1, 128, generator=gen) - x[:, None, None] * u * (128 ** 0.5 / float(u @ u))
    v = torch.exp(x)[:, None, None] * torch.randn(n, 1, 128, generator=gen)
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    cache = make(HQ, 1, n // 64, n_seqs, n // 64, bits=bits)
    grow(cache, [0], [n], 0, rows=(k, v))
    cache.fork(ints([0] * (n_seqs - 1)), ints(list(range(1, n_seqs))))
    q = (u + 0.02 * torch.randn(1, n_q, HQ, 128, generator=gen)).to(torch.bfloat16).expand(n_seqs, -1, -1, -1).contiguous()
    kd, vd = (P.dequantised(np64(r[:, 0]), b)[0] for r, b in zip((k, v), bits))
    want = np.stack([[P.attend(np64(q[0, i, h]), kd, vd, np.arange(n) < n - n_q + 1 + i) for h in range(HQ)]
                     for i in range(n_q)])
    q, out = q.cuda(), torch.full((n_seqs, n_q, HQ, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    cache.attention(0, q, out)
    print(f"bits {bits} rising {rising}: {off(out, want):.5f}")
    assert off(out, want) < RMS


def check_bound(cache, hist, q, out, seqs):
    """Elementwise, within attend_bound."""
    hkv, bits = cache.cfg.num_kv_heads, (cache.cfg.bits_k, cache.cfg.bits_v)
    g, qn, on, worst = cache.cfg.num_q_heads // hkv, np64(q), np64(out), 0.0
    assert np.isfinite(on).all()
    for b, s in enumerate(seqs):
        n = len(hist.k[s])
        if n == 0:
            assert not on[b].any()
            continue
        for h in range(hkv):
            kd, kp, _ = P.dequantised(hist.k[s][:, h], bits[0])
            vd, vp, vc = P.dequantised(hist.v[s][:, h], bits[1])
            vs = quantize(hist.v[s][:, h], bits[1])[1]
            for i in range(q.shape[1]):
                vis = np.arange(n) < n - q.shape[1] + 1 + i
                for r in range(h * g, h * g + g):
                    if not vis.any():
                        assert not on[b, i, r].any()
                        continue
                    want = P.attend(qn[b, i, r], kd, vd, vis)
                    tol = P.attend_bound(qn[b, i, r], kd, kp, vp, vc, vs, vis, want)
                    err = np.abs(on[b, i, r] - want)
                    assert (err <= tol).all(), (b, i, r, float((err / np.maximum(tol, 1e-300)).max()))
                    worst = max(worst, float((err / np.maximum(tol, 1e-300)).max()))
    return worst


@pytest.mark.parametrize("bits,HQ,n_q", [((4, 4), 2, 1), ((8, 8), 2, 1), ((8, 4), 2, 3), ((8, 8), 8, 4), ((4, 8), 8, 4),
                                         ((4, 4), 8, 8)])
def test_values_of_any_size_within_a_bound_that_shrinks_with_them(hyq, bits, HQ, n_q):
    """Peaked logits late in the sequence, equal ones, zero queries; values from 1e-6 to 30000, and groups of unlike sizes."""
    n = 290
    gen = torch.Generator().manual_seed(8)
    base = torch.randn(n, 1, 128, generator=gen)
    unlike = torch.tensor([1e-5, 30.0, 0.01, 3000.0]).repeat_interleave(32)
    ks = [base * 200, torch.ones(n, 1, 128), base, base * 1e-5, base, base, base]
    ks[0][240] *= 3
    vs = [base * 1000, base * 1e-3, base * 30000 / base.abs().max(), base * 1e-6, base * 0.02, base * 1e-4,
          base * unlike]
    m = len(ks)
    cache, hist = make(HQ, 1, 5 * m, m, 5, bits=bits), History(m, 1)
    for s in range(m):
        k, v = ks[s].to(torch.bfloat16), vs[s].to(torch.bfloat16)
        grow(cache, [s], [n], 0, rows=(k, v))
        hist.add([s], [n], k, v)
    q = queries(9, m, n_q, HQ)
    q[4] = 0
    out = torch.full_like(q, float("nan"))
    cache.attention(0, q, out)
    assert hyq_read_device_error(cache.err()) == 0
    print(f"bits {bits} n_q {n_q} error / bound: {check_bound(cache, hist, q, out, range(m)):.3f}")


@pytest.mark.parametrize("bits,HQ,n_q", [((4, 4), 2, 1), ((8, 8), 2, 1), ((8, 4), 8, 4), ((4, 4), 8, 8)])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** 118, 2.0 ** 121, 2.0 ** -100, 2.0 ** -130])
def test_queries_of_any_size(hyq, bits, HQ, n_q, size):
    """Up to where logits leave float32 (one row takes all, and it has to be the right one) and down to nothing (all rows
    count alike)."""
    n = 200
    cache, hist = make(HQ, 1, 4, 1, 4, bits=bits), History(1, 1)
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn(n, 1, 128, generator=gen).to(torch.bfloat16) for _ in range(2))
    grow(cache, [0], [n], 0, rows=(k, v))
    hist.add([0], [n], k, v)
    q = (torch.randn(1, n_q, HQ, 128, generator=gen).to(torch.bfloat16).double() * size).to(torch.bfloat16)
    out = torch.full((1, n_q, HQ, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    cache.attention(0, q.cuda(), out)
    kd, kp, _ = P.dequantised(hist.k[0][:, 0], bits[0])
    vd, vp, _ = P.dequantised(hist.v[0][:, 0], bits[1])
    for i in range(n_q):
        vis = np.arange(n) < n - n_q + 1 + i
        for h in range(HQ):
            x = kd[vis] @ np64(q[0, i, h])
            if size > 1:     # the next row is far below, for logits off by 2^-18 of their products' sizes
                second, first = np.sort(x)[-2:]
                assert first - second > 2.0 ** -14 * (kp[vis] @ np.abs(np64(q[0, i, h]))).max()
                want, mean = vd[vis][x.argmax()], vp[vis][x.argmax()]
            else:
                want, mean = vd[vis].mean(0), vp[vis].mean(0)
            assert (np.abs(np64(out[0, i, h]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mean).all(), (i, h)
    assert hyq_read_device_error(cache.err()) == 0


@pytest.mark.parametrize("HQ,HKV,bits,n_q", [(8, 1, (8, 8), 7), (7, 1, (8, 4), 8), (16, 2, (4, 8), 11), (5, 1, (8, 8), 11),
                                             (8, 1, (8, 8), 3), (8, 1, (8, 8), 6), (8, 1, (4, 4), 7), (3, 1, (4, 8), 64)])
def test_query_rows_that_end_early_in_a_four_of_tiles(hyq, HQ, HKV, bits, n_q):
    """Three, six, seven and eleven tiles of query rows, the last of them filled or not, over ragged lengths and a long one."""
    lens = [0, 1, 3, n_q - 1, n_q, 63, 65, 300, 9000]
    m = len(lens)
    cache, hist = make(HQ, HKV, 170, m, 150, bits=bits), History(m, HKV)
    k, v, _, _ = grow(cache, list(range(m)), lens, HQ + n_q)
    hist.add(range(m), lens, k, v)
    q = queries(HQ, m, n_q, HQ)
    outs = []
    for _ in range(2):
        out = torch.full_like(q, float("nan"))
        cache.attention(0, q, out)
        outs.append(out)
    assert torch.equal(*outs) and hyq_read_device_error(cache.err()) == 0
    check_bound(cache, hist, q, outs[0], range(m))
