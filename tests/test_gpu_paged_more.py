"""GPU parity of shared prefixes, cross attention, accumulated weights and eviction: attention within bounds counted from
its roundings, weights likewise, evicted pages byte for byte."""
import numpy as np
import pytest
import torch

from hybrid_precision_quantized_gb300 import HyqError, hyq_read_device_error, pack_qblocks, unpack_qblocks
from hybrid_precision_quantized_gb300 import _lib as L
from oracle import paged as P
from tests.test_gpu_paged import History, grow, ints, make, np64, queries

pytestmark = pytest.mark.gpu

HEADS = [(4, 4), (8, 2), (8, 1), (10, 2)]
BITS = [(4, 4), (8, 8), (8, 4), (4, 8)]


def err(cache):
    e = hyq_read_device_error(cache.err())
    cache.err().zero_()
    return e


def held(cache, hist, s, h):
    """Keys, their |c s| + |z|, values, likewise, and value codes of a sequence's rows as they are held."""
    kd, kp, _ = P.dequantised(hist.k[s][:, h], cache.cfg.bits_k)
    vd, vp, vc = P.dequantised(hist.v[s][:, h], cache.cfg.bits_v)
    return kd, kp, vd, vp, vc


def filled(HQ, HKV, lens, bits=(4, 4), seed=1, n_layers=1, spare=3):
    nb = [-(-n // 64) for n in lens]
    cache = make(HQ, HKV, sum(nb) + spare, len(lens), max(max(nb), 1) + 2, n_layers, bits=bits)
    hist = History(len(lens), HKV)
    seqs = [i for i, n in enumerate(lens) if n]
    counts = [lens[i] for i in seqs]
    if seqs:
        k, v, _, _ = grow(cache, seqs, counts, seed)
        hist.add(seqs, counts, k, v)
    return cache, hist


def check_cross(cache, hist, q, out, seqs, toks, far=0):
    hkv, g = cache.cfg.num_kv_heads, cache.cfg.num_q_heads // cache.cfg.num_kv_heads
    qn, on, at, worst = np64(q), np64(out), 0, 0.0
    assert np.isfinite(on).all()
    for s, t in zip(seqs, toks):
        for h in range(hkv):
            if t and len(hist.k[s]):
                kd, _, vd, _, _ = held(cache, hist, s, h)
                vis = np.ones(len(kd), bool)
            for i in range(at, at + t):
                for r in range(h * g, h * g + g):
                    if not len(hist.k[s]):
                        assert not on[i, r].any()
                        continue
                    want = P.attend(qn[i, r], kd, vd, vis)
                    tol = P.span_error(qn[i, r], kd, vd, vis, want, far)
                    e = np.abs(on[i, r] - want)
                    worst = max(worst, float((e / tol).max()))
                    assert (e <= tol).all(), (s, i, r, worst)
        at += t
    return worst


def tokens(seed, n, hq, scale=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(n, hq, 128, generator=gen) * scale).to(torch.bfloat16).cuda()


def cu(counts):
    return ints(np.concatenate([[0], np.cumsum(counts)]).tolist())


# --- cross attention -----------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("HQ, HKV", HEADS)
@pytest.mark.parametrize("bits", BITS)
def test_cross_attention_over_ragged_lengths_and_tokens(hyq, HQ, HKV, bits):
    lens = [300, 1, 0, 63, 64, 65, 127, 128, 129]
    toks = [7, 1, 3, 33, 0, 2, 17, 40, 5]
    cache, hist = filled(HQ, HKV, lens, bits)
    order = [3, 0, 8, 1, 2, 4, 7, 5, 6]
    t = [toks[s] for s in order]
    q = tokens(3, sum(t), HQ)
    out = torch.full_like(q, float("nan"))
    cache.cross_attention(0, q, out, seqs=ints(order), cu_q=cu(t))
    assert err(cache) == 0
    check_cross(cache, hist, q, out, order, t)
    again = torch.full_like(q, float("nan"))
    cache.cross_attention(0, q, again, seqs=ints(order), cu_q=cu(t))
    assert torch.equal(out, again)


@pytest.mark.parametrize("n, t, HQ, HKV", [(1000, 300, 8, 2), (4100, 33, 8, 1), (20000, 3, 2, 2), (129, 700, 4, 4), (1, 1, 1, 1)])
def test_cross_attention_of_many_tokens_or_positions(hyq, n, t, HQ, HKV):
    """Many tiles of query rows; runs that several blocks share."""
    cache, hist = filled(HQ, HKV, [n, 70])
    q = tokens(5, t + 2, HQ)
    out = torch.empty_like(q)
    cache.cross_attention(0, q, out, cu_q=cu([t, 2]))
    assert err(cache) == 0
    pick = sorted(set([0, 1, t // 2, t - 1]) & set(range(t)))
    for h in range(HKV):
        kd, _, vd, _, _ = held(cache, hist, 0, h)
        vis = np.ones(n, bool)
        for i in pick:
            for r in range(h * (HQ // HKV), (h + 1) * (HQ // HKV)):
                want = P.attend(np64(q[i, r]), kd, vd, vis)
                assert (np.abs(np64(out[i, r]) - want) <= P.span_error(np64(q[i, r]), kd, vd, vis, want)).all()


def test_cross_attention_of_a_token_each_is_attention_of_the_last_position(hyq):
    cache, _ = filled(8, 2, [300, 1, 0, 64, 129])
    q = queries(4, 5, 1, 8)
    want, out = torch.empty_like(q), torch.empty_like(q)
    cache.attention(0, q, want)
    cache.cross_attention(0, q[:, 0], out[:, 0])
    assert torch.equal(out, want) and err(cache) == 0


def test_cross_attention_writes_its_tokens_alone(hyq):
    """Tokens before the first and behind the last sequence's stay; sequences may repeat; rows may lie in a wider tensor."""
    cache, hist = filled(8, 2, [200, 90])
    wide = torch.full((20, 24, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:16] = tokens(6, 20, 8)
    q = wide[:, 8:16]
    out = torch.full((20, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    cache.cross_attention(0, q, out, seqs=ints([1, 0, 1]), cu_q=ints([3, 8, 9, 16]))
    assert err(cache) == 0
    assert (out[:3] == 5).all() and (out[16:] == 5).all()
    check_cross(cache, hist, q[3:16], out[3:16], [1, 0, 1], [5, 1, 7])


def test_cross_attention_reports_what_it_leaves_out(hyq):
    cache, hist = filled(4, 2, [200, 90, 64])
    q = tokens(7, 12, 4)
    out = torch.full_like(q, 5.0)
    cache.cross_attention(0, q, out, seqs=ints([0, 9, 1]), cu_q=ints([0, 4, 8, 12]))      # no such sequence
    assert err(cache) == L.DEVERR_INDEX
    assert not out[4:8].any()
    check_cross(cache, hist, torch.cat([q[:4], q[8:]]), torch.cat([out[:4], out[8:]]), [0, 1], [4, 4])
    for pairs, good in (([0, 4, 3, 12], [(0, 0, 3)]), ([0, 4, 40, 41], [(0, 0, 4)]), ([-3, 4, 8, 12], [(1, 4, 8), (2, 8, 12)])):
        out = torch.full_like(q, 5.0)
        cache.cross_attention(0, q, out, cu_q=ints(pairs))
        assert err(cache) == L.DEVERR_INDEX
        for s, a, b in good:
            check_cross(cache, hist, q[a:b], out[a:b], [s], [b - a])
    cache.table()[1, 1] = 10 ** 6             # a page outside the pool: its positions are not seen
    out = torch.full_like(q, 5.0)
    cache.cross_attention(0, q, out, cu_q=ints([0, 4, 8, 12]))
    assert err(cache) == L.DEVERR_INDEX
    hist.k[1], hist.v[1] = hist.k[1][:64], hist.v[1][:64]
    check_cross(cache, hist, q, out, [0, 1, 2], [4, 4, 4])
    cache.table()[1, 0] = -7                  # none is left
    cache.cross_attention(0, q, out, cu_q=ints([0, 4, 8, 12]))
    assert err(cache) == L.DEVERR_INDEX and not out[4:8].any()


@pytest.mark.parametrize("HQ, t", [(2, 3), (8, 40)])
def test_cross_attention_of_queries_that_are_not_finite(hyq, HQ, t):
    cache, _ = filled(HQ, 2, [333])
    q = tokens(8, t, HQ)
    want = torch.empty_like(q)
    cache.cross_attention(0, q, want, cu_q=ints([0, t]))
    bad = q.clone()
    bad[0, 0, 5], bad[1, 1, 0], bad[t - 1, HQ - 1, 127] = float("nan"), float("inf"), float("-inf")
    out = torch.empty_like(q)
    cache.cross_attention(0, bad, out, cu_q=ints([0, t]))
    rows = [(0, 0), (1, 1), (t - 1, HQ - 1)]
    for i in range(t):
        for r in range(HQ):
            if (i, r) in rows:
                assert out[i, r].isnan().all()
            else:
                assert torch.equal(out[i, r], want[i, r])
    assert err(cache) == 0


@pytest.mark.parametrize("bits", [(4, 4), (8, 8)])
@pytest.mark.parametrize("kscale, vscale, qscale", [(1e-3, 1e-3, 1e3), (1e-6, 1e-7, 1.0), (1.0, 2e4, 1.0), (200.0, 1.0, 1e-2),
                                                    (1e-2, 1.0, 1e30), (1.0, 1.0, 1e-38), (2e4, 1.0, 1e-4)])
def test_cross_attention_of_extreme_values(hyq, bits, kscale, vscale, qscale):
    cache = make(4, 2, 8, 1, 6, bits=bits)
    hist = History(1, 2)
    gen = torch.Generator().manual_seed(3)
    # (a group's minimum has to be an fp16 value: append reports others)
    k, v = ((torch.randn(200, 2, 128, generator=gen) * s).clamp(min=-6e4).to(torch.bfloat16) for s in (kscale, vscale))
    grow(cache, [0], [200], 1, rows=(k, v))
    hist.add([0], [200], k, v)
    q = tokens(9, 9, 4, qscale)
    out = torch.empty_like(q)
    cache.cross_attention(0, q, out, cu_q=ints([0, 9]))
    assert err(cache) == 0
    check_cross(cache, hist, q, out, [0], [9])


@pytest.mark.parametrize("bits, far", [((4, 4), 5), ((8, 8), 9)])
@pytest.mark.parametrize("late", [False, True])
def test_cross_attention_of_values_beyond_fp16(hyq, bits, far, late):
    """c s + z past 65504: groups whose span is a multiple of the largest fp16, in the first pages or in the last alone."""
    cache = make(4, 2, 8, 1, 6, bits=bits)
    hist = History(1, 2)
    gen = torch.Generator().manual_seed(4)
    k, v = (torch.randn(300, 2, 128, generator=gen).to(torch.bfloat16) for _ in range(2))
    at = slice(260, 290) if late else slice(10, 50)
    v[at, :, 32:64] = (torch.rand(v[at, :, 32:64].shape, generator=gen) * 6e5 - 5e4).to(torch.bfloat16)
    k[at, :, :32] = (torch.rand(k[at, :, :32].shape, generator=gen) * 4e5).to(torch.bfloat16)
    grow(cache, [0], [300], 1, rows=(k, v))
    hist.add([0], [300], k, v)
    q = tokens(10, 9, 4)
    q[..., :32] *= 1e-5
    out = torch.empty_like(q)
    cache.cross_attention(0, q, out, cu_q=ints([0, 9]))
    assert err(cache) == 0
    check_cross(cache, hist, q, out, [0], [9], far)


def test_cross_attention_to_the_most_sequences(hyq):
    n = 1024
    cache, hist = filled(2, 1, [1 + i % 70 for i in range(n)], spare=0)
    toks = [i % 3 for i in range(n)]
    q = tokens(11, sum(toks), 2)
    out = torch.full_like(q, float("nan"))
    cache.cross_attention(0, q, out, cu_q=cu(toks))
    assert err(cache) == 0
    check_cross(cache, hist, q, out, list(range(n)), toks)


# --- shared prefixes -----------------------------------------------------------------------------------------------------

def branches(HQ, HKV, prompts, tails, bits=(4, 4), seed=1):
    """Prompts of whole pages, each forked into branches that grow by tails[i]: the cache, the history and the branches'
    sequences by prompt."""
    n = len(prompts) + sum(len(t) for t in tails)
    pages = sum(p // 64 + sum(x // 64 + 2 for x in t) for p, t in zip(prompts, tails))
    cache = make(HQ, HKV, pages + 2, n, max(p + max(t, default=0) for p, t in zip(prompts, tails)) // 64 + 2, bits=bits)
    hist = History(n, HKV)
    own = [i for i, p in enumerate(prompts) if p]
    if own:
        k, v, _, _ = grow(cache, own, [prompts[i] for i in own], seed)
        hist.add(own, [prompts[i] for i in own], k, v)
    at, groups, src, dst, counts = len(prompts), [], [], [], []
    for i, t in enumerate(tails):
        groups.append(list(range(at, at + len(t))))
        src += [i] * len(t)
        dst += groups[-1]
        counts += t
        at += len(t)
    cache.fork(ints(src), ints(dst))
    for s, d in zip(src, dst):
        hist.k[d], hist.v[d] = hist.k[s], hist.v[s]
    k, v, _, _ = grow(cache, dst, counts, seed + 7)
    hist.add(dst, counts, k, v)
    return cache, hist, groups


def check_shared(cache, hist, q, out, seqs):
    hkv, g, nq = cache.cfg.num_kv_heads, cache.cfg.num_q_heads // cache.cfg.num_kv_heads, q.shape[1]
    qn, on = np64(q), np64(out)
    assert np.isfinite(on).all()
    for b, s in enumerate(seqs):
        n = len(hist.k[s])
        for h in range(hkv):
            if n:
                kd, kp, vd, vp, vc = held(cache, hist, s, h)
            for i in range(nq):
                lim = n - nq + 1 + i
                for r in range(h * g, h * g + g):
                    if lim <= 0:
                        assert not on[b, i, r].any()
                        continue
                    vis = np.arange(n) < lim
                    want = P.attend(qn[b, i, r], kd, vd, vis)
                    tol = P.span_error(qn[b, i, r], kd, vd, vis, want, 0, kp, vp, vc)
                    e = np.abs(on[b, i, r] - want)
                    assert (e <= tol).all(), (b, s, i, r, float((e / tol).max()))


@pytest.mark.parametrize("HQ, HKV", HEADS)
@pytest.mark.parametrize("bits, n_q", [((4, 4), 1), ((4, 4), 3), ((8, 8), 5), ((8, 4), 1), ((4, 8), 2)])
def test_shared_prefixes_of_ragged_groups(hyq, HQ, HKV, bits, n_q):
    prompts, tails = [256, 64, 0, 448], [[5, 70, 1 + n_q], [64 + n_q], [9, 130], [5, 6, 7, 8, 9, 10, 11]]
    cache, hist, groups = branches(HQ, HKV, prompts, tails, bits)
    order = [3, 0, 2, 1]
    seqs = [s for i in order for s in groups[i]]
    q = queries(2, len(seqs), n_q, HQ)
    out = torch.full_like(q, float("nan"))
    sizes, shared = [len(groups[i]) for i in order], [prompts[i] for i in order]
    cache.attention_shared(0, q, out, cu(sizes), ints(shared), seqs=ints(seqs))
    assert err(cache) == 0
    check_shared(cache, hist, q, out, seqs)
    again = torch.full_like(q, float("nan"))
    cache.attention_shared(0, q, again, cu(sizes), ints(shared), seqs=ints(seqs))
    assert torch.equal(out, again)
    # sharing less than there is, or nothing
    for less in ([64, 0, 0, 64], [0, 0, 0, 0]):
        cache.attention_shared(0, q, out, cu(sizes), ints(less), seqs=ints(seqs))
        assert err(cache) == 0
        check_shared(cache, hist, q, out, seqs)


@pytest.mark.parametrize("HQ, HKV, n_q, branch, prompt", [(8, 1, 2, 40, 2048), (4, 4, 1, 200, 640), (32, 8, 1, 9, 6400), (8, 2, 64, 3, 192)])
def test_shared_prefixes_of_many_rows(hyq, HQ, HKV, n_q, branch, prompt):
    tails = [[n_q + (5 * i) % 67 for i in range(branch)]]
    cache, hist, groups = branches(HQ, HKV, [prompt], tails)
    seqs = groups[0]
    q = queries(3, branch, n_q, HQ)
    out = torch.full_like(q, float("nan"))
    cache.attention_shared(0, q, out, ints([0, branch]), ints([prompt]), seqs=ints(seqs))
    assert err(cache) == 0
    pick = [0, 1, branch // 2, branch - 1]
    check_shared(cache, hist, q[pick], out[pick], [seqs[i] for i in pick])


def test_shared_prefix_with_nothing_behind_it(hyq):
    """A branch that has only the shared positions so far."""
    cache, hist, groups = branches(4, 2, [128], [[3, 4]])
    cache.truncate(ints([groups[0][0]]), ints([128]))
    hist.k[groups[0][0]], hist.v[groups[0][0]] = hist.k[groups[0][0]][:128], hist.v[groups[0][0]][:128]
    q = queries(4, 2, 1, 4)
    out = torch.full_like(q, float("nan"))
    cache.attention_shared(0, q, out, ints([0, 2]), ints([128]), seqs=ints(groups[0]))
    assert err(cache) == 0
    check_shared(cache, hist, q, out, groups[0])


def test_what_cannot_be_shared_is_read_by_each_row(hyq):
    cache, hist, groups = branches(4, 2, [192, 128], [[5, 70, 3], [9, 4]])
    seqs = groups[0] + groups[1]
    q = queries(5, 5, 2, 4)
    out = torch.full_like(q, float("nan"))
    for c, n in (([0, 3, 5], [100, 128]), ([0, 3, 5], [256, 128]), ([0, 3, 5], [-64, 128]), ([0, 3, 4], [192, 0]),
                 ([1, 3, 5], [192, 128]), ([0, 4, 3, 5], [64, 64, 128]), ([0, 3, 9], [192, 128]), ([0, 3, 5], [192, 64 * 1000])):
        cache.attention_shared(0, q, out.fill_(float("nan")), ints(c), ints(n), seqs=ints(seqs))
        assert err(cache) == L.DEVERR_INDEX, (c, n)
        if c == [0, 4, 3, 5]:       # (row 3 would take the first group's pages)
            check_shared(cache, hist, q[:3], out[:3], seqs[:3])
        else:
            check_shared(cache, hist, q, out, seqs)
    # a row that is too short for the group's positions
    cache.truncate(ints([groups[0][1]]), ints([150]))
    hist.k[groups[0][1]], hist.v[groups[0][1]] = hist.k[groups[0][1]][:150], hist.v[groups[0][1]][:150]
    cache.attention_shared(0, q, out.fill_(float("nan")), ints([0, 3, 5]), ints([192, 128]), seqs=ints(seqs))
    assert err(cache) == L.DEVERR_INDEX
    check_shared(cache, hist, q, out, seqs)
    # a sequence that is not there
    seqs[4] = 99
    cache.attention_shared(0, q, out.fill_(float("nan")), ints([0, 3, 5]), ints([128, 128]), seqs=ints(seqs))
    assert err(cache) == L.DEVERR_INDEX and not out[4].any()
    check_shared(cache, hist, q[:4], out[:4], seqs[:4])


def test_shared_prefix_of_queries_that_are_not_finite(hyq):
    cache, _, groups = branches(8, 2, [256], [[5, 70, 3]])
    q = queries(6, 3, 2, 8)
    want, out = torch.empty_like(q), torch.empty_like(q)
    args = ints([0, 3]), ints([256])
    cache.attention_shared(0, q, want, *args, seqs=ints(groups[0]))
    bad = q.clone()
    bad[0, 1, 3, 9], bad[2, 0, 7, 0] = float("nan"), float("inf")
    cache.attention_shared(0, bad, out, *args, seqs=ints(groups[0]))
    assert out[0, 1, 3].isnan().all() and out[2, 0, 7].isnan().all()
    out[0, 1, 3], out[2, 0, 7] = want[0, 1, 3], want[2, 0, 7]
    assert torch.equal(out, want) and err(cache) == 0


def test_workspaces_of_shared_prefixes_serve_calls_of_any_smaller_size(hyq):
    cache, hist, groups = branches(8, 2, [256], [[3 + i for i in range(30)]])
    seqs = groups[0]
    cache.workspace(L.OP_PAGED_SHARED, 30, 4)
    for n, nq in ((30, 4), (2, 1), (30, 1), (7, 3), (30, 4), (1, 1)):
        q = queries(n + nq, n, nq, 8)
        out = torch.full_like(q, float("nan"))
        cache.attention_shared(0, q, out, ints([0, n]), ints([256 if nq < 3 else 192]), seqs=ints(seqs[:n]))
        assert err(cache) == 0
        check_shared(cache, hist, q[:2], out[:2], seqs[:min(n, 2)])


# --- logarithms of softmax sums, accumulated weights --------------------------------------------------------------------

def lse_of(q, kd, kp, lim):
    """The logarithm in 64 bits and how far float32 may be off."""
    x = (kd[:lim] @ q) / 128 ** 0.5
    size = (kp[:lim] @ np.abs(q)).max() / 128 ** 0.5
    want = x.max() + np.log(np.exp(x - x.max()).sum())
    return want, 2.0 ** -18 * (size + 1) + 2.0 ** -22 * abs(want)


@pytest.mark.parametrize("HQ, HKV, n_q, bits", [(4, 4, 1, (4, 4)), (8, 1, 3, (8, 8)), (10, 2, 2, (8, 4)), (8, 1, 4, (8, 8)),
                                               (8, 1, 8, (4, 4))])
def test_attention_gives_the_logarithms_of_its_sums(hyq, HQ, HKV, n_q, bits):
    lens = [300, 1, 0, 64, 129, 5000]
    cache, hist = filled(HQ, HKV, lens, bits)
    q = queries(7, len(lens), n_q, HQ)
    want, out = torch.empty_like(q), torch.empty_like(q)
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    cache.attention(0, q, want)
    cache.attention(0, q, out, lse=lse)
    assert torch.equal(out, want) and err(cache) == 0
    g = HQ // HKV
    for b, n in enumerate(lens):
        for h in range(HKV):
            if n:
                kd, kp, _, _, _ = held(cache, hist, b, h)
            for i in range(n_q):
                for r in range(h * g, h * g + g):
                    lim, got = n - n_q + 1 + i, float(lse[b, i, r])
                    if lim <= 0:
                        assert got == -np.inf
                    else:
                        e, tol = lse_of(np64(q[b, i, r]), kd, kp, lim)
                        assert abs(got - e) <= tol, (b, i, r, got, e, tol)


def mass_tensor(cache, fill=float("nan")):
    return torch.full(cache.mass_shape, fill, device="cuda")


def mass_of(cache, mass, s, h, layer=0):
    n = int(cache.lens()[s])
    pages = cache.table()[s, : -(-n // 64)].long()
    return np64(mass[layer, pages, h].flatten()[:n])


def weights_of(cache, hist, q, lse, s, b, h):
    """What the tokens of call row b give to the rows of sequence s in 64 bits, and how far float32 may be off: the
    logits' sums (2^-18 of their size), the exponent's rounding and the sum over the rows.  A weight below 2^-126, the
    smallest normal float32, comes out as zero: up to that much a row is absent."""
    g, nq = cache.cfg.num_q_heads // cache.cfg.num_kv_heads, q.shape[1]
    kd, kp, _, _, _ = held(cache, hist, s, h)
    n = len(kd)
    rows = np64(q[b, :, h * g:h * g + g]).reshape(-1, 128)
    e = np64(lse[b, :, h * g:h * g + g]).reshape(-1)
    lims = np.repeat([max(0, n - nq + 1 + i) for i in range(nq)], g)
    add, tol = P.weights(rows, kd, e, lims), np.zeros(n)
    for row, x, lim in zip(rows, e, lims):
        if lim > 0:
            w = np.exp(kd[:lim] @ row / 128 ** 0.5 - x)
            tol[:lim] += w * (2.0 ** -18 * (kp[:lim] @ np.abs(row) / 128 ** 0.5 + 1) + 2.0 ** -21 * abs(x))
    return add, 1.05 * tol + len(rows) * (2.0 ** -22 * add + 2.0 ** -126)


@pytest.mark.parametrize("HQ, HKV", HEADS)
@pytest.mark.parametrize("bits, n_q", [((4, 4), 1), ((8, 8), 3), ((8, 4), 2), ((4, 8), 17)])
def test_weights_accumulate(hyq, HQ, HKV, bits, n_q):
    lens = [300, 1, 0, 63, 64, 65, 1000]
    cache, hist = filled(HQ, HKV, lens, bits)
    order = [6, 2, 0, 4, 1, 5, 3]
    q = queries(8, len(lens), n_q, HQ)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    cache.attention(0, q, out, seqs=ints(order), lse=lse)
    mass = mass_tensor(cache)
    cache.accumulate(0, q, lse, mass, seqs=ints(order), n_new=ints([lens[s] for s in order]))
    first = mass.clone()
    cache.accumulate(0, q, lse, mass, seqs=ints(order))        # once more: the last n_q are new
    assert err(cache) == 0
    for b, s in enumerate(order):
        n = lens[s]
        for h in range(HKV):
            if not n:
                continue
            add, tol = weights_of(cache, hist, q, lse, s, b, h)
            got = mass_of(cache, first, s, h)
            assert (np.abs(got - add) <= tol).all()
            assert abs(got.sum() - min(n, n_q) * (HQ // HKV)) <= 1e-4 * (1 + got.sum())
            twice = np.where(np.arange(n) >= n - n_q, add, 2 * add)
            assert (np.abs(mass_of(cache, mass, s, h) - twice) <= 2 * tol + 2.0 ** -23 * twice).all()
    # entries of no position
    used = torch.zeros(cache.mass_shape, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        for j in range(-(-n // 64)):
            used[0, cache.table()[s, j].long(), :, : min(64, n - 64 * j)] = True
    assert mass[~used].isnan().all() and mass[used].isfinite().all()
    again = first.clone()
    cache.accumulate(0, q, lse, again, seqs=ints(order))
    assert torch.equal(again.nan_to_num(), mass.nan_to_num())


def test_weights_of_one_layer_stay_in_it(hyq):
    cache = make(4, 2, 6, 1, 6, n_layers=3)
    hist = History(1, 2)
    k, v, _, _ = grow(cache, [0], [200], 1, layer=1)
    hist.add([0], [200], k, v)
    q = queries(9, 1, 1, 4)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    cache.attention(1, q, out, lse=lse)
    mass = mass_tensor(cache, 0.0)
    cache.accumulate(1, q, lse, mass)
    assert not mass[0].any() and not mass[2].any() and err(cache) == 0
    add, tol = weights_of(cache, hist, q, lse, 0, 0, 1)
    assert (np.abs(mass_of(cache, mass, 0, 1, 1) - add) <= tol).all()


def test_what_gives_no_weight_is_reported(hyq):
    cache, hist = filled(4, 2, [200, 90, 1])
    q = queries(10, 3, 2, 4)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    cache.attention(0, q, out, lse=lse)
    want = mass_tensor(cache, 0.0)
    cache.accumulate(0, q, lse, want)
    assert err(cache) == 0                       # the first token of sequence 2 sees nothing: minus infinity there
    new = ints([200, 90, 1])
    for at, bad in (((1, 0, 3), "q"), ((0, 1, 1), "lse"), ((0, 0, 0), "inf")):
        q2, l2 = q.clone(), lse.clone()
        if bad == "q":
            q2[at][7] = float("nan")
        else:
            l2[at] = float("nan") if bad == "lse" else float("-inf")
        mass = mass_tensor(cache)
        cache.accumulate(0, q2, l2, mass, n_new=new)
        assert err(cache) == L.DEVERR_SCORE
        # as if that row were not there: its lse so large that it gives nothing
        l3 = lse.clone()
        l3[at] = 1e30
        ref = mass_tensor(cache)
        cache.accumulate(0, q, l3, ref, n_new=new)
        assert err(cache) == 0
        assert torch.equal(mass.nan_to_num(-1), ref.nan_to_num(-1))
    for seqs in ([0, 1, 0], [0, 1, 3], [0, 1, -1]):
        mass = mass_tensor(cache, 0.0)
        cache.accumulate(0, q, lse, mass, seqs=ints(seqs))
        assert err(cache) == L.DEVERR_INDEX
        for s in (0, 1):
            for h in range(2):
                assert np.array_equal(mass_of(cache, mass, s, h), mass_of(cache, want, s, h))
        assert not mass_of(cache, mass, 2, 0).any()
    grown = make(4, 2, 12, 3, 8)
    grow(grown, [0], [150], 1)
    grown.fork(ints([0]), ints([1]))
    grow(grown, [1], [80], 2)                    # pages 0, 1 shared, the last one copied
    mass = mass_tensor(grown, 3.0)
    grown.attention(0, q[:1], out[:1], seqs=ints([1]), lse=lse[:1])
    grown.accumulate(0, q[:1], lse[:1], mass, seqs=ints([1]))
    assert err(grown) == L.DEVERR_PAGES
    pages = grown.table()[1].tolist()
    assert (mass[0, pages[:2]] == 3).all() and (mass[0, pages[2]] > 3).any()
    grown.table()[1, 2] = 77
    grown.accumulate(0, q[:1], lse[:1], mass, seqs=ints([1]))
    assert err(grown) == L.DEVERR_PAGES | L.DEVERR_INDEX


def test_weights_of_the_most_query_rows(hyq):
    cache, hist = filled(8, 1, [700])
    q = queries(12, 1, 64, 8)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    cache.attention(0, q, out, lse=lse)
    mass = mass_tensor(cache)
    cache.accumulate(0, q, lse, mass, n_new=ints([700]))
    assert err(cache) == 0
    add, tol = weights_of(cache, hist, q, lse, 0, 0, 0)
    assert (np.abs(mass_of(cache, mass, 0, 0) - add) <= tol).all()


# --- eviction --------------------------------------------------------------------------------------------------------------

def snapshot(cache, s):
    """Rows of a sequence by (layer, head): the six arrays of unpack_qblocks over its whole pages."""
    n = int(cache.lens()[s])
    pages = cache.table()[s, : -(-n // 64)].long()
    bk, bv = cache.cfg.bits_k, cache.cfg.bits_v
    out = {}
    for layer in range(cache.n_layers):
        for h in range(cache.cfg.num_kv_heads):
            out[layer, h] = unpack_qblocks(cache.pool()[layer, pages, h].cpu().numpy(), len(pages) * 64, bk, bv)
    return n, pages.tolist(), out


def expect_evicted(cache, mass, seqs, keep, first, last):
    """The whole pool, bounds, masses, refs and lens after the call, from the rules."""
    bk, bv = cache.cfg.bits_k, cache.cfg.bits_v
    pool, bounds, m = cache.pool().cpu().numpy().copy(), cache.bounds().cpu().numpy().copy(), mass.cpu().numpy().copy()
    refs, lens = cache.refs().cpu().numpy().copy(), cache.lens().cpu().numpy().copy()
    for s, k in zip(seqs, keep):
        n, pages, rows = snapshot(cache, s)
        if n <= k:
            continue
        kb = -(-k // 64)
        for (layer, h), parts in rows.items():
            w = mass[layer, pages, h].flatten().cpu().numpy()
            src = P.keep_positions(w[:n].astype(np.float64), n, k, first, last)
            full = np.concatenate([np.array(src, int), np.arange(k, kb * 64)])
            new = [x[full] for x in parts]
            if kb:
                pool[layer, pages[:kb], h] = pack_qblocks(new[0], new[1], new[2], new[3], new[4], new[5], bk, bv)
                m[layer, pages[:kb], h] = w[full].reshape(kb, 64)
            for j in range(kb):
                r = slice(64 * j, min(k, 64 * j + 64))
                if any(src[i] != i for i in range(r.start, r.stop)):
                    c, s16, z16 = new[0][r], new[2][r], new[3][r]
                    x = (c.astype(np.float32) * np.repeat(s16.astype(np.float32), 32, -1)
                         + np.repeat(z16.astype(np.float32), 32, -1))
                    lo, hi, e = P.bounds(x.astype(np.float64))
                    rec = np.zeros(272, np.uint8)
                    rec[:128], rec[128:256] = lo.astype(np.int8).view(np.uint8), hi.astype(np.int8).view(np.uint8)
                    rec[256:260] = np.array([e], np.int32).view(np.uint8)
                    bounds[layer, pages[j], h] = rec
        for p in pages[kb:]:
            refs[p] -= 1
        lens[s] = k
    return pool, bounds, m, refs, lens


def check_evicted(cache, mass, want):
    pool, bounds, m, refs, lens = want
    assert np.array_equal(cache.lens().cpu().numpy(), lens) and np.array_equal(cache.refs().cpu().numpy(), refs)
    assert np.array_equal(cache.pool().cpu().numpy(), pool)
    assert np.array_equal(mass.cpu().numpy().view(np.uint32), m.view(np.uint32))
    assert np.array_equal(cache.bounds().cpu().numpy(), bounds)


def random_mass(cache, seed, ties=True):
    gen = torch.Generator().manual_seed(seed)
    m = torch.rand(cache.mass_shape, generator=gen)
    if ties:
        m = torch.where(torch.rand(m.shape, generator=gen) < 0.6, (m * 4).floor(), m)
    return m.cuda()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("first, last", [(0, 0), (4, 0), (0, 7), (3, 70), (1, 64), (20, 20)])
def test_eviction_moves_rows_byte_for_byte(hyq, bits, first, last):
    lens = [300, 64, 5, 0, 129, 640, 200]
    keep = [max(first + last, k) for k in (200, 63, 9, 0, 128, 130, 100)]
    cache, _ = filled(4, 2, lens, bits, n_layers=2)
    grow(cache, [i for i, n in enumerate(lens) if n], [n for n in lens if n], 5, layer=1, reserve=False)
    mass = random_mass(cache, first + 10 * last)
    order = [4, 0, 6, 2, 5, 3, 1]
    want = expect_evicted(cache, mass, order, [keep[s] for s in order], first, last)
    cache.evict(mass, ints([keep[s] for s in order]), seqs=ints(order), n_first=first, n_last=last)
    assert err(cache) == 0
    check_evicted(cache, mass, want)
    cache.evict(mass, ints(keep), n_first=first, n_last=last)        # nothing more to drop
    assert err(cache) == 0
    check_evicted(cache, mass, want)


@pytest.mark.parametrize("n, keep, first, last", [(20000, 4096, 4, 128), (40000, 39000, 0, 0), (3000, 10, 2, 3), (2000, 1, 0, 1),
                                                  (1000, 0, 0, 0), (700, 690, 600, 64), (129, 128, 0, 128)])
def test_eviction_of_long_sequences(hyq, n, keep, first, last):
    cache, _ = filled(1, 1, [n])
    mass = random_mass(cache, n)
    want = expect_evicted(cache, mass, [0], [keep], first, last)
    cache.evict(mass, ints([keep]), n_first=first, n_last=last)
    assert err(cache) == 0
    check_evicted(cache, mass, want)


def test_eviction_by_masses_of_any_kind(hyq):
    """Infinities, NaN, negative and equal masses."""
    cache, _ = filled(2, 2, [400, 400, 400])
    mass = random_mass(cache, 3)
    mass[mass > 3.5] = float("nan")
    mass[(mass > 2.9) & (mass < 3.1)] = float("inf")
    mass[(mass > 0.9) & (mass < 1.0)] *= -1
    mass[(mass > 0.8) & (mass < 0.9)] = float("-inf")
    mass[(mass > 0.7) & (mass < 0.8)] = -0.0
    mass[0, cache.table()[1, :7].long()] = 1.0        # one sequence's all equal
    want = expect_evicted(cache, mass, [0, 1, 2], [350, 60, 30], 1, 2)
    cache.evict(mass, ints([350, 60, 30]), n_first=1, n_last=2)
    assert err(cache) == 0
    check_evicted(cache, mass, want)


@pytest.mark.parametrize("n,keep", [(400, 90), (9000, 700)])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf", "zero", "tiny", "mostly zero", "half nan"])
def test_eviction_by_masses_that_tie(hyq, n, keep, what):
    """More equal masses than places: the lower positions stay."""
    cache, _ = filled(2, 1, [n, 100])
    mass = random_mass(cache, 6)
    own = mass[:, cache.table()[0, :(n + 63) // 64].long()]
    some = torch.rand(own.shape, generator=torch.Generator("cuda").manual_seed(n), device="cuda")
    if what == "half nan":
        own[some < 0.5] = float("nan")
    elif what == "mostly zero":
        own[some < 0.97] = 0.0
    else:
        own.fill_({"nan": float("nan"), "inf": float("inf"), "-inf": float("-inf"), "zero": 0.0, "tiny": 1e-42}[what])
        own[some < 0.01] = 1e-43 if what == "tiny" else 0.0
    mass[:, cache.table()[0, :(n + 63) // 64].long()] = own
    want = expect_evicted(cache, mass, [0], [keep], 3, 20)
    cache.evict(mass, ints([keep]), seqs=ints([0]), n_first=3, n_last=20)
    assert err(cache) == 0
    check_evicted(cache, mass, want)


def test_eviction_leaves_out_what_it_reports(hyq):
    def start():
        cache, _ = filled(2, 1, [200, 150, 300], spare=12)
        return cache, random_mass(cache, 4)
    for seqs, keep, good in (([0, 7, 1], [100, 50, 90], [0, 2]), ([0, -1, 1], [100, 50, 90], [0, 2]), ([0, 1, 0], [100, 90, 80], [0, 1]),
                             ([0, 2, 1], [100, 9, 90], [0, 2])):
        cache, mass = start()
        want = expect_evicted(cache, mass, [seqs[i] for i in good], [keep[i] for i in good], 4, 6)
        cache.evict(mass, ints(keep), seqs=ints(seqs), n_first=4, n_last=6)
        assert err(cache) == L.DEVERR_INDEX
        check_evicted(cache, mass, want)
    cache, mass = start()
    cache.table()[1, 1] = 10 ** 6
    pool, lens = cache.pool().clone(), cache.lens().clone()
    cache.evict(mass, ints([90]), seqs=ints([1]))
    assert err(cache) == L.DEVERR_INDEX and torch.equal(cache.pool(), pool) and torch.equal(cache.lens(), lens)


def test_eviction_of_forked_sequences(hyq):
    """A kept page that another sequence holds is not written; one that is only dropped may be shared."""
    cache, _ = filled(2, 1, [200, 0, 0], spare=12)
    cache.fork(ints([0, 0]), ints([1, 2]))
    mass = random_mass(cache, 5)
    pool, refs = cache.pool().clone(), cache.refs().clone()
    cache.evict(mass, ints([100]), seqs=ints([1]))
    assert err(cache) == L.DEVERR_PAGES and torch.equal(cache.pool(), pool) and torch.equal(cache.refs(), refs)
    assert cache.lens().tolist() == [200, 200, 200]
    cache.evict(mass, ints([0]), seqs=ints([1]))      # no page is kept
    assert err(cache) == 0 and cache.lens().tolist() == [200, 0, 200] and torch.equal(cache.pool(), pool)
    assert torch.equal(cache.refs()[cache.table()[0, :4].long()], torch.full((4,), 2, dtype=torch.int32, device="cuda"))


def test_eviction_of_the_most_sequences(hyq):
    n = 1024
    lens = [1 + (7 * i) % 150 for i in range(n)]
    cache, _ = filled(1, 1, lens, spare=0)
    mass = random_mass(cache, 6)
    keep = [max(3, x - i % 80) for i, x in enumerate(lens)]
    want = expect_evicted(cache, mass, range(n), keep, 1, 2)
    cache.evict(mass, ints(keep), n_first=1, n_last=2)
    assert err(cache) == 0
    check_evicted(cache, mass, want)


# --- together ----------------------------------------------------------------------------------------------------------------

def test_serving_at_a_budget(hyq):
    """Append, attend, accumulate, and every few steps evict: outputs and masses follow a plain restatement per head."""
    HQ, HKV, budget = 8, 2, 100
    g = HQ // HKV
    cache = make(HQ, HKV, 12, 2, 6)
    mass = mass_tensor(cache)
    rows = {(s, h): [np.zeros((0, 128)) for _ in range(5)] + [np.zeros(0)] for s in range(2) for h in range(HKV)}
    for step in range(9):
        counts = [90, 130] if step == 0 else [1, 1 + step % 3]
        nq = 1 if step else 5
        k, v, _, _ = grow(cache, [0, 1], counts, 20 + step)
        at = 0
        for s, n in enumerate(counts):
            for h in range(HKV):
                kd, kp, _ = P.dequantised(np64(k[at:at + n, h]), 4)
                vd, vp, vc = P.dequantised(np64(v[at:at + n, h]), 4)
                r = rows[s, h]
                rows[s, h] = [np.concatenate([a, b]) for a, b in zip(r, (kd, kp, vd, vp, vc, np.zeros(n)))]
            at += n
        q = queries(50 + step, 2, nq, HQ)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        cache.attention(0, q, out, lse=lse)
        cache.accumulate(0, q, lse, mass, n_new=ints(counts))
        assert err(cache) == 0
        for (s, h), (kd, kp, vd, vp, vc, w) in rows.items():
            n = len(kd)
            add = P.weights(np64(q[s, :, h * g:h * g + g]).reshape(-1, 128), kd,
                            np64(lse[s, :, h * g:h * g + g]).reshape(-1), np.repeat([n - nq + 1 + i for i in range(nq)], g))
            rows[s, h][5] = w + add
            got = mass_of(cache, mass, s, h)
            assert np.allclose(got, rows[s, h][5], rtol=1e-3, atol=1e-5)
            rows[s, h][5] = got                  # the choice below is the kernel's own numbers'
            for i in range(nq):
                vis = np.arange(n) < n - nq + 1 + i
                for r in range(h * g, h * g + g):
                    want = P.attend(np64(q[s, i, r]), kd, vd, vis)
                    tol = P.attend_error(np64(q[s, i, r]), kd, kp, vp, vc, vis, want)
                    assert (np.abs(np64(out[s, i, r]) - want) <= tol).all()
        if step % 3 == 0:
            cache.evict(mass, ints([budget, budget]), n_first=2, n_last=16)
            assert err(cache) == 0
            for key, r in rows.items():
                src = P.keep_positions(r[5], len(r[0]), budget, 2, 16)
                rows[key] = [x[src] for x in r]
            # what is chosen from the new bounds is still chosen from bounds
            sel = torch.empty(2, nq, HKV, 2, dtype=torch.int32, device="cuda")
            cache.select(0, q, sel)
            cache.attention_blocks(0, q, sel, out)
            assert err(cache) == 0 and out.isfinite().all()
    assert max(cache.lens().tolist()) <= budget + 6


def test_captured_steps_follow_lengths_groups_and_budgets(hyq):
    """Append, shared attention, weights, eviction and cross attention in one graph, replayed as the tables change; the
    same calls made one by one give the same bytes."""
    def build():
        cache, hist, groups = branches(8, 2, [128], [[5, 9, 70]])
        enc, _ = filled(8, 2, [200, 333], seed=9)
        return cache, groups[0], enc
    results = []
    for captured in (False, True):
        cache, seqs, enc = build()
        own = make(8, 2, 8, 1, 6)
        grow(own, [0], [140], 3)
        mass = torch.zeros(own.mass_shape, device="cuda")
        q, x = queries(1, 3, 1, 8), tokens(2, 11, 8)
        out, xo, oo = torch.empty_like(q), torch.empty_like(x), torch.empty_like(q[:1])
        lse = torch.empty(1, 1, 8, device="cuda")
        k, v = (torch.randn(3, 2, 128, generator=torch.Generator().manual_seed(5 + i)).to(torch.bfloat16).cuda() for i in range(2))
        s3, groups, shared, counts, keep = ints(seqs), ints([0, 3]), ints([128]), cu([4, 7]), ints([139])

        def step():
            cache.reserve(s3)
            cache.append(0, k, v, seqs=s3)
            cache.attention_shared(0, q, out, groups, shared, seqs=s3)
            enc.cross_attention(0, x, xo, cu_q=counts)
            own.reserve()
            own.append(0, k[:1], v[:1])
            own.attention(0, q[:1], oo, lse=lse)
            own.accumulate(0, q[:1], lse, mass)
            own.evict(mass, keep, n_first=1, n_last=8)
        step()
        if captured:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        got = []
        for i in range(4):
            q.copy_(queries(10 + i, 3, 1, 8))
            x.copy_(tokens(20 + i, 11, 8))
            shared.fill_(128 if i != 2 else 64)
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            got += [out.clone(), xo.clone(), oo.clone(), mass.clone(), own.pool().clone(), cache.lens().clone()]
        assert err(cache) == 0 and err(own) == 0 and err(enc) == 0
        results.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_calls_on_other_streams(hyq):
    """Two caches' calls under way at once on streams of their own, and a given stream that the call must follow."""
    a, b = (branches(8, 2, [256], [[5, 9, 70]], seed=s) for s in (1, 2))
    want, got = [], []
    qs = [queries(s, 3, 1, 8) for s in range(2)]
    args = ints([0, 3]), ints([256])
    for (cache, _, groups), q in zip((a, b), qs):
        out, x = torch.empty_like(q), torch.empty_like(q[:, 0])
        cache.attention_shared(0, q, out, *args, seqs=ints(groups[0]))
        cache.cross_attention(0, q[:, 0], x, seqs=ints(groups[0][:1]), cu_q=ints([0, 3]))
        want += [out, x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for (cache, _, groups), q, s in zip((a, b), qs, streams):
        out, x = torch.empty_like(q), torch.empty_like(q[:, 0])
        seqs, one, three = ints(groups[0]), ints(groups[0][:1]), ints([0, 3])
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            cache.attention_shared(0, q, out, *args, seqs=seqs, stream=s)
            cache.cross_attention(0, q[:, 0], x, seqs=one, cu_q=three, stream=s)
        got += [out, x]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_refused_calls_raise_and_change_nothing(hyq):
    cache, _ = filled(4, 2, [200])
    q, t = queries(1, 1, 1, 4), tokens(1, 3, 4)
    out, xo = torch.full_like(q, 5.0), torch.full_like(t, 5.0)
    mass = mass_tensor(cache, 1.0)
    lse = torch.zeros(1, 1, 4, device="cuda")
    for f in (lambda: cache.attention_shared(3, q, out, ints([0, 1]), ints([64])),
              lambda: cache.cross_attention(1, t, xo, cu_q=ints([0, 3])),
              lambda: cache.cross_attention(0, t, xo, cu_q=ints([0, 1, 2, 3])),         # more rows than the table has
              lambda: cache.accumulate(-1, q, lse, mass),
              lambda: cache.evict(mass, ints([100]), n_first=-1),
              lambda: cache.evict(mass, ints([100, 100]))):
        with pytest.raises(HyqError):
            f()
    for f in (lambda: cache.attention_shared(0, q, out, ints([0, 1]).cpu(), ints([64])),
              lambda: cache.cross_attention(0, t.cpu(), xo, cu_q=ints([0, 3])),
              lambda: cache.accumulate(0, q, lse.cpu(), mass), lambda: cache.evict(mass.cpu(), ints([100]))):
        with pytest.raises(ValueError):
            f()
    assert (out == 5).all() and (xo == 5).all() and (mass == 1).all() and cache.lens().tolist() == [200]
    assert err(cache) == 0


def test_wide_pool_offsets_past_32_bits(hyq):
    """Pages, masses and bounds whose byte offsets pass 2^32."""
    n_pages = 60000                                   # 8 KV heads, 8-bit codes: 8.8 GB
    cache = make(8, 8, n_pages, 2, n_pages, bits=(8, 8))
    hist = History(2, 8)
    k, v, _, _ = grow(cache, [0], [300], 1)
    hist.add([0], [300], k, v)
    last = list(range(n_pages - 5, n_pages))
    pages = cache.table()[0, :5].tolist()
    cache.pool()[0, last] = cache.pool()[0, pages]
    cache.bounds()[0, last] = cache.bounds()[0, pages]
    cache.table()[1, :5] = ints(last)
    cache.lens()[1] = 300
    cache.refs()[last] = 1
    q = tokens(1, 4, 8)
    out = torch.empty_like(q)
    cache.cross_attention(0, q, out, seqs=ints([1]), cu_q=ints([0, 4]))
    same = torch.empty_like(q)
    cache.cross_attention(0, q, same, seqs=ints([0]), cu_q=ints([0, 4]))
    assert torch.equal(out, same)
    check_cross(cache, hist, q, same, [0], [4])
    mass = torch.zeros(cache.mass_shape, device="cuda")
    qq = q[None, :1].contiguous()
    o, lse = torch.empty_like(qq), torch.empty(1, 1, 8, device="cuda")
    for s in (0, 1):
        cache.attention(0, qq, o, seqs=ints([s]), lse=lse)
        cache.accumulate(0, qq, lse, mass, seqs=ints([s]))
    assert torch.equal(mass[0, last], mass[0, pages]) and mass[0, last].any()
    cache.evict(mass, ints([100, 100]), n_last=4)
    assert err(cache) == 0
    assert torch.equal(cache.pool()[0, last], cache.pool()[0, pages]) and torch.equal(mass[0, last], mass[0, pages])
    assert torch.equal(cache.bounds()[0, last], cache.bounds()[0, pages])
