"""Attention over the paged cache where its arithmetic is at its limits: values
of any size under few large probabilities, queries that are not finite."""
import numpy as np
import pytest
import torch

from hybrid_precision_quantized_gb300 import hyq_read_device_error
from oracle import paged as P
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
