"""Calls on the paged cache that its documentation allows, beside those of
test_gpu_paged.py."""
import pytest
import torch

from hybrid_precision_quantized_gb300 import hyq_read_device_error
from hybrid_precision_quantized_gb300 import _lib as L
from tests.test_gpu_paged import grow, ints, make, queries

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
