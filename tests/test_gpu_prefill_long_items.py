"""Prompt weights whose items each take longer than a pipeline wait may: a CTA's next items are
found long before there is room to hand them over."""
import pytest
import torch

import paged_kv_cache_335_b200 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_items_of_over_a_second():
    """2000 heads of one kv head over 116K tokens: 912 items, the longest of 1000 heads and 908
    query tiles (about 1.2 s). With every score and log-sum-exp 0 a token's weight is the number of
    (head, query) pairs that see it."""
    t, h, d = 116_001, 2000, 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 31 GB for q")
    q = torch.zeros((t, h, d), device=DEV, dtype=torch.bfloat16)
    k = torch.ones((t, 1, d), device=DEV, dtype=torch.bfloat16)
    lse = torch.zeros((h, t), device=DEV)
    cu = torch.tensor([0, t], dtype=torch.int32, device=DEV)
    w = torch.full((1, 1, t), -1.0, device=DEV)
    pa.pa_prefill_weights(w, q, k, lse, cu, 0.125, max_seq_len=t)
    pa.pa_sync_check()
    want = (t - torch.arange(t, device=DEV)).double() * h
    # a thread's sum takes one rounded addition per head of its item and query tile, and a few to
    # form each addend; the polynomial exponential of 0 is off by 2 EPS32
    tol = want * (h // 2 * (t // 128 + 1) + 16) * 2.0 ** -24
    assert bool(((w[0, 0].double() - want).abs() <= tol).all())
    last = t % 128                                  # the diagonal's own exponentials of 0 are 1
    assert torch.equal(w[0, 0, -last:].double(), want[-last:])
    del q, lse
    torch.cuda.empty_cache()
