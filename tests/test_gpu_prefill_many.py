"""pa_prefill and pa_prefill_weights over more prompts than a warp has lanes, of several tiles
each, with more items than the GPU has SMs (a CTA takes one after another)."""
import math

import pytest
import torch

import paged_kv_cache_335_b200 as pa
from tests import plain_forms as P
from tests.test_gpu_prefill import BF16, DEV, F32, _check, _inputs

pytestmark = pytest.mark.gpu

MANY = [
    ([2048] * 64, 1, 1, 64, BF16),
    ([1024] * 64, 8, 2, 128, BF16),
    ([(977 * i) % 3000 + 1 for i in range(48)], 8, 2, 64, BF16),
    ([700] * 64, 4, 2, 128, BF16),
    ([1] * 33 + [5000, 0, 129], 10, 2, 64, BF16),          # the long one in the second 32
    ([(389 * i) % 500 for i in range(70)], 4, 2, 64, F32),  # (more than two CTAs per SM)
]


@pytest.mark.parametrize("lens,h,hkv,d,dtype", MANY, ids=range(len(MANY)))
def test_prefill_of_many_prompts(lens, h, hkv, d, dtype):
    scale = 1 / math.sqrt(d)
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=len(lens), front=1, behind=2)
    out = torch.full(q.shape, 7.0, device=DEV, dtype=dtype)
    lse = torch.full((h, q.shape[0]), 7.0, device=DEV)
    pa.pa_prefill(out, q, k, v, cut, scale, max_seq_len=max(lens), lse=lse)
    pa.pa_sync_check()
    _check(lens, h, hkv, d, dtype, scale, q, k, v, cu, out, lse)
    assert bool((out[:1] == 7).all()) and bool((out[-2:] == 7).all())


@pytest.mark.parametrize("last", [0, 64])
@pytest.mark.parametrize("lens,h,hkv,d,dtype", MANY, ids=range(len(MANY)))
def test_weights_of_many_prompts(lens, h, hkv, d, dtype, last):
    scale = 1 / math.sqrt(d)
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=len(lens), front=1, behind=2)
    lse = torch.full((h, q.shape[0]), float("nan"), device=DEV)
    for s, n in enumerate(lens):
        if n:
            a, b = cu[s], cu[s + 1]
            lse[:, a:b] = P.prompt_attention(q[a:b], k[a:b], v[a:b], scale)[1].float()
    w = torch.full((len(lens), hkv, max(lens) + 3), 7.0, device=DEV)
    pa.pa_prefill_weights(w, q, k, lse, cut, scale, max_seq_len=max(lens), last_queries=last)
    pa.pa_sync_check()
    for s, n in enumerate(lens):
        assert not w[s, :, n:].any()
        if n == 0:
            continue
        a, b = cu[s], cu[s + 1]
        ref, mag = P.prompt_weights(q[a:b], k[a:b], lse[:, a:b], scale, last)
        tol = P.EPS32 * (mag + ref * ((h // hkv) * n + 16)) + 1e-37
        err = (w[s, :, :n].double() - ref).abs()
        assert bool((err <= tol).all()), f"prompt {s}: {float((err / tol).max()):.2f} of the bound"


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_overlapping_prompts_are_skipped(dtype):
    """The third prompt's rows are the first one's: the first is whole, the third reported."""
    h, hkv, d = 4, 2, 64
    q, k, v, cu, _ = _inputs([700], h, hkv, d, dtype, seed=3)
    cut = torch.tensor([0, 700, 0, 700], dtype=torch.int32, device=DEV)
    out = torch.full(q.shape, 7.0, device=DEV, dtype=dtype)
    lse = torch.full((h, 700), 7.0, device=DEV)
    w = torch.full((3, hkv, 700), 7.0, device=DEV)
    for call in (lambda: pa.pa_prefill(out, q, k, v, cut, 0.125, max_seq_len=700, lse=lse),
                 lambda: pa.pa_prefill_weights(w, q, k, lse, cut, 0.125, max_seq_len=700)):
        call()
        with pytest.raises(pa.PAError) as e:
            pa.pa_sync_check()
        assert e.value.code == pa.PA_ERR_BAD_INDEX
    _check([700], h, hkv, d, dtype, 0.125, q, k, v, cu, out, lse)
    total = w.sum(-1)
    assert torch.allclose(total[0], torch.full_like(total[0], 700.0 * h / hkv), rtol=1e-3)
    assert not w[1:].any()
