"""pa_evict over long contexts, up to the longest: the keys of the selection lie in shared memory
up to 46848 tokens and are made of the weights in every pass above."""
import pytest
import torch

import paged_kv_cache_335_b200 as pa
from tests import plain_forms as P
from tests.test_gpu_evict import BF16, DEV, FP8, _pool, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("n,budget,recent,room,dtype", [
    (46848, 30000, 100, 0, FP8), (46849, 46848, 0, 3, FP8), (60000, 25000, 5, 1, BF16),
    (131072, 131000, 4096, 0, FP8), (100001, 1, 0, 0, FP8), (70000, 9000, 9000, 2, BF16)])
def test_long_contexts(n, budget, recent, room, dtype, inplace):
    hkv, bs = 3, 64
    lens = [n, n - 1, 17]
    tables, tt, kc, vc = _pool(lens, hkv, 64, bs, dtype, seed=n)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    w = torch.rand((3, hkv, n + room), device=DEV, generator=torch.Generator(device=DEV).manual_seed(n))
    w[0, 1, :n] = torch.arange(n, device=DEV).float()              # the last ones: every slot is a hole
    w[0, 2] = torch.round(w[0, 2] * 3)                             # nothing but ties
    w[1, 0, ::7] = float("nan")
    w[1, 1] = -w[1, 1] * 1e-38
    before = [[_rows(c, tables[s], m, bs).clone() for c in (kc, vc)] for s, m in enumerate(lens)]
    w_in = w.clone()
    w_out = w_in if inplace else torch.full_like(w, 7.0)
    new = torch.full_like(ctx, -5)
    kept = torch.full((3, hkv, budget), -7, dtype=torch.int32, device=DEV)
    pa.pa_evict(kc, vc, tt, ctx, w_in, w_out, new, kept, budget, recent, max_context_len=n)
    pa.pa_sync_check()
    assert new.tolist() == [min(m, budget) for m in lens]
    for s, m in enumerate(lens):
        left = min(m, budget)
        for kh in range(hkv):
            want = P.evict(w[s, kh].tolist(), m, budget, recent)
            assert kept[s, kh].tolist() == want
            idx = torch.tensor(want[:left], device=DEV)
            assert torch.equal(w_out[s, kh, :left].view(torch.int32), w[s, kh, idx].view(torch.int32))
            assert not w_out[s, kh, left:].any()
            for b, c in zip(before[s], (kc, vc)):
                assert torch.equal(_rows(c, tables[s], left, bs)[kh], b[kh][idx])


def test_the_longest_context():
    n = pa.pa_evict_max_context()
    budget, recent, bs = n // 2 + 1, 1000, 256
    tables, tt, kc, vc = _pool([n], 1, 64, bs, FP8, seed=1)
    ctx = torch.tensor([n], dtype=torch.int32, device=DEV)
    w = torch.rand((1, 1, n), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    before = [_rows(c, tables[0], n, bs).clone() for c in (kc, vc)]
    w_out, new = w.clone(), torch.empty_like(ctx)
    kept = torch.empty((1, 1, budget), dtype=torch.int32, device=DEV)
    pa.pa_evict(kc, vc, tt, ctx, w_out, w_out, new, kept, budget, recent)
    pa.pa_sync_check()
    want = P.evict(w[0, 0].tolist(), n, budget, recent)
    assert kept[0, 0].tolist() == want
    idx = torch.tensor(want, device=DEV)
    assert torch.equal(w_out[0, 0, :budget], w[0, 0, idx]) and not w_out[0, 0, budget:].any()
    for b, c in zip(before, (kc, vc)):
        assert torch.equal(_rows(c, tables[0], budget, bs)[0], b[0][idx])
    with pytest.raises(pa.PAError) as e:
        pa.pa_evict(kc, vc, torch.zeros((1, n // bs + 2), dtype=torch.int32, device=DEV), ctx,
                    torch.zeros((1, 1, n + 1), device=DEV), torch.zeros((1, 1, n + 1), device=DEV), new, kept, budget,
                    recent, max_context_len=n + 1)
    assert e.value.code == pa.PA_ERR_UNSUPPORTED
