"""pa_decode_weights and pa_evict: accumulated attention weights and eviction by them."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_335_b200 as pa
from tests import plain_forms as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, FP8, I8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8


def _pool(lens, hkv, d, bs, dtype, seed):
    """Scattered blocks; the slots past each context hold NaN (255 for codes: E4M3's NaN)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 5
    order = rng.permutation(nb)
    tables = np.full((len(lens), max(need + [1]) + 1), -1, dtype=np.int32)
    at = 0
    caches = []
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n]
        at += n
    for _ in range(2):
        x = torch.randn((nb, hkv, bs, d), generator=g, device=DEV)
        c = (x * 40).to(dtype) if dtype in (FP8, I8) else x.to(dtype)
        raw = c.view(torch.uint8) if c.element_size() == 1 else c
        for i, n in enumerate(lens):
            if n % bs:
                raw[int(tables[i, n // bs]), :, n % bs:] = 255 if c.element_size() == 1 else float("nan")
        caches.append(c)
    return tables, torch.as_tensor(tables, device=DEV), *caches


def _rows(cache, table, n, bs):
    """[Hkv][n][D] of one sequence, codes as bytes."""
    raw = cache.view(torch.uint8) if cache.element_size() == 1 else cache
    hkv, d = cache.shape[1], cache.shape[3]
    b = torch.as_tensor(table[:-(-n // bs)], device=DEV).long()
    return raw[b].permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n]


LENS = [1, 16, 17, 333, 0, 700]


@pytest.mark.parametrize("h,hkv,d,dtype", [
    (8, 8, 128, BF16), (16, 2, 128, BF16), (8, 4, 64, BF16), (20, 2, 64, BF16), (36, 1, 128, BF16),
    (6, 2, 128, F32), (3, 3, 64, F32),
    (16, 2, 128, FP8), (4, 4, 64, FP8), (16, 4, 128, I8), (5, 5, 128, I8), (8, 2, 64, I8)])
@pytest.mark.parametrize("ps", [0, -1, 64])
def test_decode_weights(h, hkv, d, dtype, ps):
    bs, scale = 16, 1 / math.sqrt(d)
    tables, tt, kc, vc = _pool(LENS, hkv, d, bs, dtype, seed=h + d)
    ctx = torch.tensor(LENS, dtype=torch.int32, device=DEV)
    act = F32 if dtype == F32 else BF16
    q = torch.randn((len(LENS), h, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(act)
    quant = dtype in (FP8, I8)
    scales = (torch.linspace(0.02, 0.03, hkv, device=DEV), torch.linspace(0.01, 0.02, hkv, device=DEV)) if quant else ()
    w0 = torch.rand((len(LENS), hkv, 720), device=DEV)
    w, out, ref = w0.clone(), torch.empty_like(q), torch.empty_like(q)
    (pa.pa_decode_quant if quant else pa.pa_decode)(ref, q, kc, vc, *scales, tt, ctx, scale,
                                                    max_context_len=704, partition_size=ps)
    (pa.pa_decode_weights_quant if quant else pa.pa_decode_weights)(
        out, w, q, kc, vc, *scales, tt, ctx, scale, max_context_len=704, partition_size=ps)
    pa.pa_sync_check()
    assert torch.equal(out, ref)                                   # the same out, bit for bit
    for s, n in enumerate(LENS):
        assert torch.equal(w[s, :, n:], w0[s, :, n:])
        if n == 0:
            continue
        k = _rows(kc, tables[s], n, bs)
        k = (k.view(dtype).double() * scales[0].double()[:, None, None]) if quant else k.double()
        qs = q[s].double().reshape(hkv, h // hkv, d)
        x = torch.einsum("kgd,ktd->kgt", qs, k) * scale
        sabs = (torch.einsum("kgd,ktd->kgt", qs.abs(), k.abs()) * scale).amax((1, 2), keepdim=True)[..., 0]
        p = torch.softmax(x, -1).sum(1)
        # a score's error moves a weight and its sum by that factor each; q is rounded to f16
        # (2^-11, half a step) over codes
        rel = 2 * ((d + 4) * P.EPS32 + (2.0 ** -11 if quant else 0)) * sabs + 2 * (n + 32) * P.EPS32
        tol = p * rel + (w0[s, :, :n].double() + p) * (h // hkv + 2) * P.EPS32
        err = (w[s, :, :n].double() - (w0[s, :, :n].double() + p)).abs()
        assert bool((err <= tol).all()), f"seq {s}: {float((err / tol).max()):.2f} of the bound"


def test_decode_weights_skips_bad_blocks():
    """A block id outside the pool: its tokens get no weight, the others share the whole."""
    for h, hkv in ((4, 4), (16, 2)):
        tables, tt, kc, vc = _pool([100, 40], hkv, 128, 16, BF16, seed=2)
        bad = tt.clone()
        bad[0, 2] = kc.shape[0]
        q = torch.randn((2, h, 128), device=DEV).to(BF16)
        w, out = torch.zeros((2, hkv, 112), device=DEV), torch.empty_like(q)
        pa.pa_decode_weights(out, w, q, kc, vc, bad, torch.tensor([100, 40], dtype=torch.int32, device=DEV), 0.1)
        with pytest.raises(pa.PAError):
            pa.pa_sync_check()
        assert not w[0, :, 32:48].any() and bool((w[0, :, :32] > 0).all())
        assert torch.allclose(w.sum(-1), torch.full((2, hkv), float(h // hkv), device=DEV), rtol=1e-4)


@pytest.mark.parametrize("dtype,d,hkv,bs", [(BF16, 128, 3, 16), (F32, 64, 2, 32), (FP8, 64, 5, 16), (I8, 128, 1, 64),
                                            (F32, 128, 2, 16), (BF16, 64, 4, 256), (BF16, 64, 24, 16), (I8, 64, 23, 32)])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (32, 0), (33, 32), (100, 7), (320, 64), (333, 333),
                                           (699, 20), (1000, 10)])
def test_evict(dtype, d, hkv, bs, budget, recent):
    lens = [1, 16, 33, 333, 0, 700, 650]
    tables, tt, kc, vc = _pool(lens, hkv, d, bs, dtype, seed=budget + recent)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(budget)
    w = (torch.randn((len(lens), hkv, 1024), generator=g, device=DEV) * 2).exp()
    w[5] = torch.round(w[5])                                       # many ties
    w[6, 0, :40] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 0.0] * 8, device=DEV)
    w[6, -1] = 0.0                                                 # nothing but ties
    for inplace in (False, True):
        k1, v1 = kc.clone(), vc.clone()
        w_in = w.clone()
        w_out = w_in if inplace else torch.full_like(w, 7.0)
        new = torch.full_like(ctx, -5)
        kept = torch.full((len(lens), hkv, budget), -7, dtype=torch.int32, device=DEV)
        pa.pa_evict(k1, v1, tt, ctx, w_in, w_out, new, kept, budget, recent)
        pa.pa_sync_check()
        assert new.tolist() == [min(n, budget) for n in lens]
        for s, n in enumerate(lens):
            m = min(n, budget)
            for kh in range(hkv):
                want = P.evict(w[s, kh].tolist(), n, budget, recent)
                assert kept[s, kh].tolist() == want, (s, kh)
                idx = torch.tensor(want[:m], dtype=torch.long, device=DEV)
                assert torch.equal(w_out[s, kh, :m].view(torch.int32), w[s, kh, idx].view(torch.int32))
                assert not w_out[s, kh, m:].any()
                for before, after in ((kc, k1), (vc, v1)):
                    a = _rows(before, tables[s], n, bs)[kh][idx]
                    b = _rows(after, tables[s], m, bs)[kh]
                    assert torch.equal(a, b)
        # blocks of no sequence are left alone
        free = sorted(set(range(kc.shape[0])) - set(tables[tables >= 0].tolist()))
        for before, after in ((kc, k1), (vc, v1)):
            raw = [x.view(torch.uint8 if x.element_size() == 1 else torch.int16 if x.element_size() == 2
                          else torch.int32) for x in (before, after)]
            assert torch.equal(raw[0][free], raw[1][free])


def test_evict_long_context():
    """More movers than one round of the selection lists, and the 32-bit key's every digit."""
    n, budget, hkv = 40000, 25000, 2
    tables, tt, kc, vc = _pool([n], hkv, 64, 64, FP8, seed=4)
    ctx = torch.tensor([n], dtype=torch.int32, device=DEV)
    w = torch.rand((1, hkv, n), device=DEV)
    w[0, 1] = torch.arange(n, device=DEV)                          # the last ones: every slot is a hole
    before = [_rows(c, tables[0], n, 64).clone() for c in (kc, vc)]
    w_out, new = torch.empty_like(w), torch.empty_like(ctx)
    kept = torch.empty((1, hkv, budget), dtype=torch.int32, device=DEV)
    pa.pa_evict(kc, vc, tt, ctx, w, w_out, new, kept, budget, 5)
    pa.pa_sync_check()
    for kh in range(hkv):
        want = P.evict(w[0, kh].tolist(), n, budget, 5)
        assert kept[0, kh].tolist() == want
        idx = torch.tensor(want, device=DEV)
        for b, c in zip(before, (kc, vc)):
            assert torch.equal(_rows(c, tables[0], budget, 64)[kh], b[kh][idx])


def test_evict_bad_inputs_touch_nothing_else():
    tables, tt, kc, vc = _pool([64, 64], 2, 128, 16, BF16, seed=5)
    ctx = torch.tensor([64, 64], dtype=torch.int32, device=DEV)
    w = torch.rand((2, 2, 64), device=DEV)
    bad = tt.clone()
    bad[0, 3] = kc.shape[0] + 3
    k1, v1 = kc.clone(), vc.clone()
    new = torch.empty_like(ctx)
    kept = torch.empty((2, 2, 32), dtype=torch.int32, device=DEV)
    pa.pa_evict(k1, v1, bad, ctx, w, torch.empty_like(w), new, kept, 32, 16)
    with pytest.raises(pa.PAError) as e:
        pa.pa_sync_check()
    assert e.value.code == pa.PA_ERR_BAD_INDEX
    want = kept[1].long()
    for kh in range(2):
        assert torch.equal(_rows(k1, tables[1], 32, 16)[kh], _rows(kc, tables[1], 64, 16)[kh][want[kh]])
    # a context above the bound is clipped to it
    pa.pa_evict(k1, v1, tt, torch.tensor([65, 10], dtype=torch.int32, device=DEV), w, torch.empty_like(w), new,
                kept, 32, 16, max_context_len=64)
    with pytest.raises(pa.PAError):
        pa.pa_sync_check()
    assert new.tolist() == [32, 10]
