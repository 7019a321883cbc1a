"""pa_decode_weights with enough work items that the grouped-head kernel claims them from its
counter: the same out as pa_decode's, and the same weights as sequence by sequence."""
import math

import pytest
import torch

import paged_kv_cache_335_b200 as pa
from tests import plain_forms as P
from tests.test_gpu_evict import BF16, DEV, FP8, I8, _pool, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h,hkv,d,dtype", [(32, 8, 128, BF16), (20, 10, 64, BF16), (32, 8, 128, FP8), (64, 8, 64, I8)])
def test_many_items(h, hkv, d, dtype):
    lens = [(211 * i) % 320 for i in range(80)]                    # 80 x hkv x 5 partitions of 64
    scale, quant = 1 / math.sqrt(d), dtype != BF16
    tables, tt, kc, vc = _pool(lens, hkv, d, 16, dtype, seed=h + d)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.randn((len(lens), h, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF16)
    scales = (torch.linspace(0.02, 0.03, hkv, device=DEV), torch.linspace(0.01, 0.02, hkv, device=DEV)) if quant else ()
    w0 = torch.rand((len(lens), hkv, 323), device=DEV)
    w, out, ref = w0.clone(), torch.empty_like(q), torch.empty_like(q)
    kw = dict(max_context_len=320, partition_size=64)
    plain = pa.pa_decode_quant if quant else pa.pa_decode
    call = pa.pa_decode_weights_quant if quant else pa.pa_decode_weights
    need = pa.pa_decode_weights_workspace_size(len(lens), h, 320, kc, 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)   # (NaN wherever nothing is written)
    plain(ref, q, kc, vc, *scales, tt, ctx, scale, **kw)
    call(out, w, q, kc, vc, *scales, tt, ctx, scale, workspace=ws, **kw)
    pa.pa_sync_check()
    assert pa.load_library().pa_test_last_decode_kernel() == pa.PA_KERNEL_MMA
    assert torch.equal(out, ref)
    again = w0.clone()
    for s in range(len(lens)):                                     # 1 x hkv x 5 items: dealt out in order
        o = torch.empty_like(q[:1])
        call(o, again[s:s + 1], q[s:s + 1], kc, vc, *scales, tt[s:s + 1], ctx[s:s + 1], scale, **kw)
        assert torch.equal(o[0], ref[s])
    assert torch.equal(again, w)
    for s, n in enumerate(lens):
        assert torch.equal(w[s, :, n:], w0[s, :, n:])
        if n == 0:
            continue
        k = _rows(kc, tables[s], n, 16)
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
