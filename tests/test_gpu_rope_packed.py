"""A packed projection's q and k turned together: the rotated keys come out beside the queries, as
prompt attention takes them, whatever the pool holds."""
import pytest
import torch

import paged_kv_cache_335_b200 as pa
from tests import plain_forms as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                         (torch.bfloat16, torch.float8_e4m3fn), (torch.bfloat16, torch.int8)])
def test_prompt_attention_of_rows_turned_together(dtype, cache):
    lens, h, hkv, d, bs = [200, 1, 77], 8, 2, 64, 16
    t = sum(lens)
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((t, h + 2 * hkv, d), generator=g, device=DEV).to(dtype)
    q, k, v, qk = x[:, :h], x[:, h:h + hkv], x[:, h + hkv:], x[:, :h + hkv]
    pos = torch.cat([torch.arange(n) for n in lens])[None].to(torch.int32).to(DEV)
    nb = -(-t // bs)
    kc, vc = (torch.zeros((nb, hkv, bs, d), device=DEV).to(cache) for _ in range(2))
    rope, slots = pa.rope_desc(d), torch.arange(t, device=DEV)
    out = torch.empty((t, h + hkv, d), device=DEV, dtype=dtype)
    scales = () if cache == dtype else (torch.full((hkv,), 0.02, device=DEV), torch.full((hkv,), 0.02, device=DEV))
    call = pa.pa_rope_append if cache == dtype else pa.pa_rope_append_quant
    call(out, qk, k, v, pos, slots, kc, vc, *scales, rope)
    qr, kr = out[:, :h], out[:, h:]
    # as with q alone, and k as the pool has it
    one = torch.empty((t, h, d), device=DEV, dtype=dtype)
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    call(one, q, k, v, pos, slots, kc2, vc2, *scales, rope)
    pa.pa_sync_check()
    assert torch.equal(qr, one)
    assert torch.equal(kc.view(torch.uint8), kc2.view(torch.uint8)) and torch.equal(vc.view(torch.uint8), vc2.view(torch.uint8))
    if cache == dtype:
        assert torch.equal(kr, kc.transpose(1, 2).reshape(-1, hkv, d)[:t])
    ref, mag = P.rotate(k, pos, [10000.0 ** (-2.0 * i / d) for i in range(d // 2)], [0] * (d // 2), d, "half")
    tol = 12 * P.EPS32 * mag
    tol = tol + (P.EPS_BF16 if dtype == torch.bfloat16 else P.EPS32) * (ref.abs() + tol)
    assert bool(((kr.double() - ref).abs() <= tol).all())
    # and straight into prompt attention and weights, by their strides
    cu = torch.tensor([0, 200, 201, 278], dtype=torch.int32, device=DEV)
    o, lse = torch.empty_like(one), torch.empty((h, t), device=DEV)
    w = torch.empty((3, hkv, 200), device=DEV)
    pa.pa_prefill(o, qr, kr, v, cu, 0.125, lse=lse)
    pa.pa_prefill_weights(w, qr, kr, lse, cu, 0.125)
    o2, lse2, w2 = torch.empty_like(o), torch.empty_like(lse), torch.empty_like(w)
    pa.pa_prefill(o2, qr.contiguous(), kr.contiguous(), v.contiguous(), cu, 0.125, lse=lse2)
    pa.pa_prefill_weights(w2, qr.contiguous(), kr.contiguous(), lse2, cu, 0.125)
    pa.pa_sync_check()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(w, w2)
