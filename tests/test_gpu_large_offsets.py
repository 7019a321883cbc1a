"""The calls around decode where offsets pass 2^31 elements: packed rows, weights, scores, pools."""
import math

import pytest
import torch

import paged_kv_cache_335_b200 as pa
from tests import plain_forms as P
from tests.test_gpu_prefill import BF16, DEV, F32

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 60 GB")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompts(dtype):
    n, s, h, hkv, d = 1000, 270, 64, 8, 128
    t, scale = n * s, 1 / math.sqrt(d)
    x = torch.empty((t, h + 2 * hkv, d), device=DEV, dtype=dtype).normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    q, k, v = x[:, :h], x[:, h:h + hkv], x[:, h + hkv:]
    assert t * h * d > 2 ** 31
    cu = torch.arange(0, t + 1, n, dtype=torch.int32, device=DEV)
    out, lse = torch.empty((t, h, d), device=DEV, dtype=dtype), torch.empty((h, t), device=DEV)
    pa.pa_prefill(out, q, k, v, cu, scale, max_seq_len=n, lse=lse)
    stride = 1_000_000
    assert s * hkv * stride > 2 ** 31
    w = torch.full((s, hkv, stride), 7.0, device=DEV)
    pa.pa_prefill_weights(w, q, k, lse, cu, scale, max_seq_len=n)
    pa.pa_sync_check()
    for i in (0, 205, s - 1):
        a, b = i * n, (i + 1) * n
        ref, rl, mag, sabs = P.prompt_attention(q[a:b], k[a:b], v[a:b], scale)
        assert bool(((out[a:b].double() - ref).abs() <= P.attention_bound(ref, mag, sabs, d, n, dtype)).all()), i
        assert bool(((lse[:, a:b].double() - rl).abs() <= P.lse_bound(rl, sabs, d, n)).all()), i
        ref, mag = P.prompt_weights(q[a:b], k[a:b], lse[:, a:b], scale)
        tol = P.EPS32 * (mag + ref * ((h // hkv) * n + 16)) + 1e-37
        assert bool(((w[i, :, :n].double() - ref).abs() <= tol).all()), i
        assert not w[i, :, n:].any()


def test_rotary_append():
    t, h, hkv, d, bs = 270_000, 64, 8, 128, 64
    nb = 2_200_000 // bs
    x = torch.empty((t, h + 2 * hkv, d), device=DEV, dtype=BF16).normal_(generator=torch.Generator(device=DEV).manual_seed(2))
    kc, vc = (torch.zeros((nb, hkv, bs, d), device=DEV, dtype=BF16) for _ in range(2))
    assert t * h * d > 2 ** 31 and nb * hkv * bs * d > 2 ** 31
    slots = (nb * bs - 1 - 7 * torch.arange(t, device=DEV))        # over most of the pool, from its end
    pos = torch.arange(t, dtype=torch.int32, device=DEV)[None].contiguous()
    out = torch.empty((t, h, d), device=DEV, dtype=BF16)
    pa.pa_rope_append(out, x[:, :h], x[:, h:h + hkv], x[:, h + hkv:], pos, slots, kc, vc, pa.rope_desc(d))
    pa.pa_sync_check()
    freq = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    pick = torch.tensor([0, 1, 131071, t - 2, t - 1], device=DEV)
    at = slots[pick]
    for src, got in ((x[pick, :h], out[pick]), (x[pick, h:h + hkv], kc[at // bs, :, at % bs])):
        ref, mag = P.rotate(src, pos[:, pick], freq, [0] * (d // 2), d, "half")
        tol = 12 * P.EPS32 * mag
        tol = tol + P.EPS_BF16 * (ref.abs() + tol)
        assert bool(((got.double() - ref).abs() <= tol).all())
    assert torch.equal(vc[at // bs, :, at % bs], x[pick, h + hkv:])


@pytest.mark.parametrize("h,hkv", [(32, 4), (32, 32)])
def test_decode_weights(h, hkv):
    """Contexts of 600000 tokens over the same four blocks: the weights repeat every 64 tokens."""
    s, d, bs, n = 128, 64, 16, 600_000
    assert s * h * n > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(3)
    kc, vc = (torch.randn((4, hkv, bs, d), generator=g, device=DEV).to(BF16) for _ in range(2))
    q = torch.randn((s, h, d), generator=g, device=DEV).to(BF16)
    tables = (torch.arange(n // bs, device=DEV) % 4).to(torch.int32).expand(s, -1).contiguous()
    ctx = torch.full((s,), n, dtype=torch.int32, device=DEV)
    w, out = torch.zeros((s, hkv, n), device=DEV), torch.empty_like(q)
    pa.pa_decode_weights(out, w, q, kc, vc, tables, ctx, 0.125, max_context_len=n)
    pa.pa_sync_check()
    k = kc.permute(1, 0, 2, 3).reshape(hkv, 64, d).double()
    for i in (0, 70, s - 1):
        qs = q[i].double().reshape(hkv, h // hkv, d)
        sc = torch.einsum("kgd,ktd->kgt", qs, k) * 0.125
        p = (torch.softmax(sc, -1) / (n / 64)).sum(1)
        got = w[i].double().reshape(hkv, n // 64, 64)
        sabs = (torch.einsum("kgd,ktd->kgt", qs.abs(), k.abs()) * 0.125).amax()
        # sums of n weights in fp32: a thread adds at most n / 16 of them, then the threads' and
        # the partitions' sums
        rel = 2 * (d + 4) * P.EPS32 * float(sabs) + 2 * (n // 16 + 64) * P.EPS32
        assert bool(((got - p[:, None]).abs() <= p[:, None] * rel).all()), i


def test_evict():
    n, budget, recent, d, bs, hkv = 2900, 1000, 64, 128, 64, 8
    nb = 2_200_000 // bs
    kc, vc = (torch.zeros((nb, hkv, bs, d), device=DEV, dtype=torch.int8) for _ in range(2))
    assert nb * hkv * bs * d > 2 ** 31
    blocks = nb - 1 - torch.randperm(nb // 2, device=DEV)[:-(-n // bs)]   # the pool's upper half
    blocks[::2] -= nb // 2                                          # and its lower one
    rows = torch.randint(-128, 128, (len(blocks), hkv, bs, d), device=DEV, dtype=torch.int8)
    kc[blocks], vc[blocks] = rows, rows.flip(-1)
    tables = blocks.to(torch.int32)[None].contiguous()
    w = torch.rand((1, hkv, n), device=DEV)
    w_out, new = torch.empty_like(w), torch.empty((1,), dtype=torch.int32, device=DEV)
    kept = torch.empty((1, hkv, budget), dtype=torch.int32, device=DEV)
    pa.pa_evict(kc, vc, tables, torch.tensor([n], dtype=torch.int32, device=DEV), w, w_out, new, kept, budget, recent)
    pa.pa_sync_check()
    flat = rows.permute(1, 0, 2, 3).reshape(hkv, -1, d)
    for kh in range(hkv):
        want = P.evict(w[0, kh].tolist(), n, budget, recent)
        assert kept[0, kh].tolist() == want
        for cache, src in ((kc, flat), (vc, flat.flip(-1))):
            got = cache[blocks, kh].reshape(-1, d)[:budget]
            assert torch.equal(got, src[kh][torch.tensor(want, device=DEV)])
