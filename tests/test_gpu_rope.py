"""pa_rope_append / pa_rope_append_quant against the rotation in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_335_b200 as pa
from tests import plain_forms as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _case(t, h, hkv, d, dtype, seed, far=100000, axes=1, bs=16, cache=None, pad=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    qkv = torch.randn((t, h + 2 * hkv, d), generator=g, device=DEV).to(dtype)
    nb = -(-t // bs) + 2
    kc = torch.zeros((nb, hkv, bs, d), device=DEV).to(cache or dtype)
    slots = rng.permutation(nb * bs)[:t].astype(np.int64)
    if pad and t > 2:
        slots[1::7] = -1
    pos = rng.integers(-far // 10, far, (axes, t), dtype=np.int32)
    return dict(q=qkv[:, :h], k=qkv[:, h:h + hkv], v=qkv[:, h + hkv:], kc=kc, vc=kc.clone(),
                slots=torch.as_tensor(slots, device=DEV), pos=torch.as_tensor(pos, device=DEV),
                out=torch.full((t, h, d), float("nan"), device=DEV, dtype=dtype))


def _freq(rotary, base=1e6):
    return [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]


def _rows(cache):
    nb, hkv, bs, d = cache.shape
    raw = cache.view(torch.uint8) if cache.element_size() == 1 else cache
    return raw.transpose(1, 2).reshape(nb * bs, hkv, d)


def _bound(ref, mag, dtype):
    # angle: half-turns rounded to fp32 (pi EPS32 radians), sine and cosine to 2 steps, two
    # products and a sum: below 12 EPS32 of |a| + |b|; then the result's own rounding
    tol = 12 * P.EPS32 * mag
    return tol + (P.EPS_BF16 if dtype == torch.bfloat16 else P.EPS32) * (ref.abs() + tol)


@pytest.mark.parametrize("t,h,hkv,d,rotary,axes,pairs,dtype", [
    (1, 8, 2, 128, 128, 1, "half", torch.bfloat16),
    (5, 5, 5, 64, 64, 2, "adjacent", torch.bfloat16),
    (8, 64, 8, 128, 48, 3, "half", torch.bfloat16),
    (37, 3, 1, 64, 16, 4, "adjacent", torch.float32),
    (700, 8, 4, 128, 64, 3, "half", torch.float32),
    (1185, 40, 40, 128, 128, 3, "adjacent", torch.bfloat16),   # the last CTA holds one token
    (2049, 16, 2, 64, 48, 2, "half", torch.bfloat16),
])
def test_rope_append(t, h, hkv, d, rotary, axes, pairs, dtype):
    c = _case(t, h, hkv, d, dtype, seed=t + h, axes=axes)
    half = rotary // 2
    sections = [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    rope = pa.rope_desc(rotary, inv_freq=_freq(rotary), sections=sections, pairs=pairs, mscale=1.25)
    pa.pa_rope_append(c["out"], c["q"], c["k"], c["v"], c["pos"], c["slots"], c["kc"], c["vc"], rope)
    pa.pa_sync_check()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for x, got in ((c["q"], c["out"]), (c["k"], None)):
        ref, mag = P.rotate(x, c["pos"], _freq(rotary), axis, rotary, pairs, 1.25)
        keep = torch.arange(t, device=DEV)
        if got is None:
            keep = torch.nonzero(c["slots"] >= 0)[:, 0]
            got = _rows(c["kc"])[c["slots"][keep]]
        err = (got.double() - ref[keep]).abs()
        assert bool((err <= _bound(ref, mag, dtype)[keep]).all()), float(err.max())
        assert torch.equal(got[..., rotary:], x[keep][..., rotary:])     # copied, not computed
    keep = torch.nonzero(c["slots"] >= 0)[:, 0]
    assert torch.equal(_rows(c["vc"])[c["slots"][keep]], c["v"][keep])
    other = torch.ones(_rows(c["kc"]).shape[0], dtype=torch.bool, device=DEV)
    other[c["slots"][keep]] = False
    assert not _rows(c["kc"])[other].any() and not _rows(c["vc"])[other].any()


def test_far_positions_keep_fp32_accuracy():
    c = _case(64, 2, 1, 64, torch.float32, seed=3)
    c["pos"] = torch.tensor([[2 ** 31 - 1 - 977 * i if i % 2 else -2 ** 31 + 31 * i for i in range(64)]],
                            dtype=torch.int32, device=DEV)
    freq = _freq(64, 10000.0)
    pa.pa_rope_append(c["out"], c["q"], c["k"], c["v"], c["pos"], c["slots"], c["kc"], c["vc"],
                      pa.rope_desc(64, inv_freq=freq))
    pa.pa_sync_check()
    # position x frequency beyond 2^31: the reference angle itself needs more than 64-bit floats
    import decimal
    decimal.getcontext().prec = 60
    tau = decimal.Decimal("6.28318530717958647692528676655900576839433879875021")
    ang = torch.tensor([[float((decimal.Decimal(p) * decimal.Decimal(f)) % tau) for f in freq]
                        for p in c["pos"][0].tolist()], dtype=torch.float64, device=DEV)[:, None]
    a, b = c["q"][..., :32].double(), c["q"][..., 32:].double()
    ref = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    mag = torch.cat([a.abs() + b.abs()] * 2, -1)
    # a frequency held to 2^-64 turns: position 2^31 moves the angle by at most 2^-33 turns
    tol = _bound(ref, mag, torch.float32) + mag * 2.0 ** -33 * 6.3
    assert bool(((c["out"].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("t,h,hkv,d,rotary,pairs", [(3, 8, 8, 64, 48, "half"),
                                                    (1300, 16, 2, 128, 128, "adjacent")])
def test_rope_append_quant(fmt, t, h, hkv, d, rotary, pairs):
    c = _case(t, h, hkv, d, torch.bfloat16, seed=t, cache=fmt, axes=2)
    ks = torch.linspace(0.01, 0.03, hkv, device=DEV)
    vs = torch.linspace(0.004, 0.02, hkv, device=DEV)                    # some values saturate
    half = rotary // 2
    pa.pa_rope_append_quant(c["out"], c["q"], c["k"], c["v"], c["pos"], c["slots"], c["kc"], c["vc"],
                            ks, vs, pa.rope_desc(rotary, inv_freq=_freq(rotary),
                                                 sections=[half - 3, 3], pairs=pairs))
    pa.pa_sync_check()
    axis = [0] * (half - 3) + [1] * 3
    keep = torch.nonzero(c["slots"] >= 0)[:, 0]
    ref, mag = P.rotate(c["k"], c["pos"], _freq(rotary), axis, rotary, pairs)
    for cache, x, m, s in ((c["kc"], ref, mag, ks), (c["vc"], c["v"].double(), c["v"].double().abs() * 0, vs)):
        y = (x / s.double()[:, None])[keep]
        slack = (m * 12 * P.EPS32 / s.double()[:, None])[keep] + y.abs() * P.EPS32
        got = _rows(cache)[c["slots"][keep]].view(fmt).double()
        if fmt == torch.int8:
            y = y.clamp(-127, 127)
            tol = 0.5 + slack
        else:
            y = y.clamp(-448, 448)
            tol = torch.maximum(y.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, device=DEV).double()) + slack
        assert bool(((got - y).abs() <= tol).all())
    # v is not turned: its codes are the quantising append's, bit for bit
    kc2, vc2 = torch.zeros_like(c["kc"]), torch.zeros_like(c["vc"])
    pa.pa_kv_append_quant(c["k"].contiguous(), c["v"].contiguous(), c["slots"], kc2, vc2, ks, vs)
    assert torch.equal(c["vc"].view(torch.uint8), vc2.view(torch.uint8))


def test_without_queries_and_bad_slots():
    c = _case(40, 4, 2, 128, torch.bfloat16, seed=9)
    empty = torch.empty((40, 0, 128), device=DEV, dtype=torch.bfloat16)
    rope = pa.rope_desc(128)
    before = c["kc"].clone()
    c["slots"][5] = before.shape[0] * 16                                  # one past the pool
    pa.pa_rope_append(empty, empty.clone(), c["k"], c["v"], c["pos"], c["slots"], c["kc"], c["vc"], rope)
    with pytest.raises(pa.PAError) as e:
        pa.pa_sync_check()
    assert e.value.code == pa.PA_ERR_BAD_INDEX
    keep = torch.nonzero((c["slots"] >= 0) & (c["slots"] < before.shape[0] * 16))[:, 0]
    assert torch.equal(_rows(c["vc"])[c["slots"][keep]], c["v"][keep])
    pa.pa_sync_check()


def test_position_zero_is_the_plain_append():
    c = _case(300, 4, 4, 64, torch.bfloat16, seed=11)
    c["pos"].zero_()
    pa.pa_rope_append(c["out"], c["q"], c["k"], c["v"], c["pos"], c["slots"], c["kc"], c["vc"],
                      pa.rope_desc(64))
    kc2, vc2 = torch.zeros_like(c["kc"]), torch.zeros_like(c["vc"])
    pa.pa_kv_append(c["k"].contiguous(), c["v"].contiguous(), c["slots"], kc2, vc2)
    assert torch.equal(c["out"], c["q"]) and torch.equal(c["kc"], kc2) and torch.equal(c["vc"], vc2)
