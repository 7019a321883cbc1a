"""Refusals of the calls around decode: the host-side checks answer without a GPU."""
import ctypes

import pytest

import paged_kv_cache_335_b200 as pa
from paged_kv_cache_335_b200 import build as pbuild

I, U, A, D = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_ERR_ALIGN, pa.PA_ERR_DTYPE


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.load_library()


def _p(x):
    return ctypes.c_void_p(x)


def _desc(**kw):
    d = dict(num_blocks=64, num_kv_heads=4, block_size=16, head_dim=128, dtype=pa.PA_BF16)
    d.update(kw)
    return pa.pa_cache_desc(**d)


def _rope(lib, quant=False, desc=None, rope=None, tokens=0, heads=8, qs=1024, ks=512, vs=512, ptr=1 << 20,
          out=1 << 30, slots=None, scale=16):
    desc = desc or _desc(dtype=pa.PA_INT8 if quant else pa.PA_BF16)
    rope = rope or pa.rope_desc(128)
    mid = (_p(scale), _p(scale)) if quant else ()
    f = lib.pa_rope_append_quant if quant else lib.pa_rope_append
    rc = f(_p(out), _p(ptr), _p(ptr), _p(ptr), qs, ks, vs, _p(16), _p(slots or 16), tokens, heads, _p(16), _p(16),
           *mid, ctypes.byref(desc), ctypes.byref(rope), None)
    if rc:
        assert lib.pa_get_last_error()
    return rc


def _bad_rope(**kw):
    r = pa.rope_desc(128)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def test_rope_refusals(lib):
    assert _rope(lib) == pa.PA_OK                                     # no tokens: nothing to do
    assert _rope(lib, quant=True) == pa.PA_OK
    assert _rope(lib, desc=_desc(dtype=pa.PA_INT8)) == D
    assert _rope(lib, quant=True, desc=_desc()) == D
    assert _rope(lib, quant=True, scale=0) == I
    for rd in (0, 8, 24, 144, -16):
        assert _rope(lib, rope=_bad_rope(rotary_dim=rd)) == U
    assert _rope(lib, desc=_desc(head_dim=64)) == U                   # rotary_dim 128 of 64
    assert _rope(lib, rope=_bad_rope(pairs=2)) == I
    assert _rope(lib, rope=_bad_rope(num_axes=0)) == I
    assert _rope(lib, rope=_bad_rope(num_axes=5)) == I
    assert _rope(lib, rope=_bad_rope(mscale=float("nan"))) == I
    r = pa.rope_desc(128)
    r.axis[63] = 1                                                    # one axis only
    assert _rope(lib, rope=r) == I
    r = pa.rope_desc(128)
    r.inv_freq[5] = float("inf")
    assert _rope(lib, rope=r) == I
    assert _rope(lib, tokens=-1) == I
    assert _rope(lib, heads=-1) == I
    assert _rope(lib, tokens=2, ptr=0) == I
    assert _rope(lib, tokens=2, ptr=(1 << 20) + 8) == A
    assert _rope(lib, tokens=2, slots=20) == A
    assert _rope(lib, tokens=2, qs=1016) == I                         # below one token
    assert _rope(lib, tokens=2, ks=516) == A                          # not a multiple of 16 bytes
    assert _rope(lib, tokens=2, vs=(1 << 36) + 8) == A
    assert _rope(lib, tokens=2, out=(1 << 20) + 2048) == I            # q_out in q


def _prefill(lib, weights=False, q=1 << 20, k=1 << 24, out=1 << 30, cu=16, seqs=1, total=64, most=64, h=8, hkv=2,
             d=128, dtype=pa.PA_BF16, scale=0.1, qs=1024, ks=256, lse=16, wstride=64, last=0):
    if weights:
        rc = lib.pa_prefill_weights(_p(out), wstride, _p(q), _p(k), qs, ks, _p(lse), _p(cu), seqs, total, most, h,
                                    hkv, d, dtype, scale, last, None)
    else:
        rc = lib.pa_prefill(_p(out), _p(q), _p(k), _p(k), qs, ks, ks, _p(cu), seqs, total, most, h, hkv, d, dtype,
                            scale, _p(lse), None)
    if rc:
        assert lib.pa_get_last_error()
    return rc


@pytest.mark.parametrize("weights", [False, True])
def test_prefill_refusals(lib, weights):
    f = lambda **kw: _prefill(lib, weights, **kw)  # noqa: E731
    assert f(seqs=0) == pa.PA_OK
    assert f(dtype=pa.PA_FP8_E4M3) == D
    assert f(d=96) == U
    assert f(h=7) == I
    assert f(hkv=0) == I
    assert f(seqs=-1) == I
    assert f(total=-1) == I
    assert f(most=-1) == I
    assert f(scale=float("inf")) == I
    assert f(qs=1000) == I
    assert f(ks=260) == A
    assert f(q=0) == I
    assert f(cu=0) == I
    assert f(q=(1 << 20) + 8) == A
    assert f(cu=18) == A
    assert f(lse=18) == A
    if weights:
        assert f(wstride=63) == I
        assert f(last=-1) == I
        assert f(out=0) == I
        assert f(lse=0) == I
    else:
        assert f(total=0) == pa.PA_OK
        assert f(out=(1 << 20) + 1024) == I                           # out in q


def _dw(lib, quant=False, desc=None, weights=16, stride=128, max_ctx=100, ws=None, ws_bytes=None, heads=4, seqs=2):
    desc = desc or _desc(dtype=pa.PA_INT8 if quant else pa.PA_BF16)
    p = _p(256)
    need = lib.pa_decode_weights_workspace_size(seqs, heads, max_ctx, ctypes.byref(desc), 0)
    mid = (p, p) if quant else ()
    f = lib.pa_decode_weights_quant if quant else lib.pa_decode_weights
    return f(p, _p(weights), stride, p, p, p, *mid, p, 8, p, max_ctx, seqs, heads, 0.1, ctypes.byref(desc), 0,
             _p(256 if ws is None else ws), need if ws_bytes is None else need + ws_bytes, None)


@pytest.mark.parametrize("quant", [False, True])
def test_decode_weights_refusals(lib, quant):
    assert _dw(lib, quant, seqs=0) == pa.PA_OK
    assert _dw(lib, quant, weights=0) == I
    assert _dw(lib, quant, weights=18) == A
    assert _dw(lib, quant, stride=99) == I
    assert _dw(lib, quant, ws=0) == pa.PA_ERR_WORKSPACE
    assert _dw(lib, quant, ws_bytes=-1) == pa.PA_ERR_WORKSPACE
    assert _dw(lib, quant, ws=128) == A
    assert _dw(lib, quant, heads=6) == I
    assert _dw(lib, quant, max_ctx=129, stride=200) == I              # past the tables
    assert _dw(lib, quant, desc=_desc(dtype=pa.PA_BF16 if quant else pa.PA_INT8)) == D


def test_decode_weights_workspace(lib):
    """pa_decode's workspace, a score per (sequence, head, token) and a pair per partition."""
    desc = _desc(num_kv_heads=8)
    base = lib.pa_decode_workspace_size(8, 64, 32768, ctypes.byref(desc), 512)
    assert lib.pa_decode_weights_workspace_size(8, 64, 32768, ctypes.byref(desc), 512) == \
        base + 8 * 64 * 32768 * 4 + 8 * 64 * 64 * 8
    assert lib.pa_decode_weights_workspace_size(8, 63, 32768, ctypes.byref(desc), 0) == 0


def _evict(lib, desc=None, kc=16, ptr=16, w=1 << 20, wo=1 << 24, new=64, stride=1024, max_ctx=128, seqs=2,
           budget=64, recent=8, tstride=64):
    desc = desc or _desc()
    rc = lib.pa_evict(_p(kc), _p(kc), _p(ptr), tstride, _p(ptr), max_ctx, seqs, _p(w), _p(wo), stride, _p(new),
                      _p(ptr), budget, recent, ctypes.byref(desc), None)
    if rc:
        assert lib.pa_get_last_error()
    return rc


def test_evict_refusals(lib):
    assert _evict(lib, seqs=0) == pa.PA_OK
    assert _evict(lib, budget=0) == I
    assert _evict(lib, recent=-1) == I
    assert _evict(lib, recent=65) == I
    assert _evict(lib, seqs=-1) == I
    assert _evict(lib, max_ctx=-1) == I
    assert _evict(lib, stride=127) == I
    assert _evict(lib, budget=1025) == I
    assert _evict(lib, tstride=7) == I
    assert _evict(lib, kc=0) == I
    assert _evict(lib, kc=24) == A
    assert _evict(lib, ptr=18) == A
    assert _evict(lib, new=16) == I                                   # context_lens itself
    assert _evict(lib, wo=(1 << 20) + 4) == I                         # shifted onto the weights
    assert _evict(lib, desc=_desc(head_dim=96)) == U
    most = lib.pa_evict_max_context()
    assert most >= 1 << 19
    assert _evict(lib, max_ctx=most + 1, stride=1 << 20, tstride=1 << 16) == U


def test_rope_desc_checks():
    with pytest.raises(ValueError):
        pa.rope_desc(130)
    with pytest.raises(ValueError):
        pa.rope_desc(64, sections=[16, 8])
    with pytest.raises(ValueError):
        pa.rope_desc(64, inv_freq=[1.0])
    with pytest.raises(ValueError):
        pa.rope_desc(64, pairs="both")
    r = pa.rope_desc(64, sections=[16, 8, 8], pairs="adjacent")
    assert r.num_axes == 3 and list(r.axis[:32]) == [0] * 16 + [1] * 8 + [2] * 8
    assert r.inv_freq[0] == 1.0 and r.pairs == pa.PA_ROPE_ADJACENT


def test_python_needs_cuda_tensors():
    import torch
    x = torch.zeros((4, 2, 64))
    with pytest.raises(ValueError):
        pa.pa_prefill(x, x, x, x, torch.tensor([0, 4], dtype=torch.int32), 0.1, max_seq_len=4)
