"""Calls of different sizes from two host threads at once, each on its own stream: a launch must
not depend on what another thread's call has set for the same kernel. (The C entries are called
directly, in tight loops, with little work for the GPU, so that the calls overlap.)"""
import ctypes
import threading

import pytest
import torch

import paged_kv_cache_335_b200 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _at_once(entry, calls, times):
    """entry(*call) `times` times for every call, each in a thread of its own; the status codes
    that are not PA_OK."""
    codes = []
    start = threading.Barrier(len(calls))

    def work(call):
        start.wait()
        codes.extend(rc for rc in (entry(*call) for _ in range(times)) if rc != pa.PA_OK)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return codes


@pytest.mark.parametrize("longest", [(30000, 5000), (90000, 60000), (4096, 100)])
def test_evictions_of_different_lengths(longest):
    """The same three tokens, within the budget, under different bounds on the context."""
    calls, kept = [], []
    keep = []
    for n in longest:
        st = torch.cuda.Stream()
        kc, vc = (torch.zeros((8, 1, 64, 64), device=DEV, dtype=torch.int8) for _ in range(2))
        blocks = -(-n // 64)
        tables = torch.zeros((1, blocks), dtype=torch.int32, device=DEV)
        ctx = torch.tensor([3], dtype=torch.int32, device=DEV)
        w = torch.ones((1, 1, n), device=DEV)
        new, k = torch.zeros_like(ctx), torch.full((1, 1, n), -7, dtype=torch.int32, device=DEV)
        w_out = torch.empty_like(w)
        desc = pa.cache_desc(kc)
        vp = lambda t: ctypes.c_void_p(t.data_ptr())
        calls.append((vp(kc), vp(vc), vp(tables), blocks, vp(ctx), n, 1, vp(w), vp(w_out), n, vp(new), vp(k), n, 0,
                      ctypes.byref(desc), ctypes.c_void_p(st.cuda_stream)))
        kept.append(k)
        keep.append((st, kc, vc, tables, ctx, w, w_out, new, desc))
    torch.cuda.synchronize()
    codes = _at_once(pa.load_library().pa_evict, calls, 20000)
    assert not codes, f"{len(codes)} calls failed, the first with {codes[0]}: {pa.load_library().pa_get_last_error()}"
    pa.pa_sync_check()
    for k in kept:
        assert k[0, 0, :4].tolist() == [0, 1, 2, -1]


def test_fp32_prompts_of_different_sizes():
    calls, outs, refs, keep = [], [], [], []
    for h in (1, 200):                                   # up to and above two CTAs per SM in all
        st = torch.cuda.Stream()
        g = torch.Generator(device=DEV).manual_seed(h)
        q, k, v = (torch.randn((64, h, 64), generator=g, device=DEV) for _ in range(3))
        cu = torch.tensor([0, 64], dtype=torch.int32, device=DEV)
        ref, out = torch.empty_like(q), torch.zeros_like(q)
        pa.pa_prefill(ref, q, k, v, cu, 0.125, max_seq_len=64)
        vp = lambda t: ctypes.c_void_p(t.data_ptr())
        calls.append((vp(out), vp(q), vp(k), vp(v), h * 64, h * 64, h * 64, vp(cu), 1, 64, 64, h, h, 64, pa.PA_F32,
                      0.125, ctypes.c_void_p(0), ctypes.c_void_p(st.cuda_stream)))
        outs.append(out)
        refs.append(ref)
        keep.append((st, q, k, v, cu))
    torch.cuda.synchronize()
    codes = _at_once(pa.load_library().pa_prefill, calls, 20000)
    assert not codes, f"{len(codes)} calls failed, the first with {codes[0]}"
    pa.pa_sync_check()
    for a, b in zip(outs, refs):
        assert torch.equal(a, b)
