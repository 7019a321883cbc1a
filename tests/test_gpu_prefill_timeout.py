"""Prompt attention's and prompt weights' pipeline waits are bounded: with one tile left
unloaded on purpose (pa_test_skip_load) every role of the kernel gives up, it terminates,
pa_sync_check reports PA_ERR_TIMEOUT, and the next call is right."""
import time

import pytest
import torch

import paged_kv_cache_335_b200 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("h,hkv,d", [(2, 1, 64), (3, 3, 128)])
@pytest.mark.parametrize("position", [0, 1, 3])
def test_skipped_tile_times_out_then_recovers(h, hkv, d, position):
    n = 500
    g = torch.Generator(device=DEV).manual_seed(position)
    q, k, v = (torch.randn((n, x, d), generator=g, device=DEV).bfloat16() for x in (h, hkv, hkv))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    lse = torch.empty((h, n), device=DEV)
    outs = [torch.empty_like(q) for _ in range(3)]
    ws = [torch.empty((1, hkv, n), device=DEV) for _ in range(3)]
    pa.pa_prefill(outs[0], q, k, v, cu, 0.1, max_seq_len=n, lse=lse)
    pa.pa_prefill_weights(ws[0], q, k, lse, cu, 0.1, max_seq_len=n)
    pa.pa_sync_check()
    lib = pa.load_library()
    for call in (lambda i: pa.pa_prefill(outs[i], q, k, v, cu, 0.1, max_seq_len=n),
                 lambda i: pa.pa_prefill_weights(ws[i], q, k, lse, cu, 0.1, max_seq_len=n)):
        lib.pa_test_skip_load(position)
        try:
            t0 = time.time()
            call(1)
            with pytest.raises(pa.PAError) as e:
                pa.pa_sync_check()
            assert e.value.code == pa.PA_ERR_TIMEOUT
            assert time.time() - t0 < 30
        finally:
            lib.pa_test_skip_load(-1)
        pa.pa_sync_check()                              # the status was cleared
        call(2)
        pa.pa_sync_check()
    assert torch.equal(outs[2], outs[0]) and torch.equal(ws[2], ws[0])
