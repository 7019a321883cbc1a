"""Calls on a stream of their own, with everything the binding makes for them, against the same
calls on the current stream."""
import pytest
import torch

import paged_kv_cache_335_b200 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _case(n=4096, h=8, hkv=8, d=64, bs=16):
    g = torch.Generator(device=DEV).manual_seed(1)
    nb = n // bs
    kc, vc = (torch.randn((nb, hkv, bs, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, h, d), generator=g, device=DEV).to(torch.bfloat16)
    tables = torch.arange(nb, dtype=torch.int32, device=DEV)[None].contiguous()
    return q, kc, vc, tables, torch.tensor([n], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("raw", [False, True])
def test_a_workspace_of_a_delayed_call_is_not_given_away(raw):
    q, kc, vc, tables, ctx = _case()
    n = int(ctx)
    ref, out = torch.empty_like(q), torch.empty_like(q)
    wr, w = torch.zeros((1, 8, n), device=DEV), torch.zeros((1, 8, n), device=DEV)
    pa.pa_decode_weights(ref, wr, q, kc, vc, tables, ctx, 0.125)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    need = pa.pa_decode_weights_workspace_size(1, 8, n, kc)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(200_000_000)               # the call's kernels run long after it returns
    pa.pa_decode_weights(out, w, q, kc, vc, tables, ctx, 0.125, max_context_len=n,
                         stream=st.cuda_stream if raw else st)
    mine = [torch.full((need,), 3, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((x == 3).all()) for x in mine)
    assert torch.equal(out, ref) and torch.equal(w, wr)
    pa.pa_sync_check()


def test_lengths_are_read_behind_the_streams_work():
    q, kc, vc, tables, ctx = _case()
    n = int(ctx)
    ref, out = torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode(ref, q, kc, vc, tables, ctx, 0.125)
    late = torch.zeros_like(ctx)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(50_000_000)
        late.copy_(ctx)
    pa.pa_decode(out, q, kc, vc, tables, late, 0.125, stream=st)
    torch.cuda.synchronize()
    pa.pa_sync_check()
    assert n == 4096 and torch.equal(out, ref)
