"""The calls together, as a serving loop makes them: a packed batch of prompts is rotated into
the pool and attended to, its tokens' weights start the totals, decode steps add theirs, and
the contexts are evicted to a budget with their blocks freed, then decoded on."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_335_b200 as pa
from paged_kv_cache_335_b200.block_manager import BlockManager
from tests import plain_forms as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_decode_evict_decode(dtype):
    lens, h, hkv, d, bs = [130, 45, 200], 8, 2, 64, 16
    budget, recent, steps = 96, 16, 3
    g = torch.Generator(device=DEV).manual_seed(21)
    scale = 1 / math.sqrt(d)
    rope = pa.rope_desc(d, base=1e6, sections=[16, 8, 8])
    mgr = BlockManager(64, bs, order=np.random.default_rng(0).permutation(64))
    seqs = [mgr.new_sequence(n) for n in lens]
    kc = torch.zeros((64, hkv, bs, d), device=DEV, dtype=dtype)
    vc = torch.zeros_like(kc)

    def slots_of(seq, positions):
        return [seq.table[p // bs] * bs + p % bs for p in positions]

    # prompts
    t = sum(lens)
    qkv = torch.randn((t, h + 2 * hkv, d), generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :h], qkv[:, h:h + hkv], qkv[:, h + hkv:]
    pos = torch.tensor(np.concatenate([np.arange(n) for n in lens])[None].repeat(3, 0).copy(), dtype=torch.int32, device=DEV)
    slots = torch.tensor(sum((slots_of(s, range(n)) for s, n in zip(seqs, lens)), []), device=DEV)
    qr = torch.empty((t, h, d), device=DEV, dtype=dtype)
    pa.pa_rope_append(qr, q, k, v, pos, slots, kc, vc, rope)
    kr = torch.empty((t, hkv, d), device=DEV, dtype=dtype)
    kr.copy_(kc.transpose(1, 2).reshape(-1, hkv, d)[slots])       # the rotated keys, from the pool
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(qr), torch.empty((h, t), device=DEV)
    pa.pa_prefill(out, qr, kr, v, cu, scale, lse=lse)
    stride = 256
    weights = torch.zeros((3, hkv, stride), device=DEV)
    pa.pa_prefill_weights(weights, qr, kr, lse, cu, scale)
    pa.pa_sync_check()
    # the last row of each prompt is what decode gives for the same query over the pool
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    tables = torch.as_tensor(mgr.tables_array(seqs, 16, -1), device=DEV)
    last = torch.tensor(np.cumsum(lens) - 1, device=DEV)
    dec = torch.empty((3, h, d), device=DEV, dtype=dtype)
    pa.pa_decode(dec, qr[last].contiguous(), kc, vc, tables, ctx, scale)
    for s, n in enumerate(lens):
        a = int(cu[s])
        ref, _, mag, sabs = P.prompt_attention(qr[a:a + n], kr[a:a + n], v[a:a + n], scale)
        tol = P.attention_bound(ref, mag, sabs, d, n, dtype)[-1]
        assert bool(((dec[s].double() - ref[-1]).abs() <= tol).all())
        assert bool(((out[a + n - 1].double() - ref[-1]).abs() <= tol).all())
    # every query of a kv head's group gives its tokens a weight of one
    for s, n in enumerate(lens):
        total = weights[s].sum(-1)
        assert torch.allclose(total, torch.full_like(total, n * h / hkv), rtol=1e-3)

    # decode steps
    def step(count):
        new = torch.randn((3, h + 2 * hkv, d), generator=g, device=DEV).to(dtype)
        sl = torch.tensor([mgr.append_slot(s) for s in seqs], device=DEV)
        p = torch.tensor([[n + count for n in lens]] * 3, dtype=torch.int32, device=DEV)
        qn = torch.empty((3, h, d), device=DEV, dtype=dtype)
        pa.pa_rope_append(qn, new[:, :h], new[:, h:h + hkv], new[:, h + hkv:], p, sl, kc, vc, rope)
        c = torch.tensor([s.length for s in seqs], dtype=torch.int32, device=DEV)
        tb = torch.as_tensor(mgr.tables_array(seqs, 16, -1), device=DEV)
        o = torch.empty_like(qn)
        pa.pa_decode_weights(o, weights, qn, kc, vc, tb, c, scale)
        return o, qn, c, tb

    before = weights.sum((1, 2))
    for i in range(steps):
        o, *_ = step(i)
    pa.pa_sync_check()
    assert torch.allclose(weights.sum((1, 2)) - before, torch.full((3,), float(steps * h), device=DEV), rtol=1e-3)

    # evict, free the blocks behind the budget, and decode on
    c = torch.tensor([s.length for s in seqs], dtype=torch.int32, device=DEV)
    tb = torch.as_tensor(mgr.tables_array(seqs, 16, -1), device=DEV)
    copies = [mgr.unshare(s) for s in seqs]
    assert copies == [0, 0, 0]
    kept = torch.empty((3, hkv, budget), dtype=torch.int32, device=DEV)
    new_c = torch.empty_like(c)
    kw, vw = kc.clone(), vc.clone()
    pa.pa_evict(kc, vc, tb, c, weights, weights, new_c, kept, budget, recent)
    pa.pa_sync_check()
    free = mgr.num_free
    for s, n in zip(seqs, new_c.tolist()):
        mgr.truncate(s, n)
    assert [s.length for s in seqs] == new_c.tolist() == [96, 48, 96]
    assert mgr.num_free > free
    o, qn, c2, tb2 = step(steps)
    pa.pa_sync_check()
    # the same query over the kept tokens, gathered from the pool before the eviction
    for s in range(3):
        n = int(c2[s])
        rows = [x.permute(0, 2, 1, 3).reshape(-1, hkv, d) for x in (kw, vw, kc, vc)]
        old = tb[s].long().clamp(min=0)[:, None] * bs + torch.arange(bs, device=DEV)
        new = tb2[s].long().clamp(min=0)[:, None] * bs + torch.arange(bs, device=DEV)
        for kh in range(hkv):
            idx = old.flatten()[kept[s, kh, :n - 1].long()]
            at = new.flatten()[n - 1]
            kk = torch.cat([rows[0][idx, kh], rows[2][at, kh][None]]).double()
            vv = torch.cat([rows[1][idx, kh], rows[3][at, kh][None]]).double()
            qg = qn[s, kh * (h // hkv):(kh + 1) * (h // hkv)].double()
            p = torch.softmax(qg @ kk.T * scale, -1)
            ref, mag = p @ vv, p @ vv.abs()
            sabs = (qg.abs() @ kk.abs().T * scale).amax(1)
            got = o[s, kh * (h // hkv):(kh + 1) * (h // hkv)].double()
            tol = P.attention_bound(ref, mag, sabs, d, n, dtype)
            assert bool(((got - ref).abs() <= tol).all())


def _step_state(seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s, h, hkv, d, bs = 5, 16, 2, 128, 16
    kc, vc = (torch.randn((160, hkv, bs, d), generator=g, device=DEV).to(dtype) for _ in range(2))
    qkv = torch.randn((s, h + 2 * hkv, d), generator=g, device=DEV).to(dtype)
    tables = torch.randperm(160, generator=g, device=DEV)[:s * 30].reshape(s, 30).int()
    ctx = torch.tensor([401, 17, 450, 300, 64], dtype=torch.int32, device=DEV)
    slots = (tables.gather(1, ((ctx - 1) // bs).long()[:, None])[:, 0] * bs + (ctx - 1) % bs).long()
    st = dict(kc=kc, vc=vc, qkv=qkv, tables=tables, ctx=ctx, slots=slots, pos=(ctx - 1)[None].repeat(3, 1).contiguous(),
              q=torch.empty((s, h, d), device=DEV, dtype=dtype), out=torch.empty((s, h, d), device=DEV, dtype=dtype),
              w=torch.rand((s, hkv, 480), generator=g, device=DEV), new=torch.zeros_like(ctx),
              kept=torch.zeros((s, hkv, 256), dtype=torch.int32, device=DEV))
    st["ws"] = torch.empty(pa.pa_decode_weights_workspace_size(s, h, 480, kc), dtype=torch.uint8, device=DEV)
    return st


def _step(st, stream=None):
    q, k, v = st["qkv"][:, :16], st["qkv"][:, 16:18], st["qkv"][:, 18:]
    pa.pa_rope_append(st["q"], q, k, v, st["pos"], st["slots"], st["kc"], st["vc"],
                      pa.rope_desc(128, sections=[32, 16, 16]), stream=stream)
    pa.pa_decode_weights(st["out"], st["w"], st["q"], st["kc"], st["vc"], st["tables"], st["ctx"], 0.09,
                         max_context_len=480, workspace=st["ws"], stream=stream)
    pa.pa_evict(st["kc"], st["vc"], st["tables"], st["ctx"], st["w"], st["w"], st["new"], st["kept"], 256, 40,
                max_context_len=480, stream=stream)


def _same(a, b):
    return all(torch.equal(a[k], b[k]) for k in ("kc", "vc", "q", "out", "w", "new", "kept"))


def test_captured_step_replays_with_new_inputs():
    want = _step_state(32)
    _step(want)
    st = _step_state(31)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(st)
    for k, v in _step_state(32).items():
        st[k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    pa.pa_sync_check()
    assert _same(st, want)


def test_two_steps_at_once():
    """Two streams with states and workspaces of their own, and prompts beside them."""
    want = [_step_state(s) for s in (33, 34)]
    for st in want:
        _step(st)
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (torch.randn((700, h, 64), generator=g, device=DEV).bfloat16() for h in (6, 2, 2))
    cu = torch.tensor([0, 300, 700], dtype=torch.int32, device=DEV)
    ref, ref_l, ref_w = torch.empty_like(q), torch.empty((6, 700), device=DEV), torch.empty((2, 2, 400), device=DEV)
    pa.pa_prefill(ref, q, k, v, cu, 0.125, max_seq_len=400, lse=ref_l)
    pa.pa_prefill_weights(ref_w, q, k, ref_l, cu, 0.125, max_seq_len=400)
    sts = [_step_state(s) for s in (33, 34)]
    outs = [[torch.empty_like(x) for x in (ref, ref_l, ref_w)] for _ in sts]
    streams = [torch.cuda.Stream() for _ in sts]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, o, stream in zip(sts, outs, streams):
            pa.pa_prefill(o[0], q, k, v, cu, 0.125, max_seq_len=400, lse=o[1], stream=stream)
            pa.pa_prefill_weights(o[2], q, k, o[1], cu, 0.125, max_seq_len=400, stream=stream)
    for st, stream in zip(sts, streams):
        _step(st, stream=stream)
    torch.cuda.synchronize()
    pa.pa_sync_check()
    assert all(_same(a, b) for a, b in zip(sts, want))
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, (ref, ref_l, ref_w)))
