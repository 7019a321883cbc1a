"""pa_prefill and pa_prefill_weights against causal attention in 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_335_b200 as pa
from tests import plain_forms as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _inputs(lens, h, hkv, d, dtype, seed, front=0, behind=0, packed=True):
    """Packed prompts; `front` / `behind` rows of no prompt around them hold NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = front + sum(lens) + behind
    x = torch.randn((t, h + 2 * hkv, d), generator=g, device=DEV).to(dtype)
    if front:
        x[:front] = float("nan")
    if behind:
        x[t - behind:] = float("nan")
    q, k, v = x[:, :h], x[:, h:h + hkv], x[:, h + hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = [front]
    for n in lens:
        cu.append(cu[-1] + n)
    return q, k, v, cu, torch.tensor(cu, dtype=torch.int32, device=DEV)


def _check(lens, h, hkv, d, dtype, scale, q, k, v, cu, out, lse):
    for s, n in enumerate(lens):
        if n == 0:
            continue
        a, b = cu[s], cu[s + 1]
        ref, rl, mag, sabs = P.prompt_attention(q[a:b], k[a:b], v[a:b], scale)
        err = (out[a:b].double() - ref).abs()
        tol = P.attention_bound(ref, mag, sabs, d, n, dtype)
        assert bool((err <= tol).all()), f"prompt {s} ({n}): {float((err - tol).max()):.2e} above the bound"
        le = (lse[:, a:b].double() - rl).abs()
        assert bool((le <= P.lse_bound(rl, sabs, d, n)).all()), f"prompt {s}: lse off by {float(le.max()):.2e}"


RAGGED = [
    ([1], 1, 1, 128),
    ([5, 0, 1, 127, 128, 129, 2], 4, 2, 128),
    ([255, 256, 257, 1, 0], 8, 1, 128),
    ([300, 77], 5, 5, 64),
    ([640, 513], 10, 2, 64),                      # groups of five: odd row blocks
    ([1, 1, 1, 1, 1], 16, 2, 64),
    ([1100], 6, 2, 128),
    ([64] * 40, 2, 2, 128),                       # more prompts than a warp has lanes
    ([2300, 17], 3, 1, 64),                       # heads of a group in two halves, 1 and 2
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,h,hkv,d", RAGGED)
def test_prefill(lens, h, hkv, d, dtype):
    scale = 1 / math.sqrt(d)
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=sum(lens) + h, front=3, behind=9)
    out = torch.full(q.shape, 7.0, device=DEV, dtype=dtype)
    lse = torch.full((h, q.shape[0]), 7.0, device=DEV)
    pa.pa_prefill(out, q, k, v, cut, scale, max_seq_len=max(lens), lse=lse)
    pa.pa_sync_check()
    _check(lens, h, hkv, d, dtype, scale, q, k, v, cu, out, lse)
    rest = torch.ones(q.shape[0], dtype=torch.bool, device=DEV)
    rest[cu[0]:cu[-1]] = False
    assert bool((out[rest] == 7).all()) and bool((lse[:, rest] == 7).all())   # rows of no prompt


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.5])
def test_scales(dtype, scale):
    """A negative scale turns the order of the scores; 1.5 makes the softmax near one-hot."""
    lens, h, hkv, d = [300, 140], 4, 2, 128
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=5)
    out, lse = torch.empty_like(q).contiguous(), torch.empty((h, q.shape[0]), device=DEV)
    pa.pa_prefill(out, q, k, v, cut, scale, lse=lse)
    pa.pa_sync_check()
    _check(lens, h, hkv, d, dtype, scale, q, k, v, cu, out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_growing_scores_move_the_reference(dtype):
    """Keys that grow along the prompt: the running maximum rises in every tile."""
    lens, h, hkv, d = [900], 2, 1, 64
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=6, packed=False)
    q.fill_(0.5)
    k.copy_((torch.arange(900, device=DEV) / 30.0)[:, None, None].expand_as(k) * 0.5)
    out, lse = torch.empty_like(q), torch.empty((h, 900), device=DEV)
    pa.pa_prefill(out, q, k, v, cut, 0.125, lse=lse)
    pa.pa_sync_check()
    _check(lens, h, hkv, d, dtype, 0.125, q, k, v, cu, out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), torch.finfo(BF16).min])
@pytest.mark.parametrize("at", [0, 130, 200, 383])
def test_masked_rows_hold_anything(dtype, value, at):
    """A row's keys and values reach no earlier query, bit for bit, whatever they hold, and the
    queries from it on see them."""
    lens, h, hkv, d = [384, 200], 4, 2, 128
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=8, packed=False)
    ref, ref_l = torch.empty_like(q), torch.empty((h, q.shape[0]), device=DEV)
    pa.pa_prefill(ref, q, k, v, cut, 0.1, lse=ref_l)
    out, lse = torch.empty_like(q), torch.empty_like(ref_l)
    bad_k, bad_v = k.clone(), v.clone()
    bad_v[at, :, ::3] = value
    pa.pa_prefill(out, q, k, bad_v, cut, 0.1, lse=lse)
    pa.pa_sync_check()
    assert torch.equal(out[:at], ref[:at]) and torch.equal(out[384:], ref[384:])
    assert torch.equal(lse, ref_l)                                # v has no part in it
    touched = out[at:384].float()
    if value != torch.finfo(BF16).min:
        assert not bool(torch.isfinite(touched[..., ::3]).any())
        if value == float("inf"):
            assert bool((touched[..., ::3] == value).all())
    keep = [i for i in range(d) if i % 3]
    assert torch.equal(out[at:384][..., keep], ref[at:384][..., keep])   # the other columns
    bad_k[at] = value
    pa.pa_prefill(out, q, bad_k, v, cut, 0.1, lse=lse)
    pa.pa_sync_check()
    assert torch.equal(out[:at], ref[:at]) and torch.equal(out[384:], ref[384:])
    assert torch.equal(lse[:, :at], ref_l[:, :at]) and torch.equal(lse[:, 384:], ref_l[:, 384:])
    if value != value:
        assert bool(torch.isnan(out[at:384]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scores_of_minus_infinity(dtype):
    """Keys whose scores are -infinity have no weight, also where they fill the first tiles; a row
    of nothing else has an lse of -infinity."""
    lens, h, hkv, d = [300], 2, 1, 64
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=16, packed=False)
    q.abs_().add_(0.1)
    dead = list(range(0, 140)) + [200]
    k[dead] = float("-inf")
    out, lse = torch.empty_like(q), torch.empty((h, 300), device=DEV)
    pa.pa_prefill(out, q, k, v, cut, 0.125, lse=lse)
    pa.pa_sync_check()
    assert bool((lse[:, :140] == -math.inf).all())
    live = [i for i in range(300) if i not in dead]
    ref, rl, mag, sabs = P.prompt_attention(q[live], k[live], v[live], 0.125)
    tol = P.attention_bound(ref, mag, sabs, d, 300, dtype)
    assert bool(((out[live].double() - ref).abs() <= tol).all())
    assert bool(((lse[:, live].double() - rl).abs() <= P.lse_bound(rl, sabs, d, 300)).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompts_do_not_depend_on_the_batch(dtype):
    lens, h, hkv, d = [129, 300, 64, 513], 8, 2, 64
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=10, packed=False)
    out, lse = torch.empty_like(q), torch.empty((h, q.shape[0]), device=DEV)
    pa.pa_prefill(out, q, k, v, cut, 0.125, lse=lse)
    for s, n in enumerate(lens):
        a, b = cu[s], cu[s + 1]
        one, one_l = torch.empty_like(q[a:b]), torch.empty((h, n), device=DEV)
        pa.pa_prefill(one, q[a:b], k[a:b], v[a:b], torch.tensor([0, n], dtype=torch.int32, device=DEV),
                      0.125, lse=one_l)
        assert torch.equal(one, out[a:b]) and torch.equal(one_l, lse[:, a:b])
    pa.pa_sync_check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_prompts_are_skipped(dtype):
    lens, h, hkv, d = [200, 50, 60], 2, 2, 64
    q, k, v, cu, _ = _inputs(lens, h, hkv, d, dtype, seed=12)
    for bad, good in (([0, 200, 190, 310], (0, 200)), ([0, 200, 250, 311], (0, 250)),
                      ([-1, 200, 250, 310], (200, 310))):
        out = torch.full(q.shape, 7.0, device=DEV, dtype=dtype)
        cut = torch.tensor(bad, dtype=torch.int32, device=DEV)
        pa.pa_prefill(out, q, k, v, cut, 0.125, max_seq_len=310)
        with pytest.raises(pa.PAError) as e:
            pa.pa_sync_check()
        assert e.value.code == pa.PA_ERR_BAD_INDEX
        assert bool((out[good[0]:good[1]] != 7).all())
    # the 40th of prompts whose tiles are all found among the first 32
    out = torch.full(q.shape, 7.0, device=DEV, dtype=dtype)
    w = torch.empty((40, h, 310), device=DEV)
    cut = torch.tensor([0, 1] + [1] * 38 + [311], dtype=torch.int32, device=DEV)
    for call in (lambda: pa.pa_prefill(out, q, k, v, cut, 0.125, max_seq_len=310),
                 lambda: pa.pa_prefill_weights(w, q, k, torch.zeros((h, 310), device=DEV), cut, 0.125, max_seq_len=310)):
        call()
        with pytest.raises(pa.PAError):
            pa.pa_sync_check()
    assert bool((out[1:] == 7).all()) and not w[1:].any()
    out = torch.full(q.shape, 7.0, device=DEV, dtype=dtype)
    pa.pa_prefill(out, q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), 0.125, max_seq_len=100)
    with pytest.raises(pa.PAError):
        pa.pa_sync_check()                                        # the first is longer than the bound
    assert bool((out[:200] == 7).all()) and bool((out[200:] != 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("last", [0, 1, 64, 130])
@pytest.mark.parametrize("lens,h,hkv,d", RAGGED)
def test_prefill_weights(lens, h, hkv, d, last, dtype):
    scale = 1 / math.sqrt(d)
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=sum(lens) + h, front=2, behind=5)
    lse = torch.full((h, q.shape[0]), float("nan"), device=DEV)
    for s, n in enumerate(lens):
        if n:
            lse[:, cu[s]:cu[s + 1]] = P.prompt_attention(
                q[cu[s]:cu[s + 1]], k[cu[s]:cu[s + 1]], v[cu[s]:cu[s + 1]], scale)[1].float()
    w = torch.full((len(lens), hkv, max(lens) + 13), 7.0, device=DEV)
    pa.pa_prefill_weights(w, q, k, lse, cut, scale, max_seq_len=max(lens), last_queries=last)
    pa.pa_sync_check()
    for s, n in enumerate(lens):
        assert not w[s, :, n:].any()
        if n == 0:
            continue
        a, b = cu[s], cu[s + 1]
        ref, mag = P.prompt_weights(q[a:b], k[a:b], lse[:, a:b], scale, last)
        count = (h // hkv) * n
        tol = P.EPS32 * (mag + ref * (count + 16)) + 1e-37
        err = (w[s, :, :n].double() - ref).abs()
        assert bool((err <= tol).all()), f"prompt {s}: {float((err / tol).max()):.2f} of the bound"
    again = torch.full_like(w, 3.0)
    pa.pa_prefill_weights(again, q, k, lse, cut, scale, max_seq_len=max(lens), last_queries=last)
    assert torch.equal(again, w)                                  # fixed order


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_weights_take_no_part_of_later_tokens(dtype, value):
    """A key's weight sums over later queries alone; another key's content is not in it."""
    lens, h, hkv, d = [300, 100], 4, 2, 64
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=13, packed=False)
    out, lse = torch.empty_like(q), torch.empty((h, q.shape[0]), device=DEV)
    pa.pa_prefill(out, q, k, v, cut, 0.125, lse=lse)
    w = torch.empty((2, hkv, 300), device=DEV)
    pa.pa_prefill_weights(w, q, k, lse, cut, 0.125)
    bad = q.clone()
    bad[150] = value                                              # a query before the keys 151 ..
    w2 = torch.empty_like(w)
    pa.pa_prefill_weights(w2, bad, k, lse, cut, 0.125)
    pa.pa_sync_check()
    assert torch.equal(w2[0, :, 151:], w[0, :, 151:]) and torch.equal(w2[1], w[1])
    for i in (128, 129, 150, 151, 152, 153, 154, 155):            # and it is in the earlier keys' weights
        lse2 = lse.clone()
        lse2[:, i] = float("nan")
        pa.pa_prefill_weights(w2, q, k, lse2, cut, 0.125)
        assert bool(torch.isnan(w2[0, :, :i + 1]).all()) and torch.equal(w2[0, :, i + 1:], w[0, :, i + 1:])


def test_negative_scale_weights():
    lens, h, hkv, d = [260], 4, 2, 128
    for dtype in (BF16, F32):
        q, k, v, cu, cut = _inputs(lens, h, hkv, d, dtype, seed=14, packed=False)
        lse = P.prompt_attention(q, k, v, -0.3)[1].float().contiguous()
        w = torch.empty((1, hkv, 260), device=DEV)
        pa.pa_prefill_weights(w, q, k, lse, cut, -0.3)
        pa.pa_sync_check()
        ref, mag = P.prompt_weights(q, k, lse, -0.3)
        assert bool(((w[0].double() - ref).abs() <= P.EPS32 * (mag + ref * (2 * 260 + 16))).all())


def test_streams_and_graph():
    """On another stream, and replayed from a graph with new inputs."""
    lens, h, hkv, d = [333, 90], 8, 2, 128
    q, k, v, cu, cut = _inputs(lens, h, hkv, d, BF16, seed=15, packed=False)
    ref, ref_l = torch.empty_like(q), torch.empty((h, q.shape[0]), device=DEV)
    rw = torch.empty((2, hkv, 333), device=DEV)
    pa.pa_prefill(ref, q, k, v, cut, 0.1, max_seq_len=333, lse=ref_l)
    pa.pa_prefill_weights(rw, q, k, ref_l, cut, 0.1, max_seq_len=333)
    out, lse, w = torch.zeros_like(ref), torch.zeros_like(ref_l), torch.zeros_like(rw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pa.pa_prefill(out, q, k, v, cut, 0.1, max_seq_len=333, lse=lse, stream=st)
    pa.pa_prefill_weights(w, q, k, lse, cut, 0.1, max_seq_len=333, stream=st)
    st.synchronize()
    assert torch.equal(out, ref) and torch.equal(w, rw)
    graph = torch.cuda.CUDAGraph()
    q2 = torch.zeros_like(q)
    with torch.cuda.graph(graph):
        pa.pa_prefill(out, q2, k, v, cut, 0.1, max_seq_len=333, lse=lse)
        pa.pa_prefill_weights(w, q2, k, lse, cut, 0.1, max_seq_len=333)
    q2.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    pa.pa_sync_check()
    assert torch.equal(out, ref) and torch.equal(w, rw)
