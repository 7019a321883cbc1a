"""The operators of a serving step around paged decode, as measured work:

* ``rope``             pa_rope_append: rotary positions with several axes, fused with the paged append;
* ``prefill``          pa_prefill: causal attention over whole packed prompts, with its log-sum-exp;
* ``prefill_weights``  pa_prefill_weights: the attention weight each prompt token received;
* ``decode_weights``   pa_decode_weights: one decode step that adds each token's weight;
* ``evict``            pa_evict: keep a budget of tokens per kv head, compact the rest away.

``run`` computes them in plain torch operations, or (``own``) through the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a 64/8-head model, 8 sequences: latency of one small launch
        dict(name="rope decode 8 tok 64/8", op="rope", tokens=8, heads=64, kv_heads=8, head_dim=128, rotary=128,
             axes=3, pairs="half", dtype="bf16", block=16, far=120000),
        # a packed batch of prompts with images (time, height, width positions) entering the pool
        dict(name="rope prompt 16K tok 64/8", op="rope", tokens=16384, heads=64, kv_heads=8, head_dim=128, rotary=128,
             axes=3, pairs="half", dtype="bf16", block=16, far=30000),
        # chat-sized prompts of a 40-head model, very different lengths, one of a single token
        dict(name="prefill ragged 40/40", op="prefill", lens="1 900 77 333 1024 128 513 250 17 640", heads=40,
             kv_heads=40, head_dim=128, dtype="bf16"),
        # narrow heads, grouped, odd lengths
        dict(name="prefill ragged 32/8 d64", op="prefill", lens="2047 1500 3001 129", heads=32, kv_heads=8,
             head_dim=64, dtype="bf16"),
        # one long document on a 64/8-head model
        dict(name="prefill 16K 64/8", op="prefill", lens="16384", heads=64, kv_heads=8, head_dim=128, dtype="bf16"),
        # fp32 inputs: accuracy checks and small models
        dict(name="prefill f32 8/2", op="prefill", lens="700 1025 300", heads=8, kv_heads=2, head_dim=64, dtype="f32"),
        # the weight every token of a prompt received from all of its queries
        dict(name="prefill_weights 8K 64/8", op="prefill_weights", lens="8192", heads=64, kv_heads=8, head_dim=128,
             dtype="bf16", last=0, room=256),
        # only the last 64 queries vote (an observation window), ragged prompts
        dict(name="prefill_weights last64 40/40", op="prefill_weights", lens="4001 1024 30 2500 777 3900", heads=40,
             kv_heads=40, head_dim=128, dtype="bf16", last=64, room=64),
        # long contexts, 64/8 heads: the decode step whose cache is due for eviction
        dict(name="decode_weights 8x32K 64/8", op="decode_weights", seqs=8, ctx=32768, least=32768, heads=64,
             kv_heads=8, head_dim=128, dtype="bf16", block=16),
        # a small ragged batch of a 40-head model
        dict(name="decode_weights 16x2K 40/40", op="decode_weights", seqs=16, ctx=2048, least=300, heads=40,
             kv_heads=40, head_dim=128, dtype="bf16", block=16),
        # halving eight 32K contexts
        dict(name="evict 8x32K to 16K", op="evict", seqs=8, ctx=32768, least=32768, kv_heads=8, head_dim=128,
             budget=16384, recent=256, dtype="bf16", block=16),
        # one block over budget, every few steps
        dict(name="evict 16x2064 to 2048", op="evict", seqs=16, ctx=2064, least=1000, kv_heads=40, head_dim=128,
             budget=2048, recent=128, dtype="bf16", block=16),
    ]


def draw(rng):
    """One more case of the listed ranges."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "prefill", "prefill_weights", "decode_weights", "evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16, 40])
    group = rng.choice([1, 2, 4, 5, 8]) if hkv <= 8 else 1
    h = hkv * group
    bs = rng.choice([16, 32, 64])
    if op == "rope":
        return dict(op=op, tokens=log(1, 8500), heads=h, kv_heads=hkv, head_dim=d,
                    rotary=rng.choice([d, d // 2, 48]), axes=rng.choice([1, 2, 3]),
                    pairs=rng.choice(["half", "adjacent"]), dtype=rng.choice(["bf16", "bf16", "f32", "fp8"]),
                    block=bs, far=log(100, 1000000))
    if op in ("prefill", "prefill_weights"):
        f32 = rng.random() < 0.2
        n = rng.choice([1, 2, 3, 7, 12])
        top = 1200 if f32 else 6000
        lens = [log(1, top) for _ in range(n)]
        case = dict(op=op, lens=" ".join(map(str, lens)), heads=h, kv_heads=hkv, head_dim=d,
                    dtype="f32" if f32 else "bf16")
        if op == "prefill_weights":
            case["last"] = rng.choice([0, log(1, 300)])
            case["room"] = rng.randrange(0, 200)
        return case
    s = log(1, 24)
    ctx = log(16, min(32768, 155000 // s // max(1, hkv // 8)))
    least = max(1, int(ctx * rng.choice([0.1, 0.6, 1.0])))
    if op == "decode_weights":
        return dict(op=op, seqs=s, ctx=ctx, least=least, heads=h, kv_heads=hkv, head_dim=d,
                    dtype=rng.choice(["bf16", "bf16", "f32", "fp8"]), block=bs)
    budget = max(1, int(ctx * rng.uniform(0.2, 1.0)))
    return dict(op=op, seqs=s, ctx=ctx, least=least, kv_heads=hkv, head_dim=d, budget=budget,
                recent=int(budget * rng.choice([0.0, 0.05, 0.5])), dtype=rng.choice(["bf16", "f32", "fp8"]), block=bs)


def _lens(case):
    return [int(x) for x in case["lens"].split()]


def _contexts(case):
    """Context lengths from `least` to `ctx`, evenly spread, the longest first."""
    s = case["seqs"]
    return [case["ctx"] - (case["ctx"] - case["least"]) * i // max(1, s - 1) for i in range(s)]


def _sections(case):
    """Frequencies per axis: time gets what the other axes' quarters leave."""
    half, a = case["rotary"] // 2, case["axes"]
    rest = [half // 4 + (half // 8 if a == 3 else 0)] * (a - 1)
    return [half - sum(rest)] + rest


def _inv_freq(case):
    return [1e6 ** (-2.0 * i / case["rotary"]) for i in range(case["rotary"] // 2)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pool(case, lens, g, rng):
    """Block tables over a shuffled pool with some spare blocks; the K and V pools."""
    bs, hkv, d = case["block"], case["kv_heads"], case["head_dim"]
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 7
    order = rng.permutation(nb)
    width = max(need) + 1
    tables = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n]
        at += n
    k, v = (_cached(torch.randn((nb, hkv, bs, d), generator=g, device="cuda", dtype=torch.bfloat16), case["dtype"])
            for _ in range(2))
    return torch.as_tensor(tables, device="cuda"), k, v


def _cached(x, dtype):
    """Pool values in the cache's type: fp8 codes stand for code x scale 0.02."""
    return (x.float() / 0.02).to(DTYPES[dtype]) if dtype == "fp8" else x.to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, d, hkv = case["op"], case["head_dim"], case["kv_heads"]
    st = dict(case=case, scale=1.0 / math.sqrt(d))
    act = torch.float32 if case["dtype"] == "f32" else torch.bfloat16

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=act)

    if op == "rope":
        t, h, bs = case["tokens"], case["heads"], case["block"]
        # q, k and v as a model's packed projection leaves them: strided by token
        qkv = randn(t, h + 2 * hkv, d)
        st["q"], st["k"], st["v"] = qkv[:, :h], qkv[:, h:h + hkv], qkv[:, h + hkv:]
        nb = -(-t // bs) + 3
        st["k_cache"] = torch.zeros((nb, hkv, bs, d), device="cuda").to(DTYPES[case["dtype"]])
        st["v_cache"] = torch.zeros((nb, hkv, bs, d), device="cuda").to(DTYPES[case["dtype"]])
        slots = rng.permutation(nb * bs)[:t].astype(np.int64)
        slots[rng.random(t) < 0.02] = -1                         # padding tokens
        st["slots"] = torch.as_tensor(slots, device="cuda")
        st["positions"] = torch.as_tensor(rng.integers(0, case["far"], (case["axes"], t), dtype=np.int32), device="cuda")
        st["q_out"] = torch.empty((t, h, d), device="cuda", dtype=act)
        if case["dtype"] == "fp8":
            st["k_scale"], st["v_scale"] = (torch.rand(hkv, generator=g, device="cuda") * 0.02 + 0.01 for _ in range(2))
        st["freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device="cuda")
        st["axis"] = torch.tensor(np.repeat(np.arange(case["axes"]), _sections(case)), device="cuda")
        if own:
            import paged_kv_cache_335_b200 as pa
            st["rope"] = pa.rope_desc(case["rotary"], inv_freq=_inv_freq(case), sections=_sections(case),
                                      pairs=case["pairs"])
        return st
    if op in ("prefill", "prefill_weights"):
        lens, h = _lens(case), case["heads"]
        t = sum(lens)
        st["lens"] = lens
        st["q"], st["k"] = randn(t, h, d), randn(t, hkv, d)
        st["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
        if op == "prefill":
            st["v"] = randn(t, hkv, d)
            st["out"] = torch.empty((t, h, d), device="cuda", dtype=act)
            st["lse"] = torch.empty((h, t), device="cuda", dtype=torch.float32)
        else:
            # the log-sum-exp that the prompt's attention returned
            st["lse"] = torch.cat([_lse(st["q"][a:b], st["k"][a:b], st["scale"]) for a, b in _spans(lens)], 1)
            st["weights"] = torch.empty((len(lens), hkv, max(lens) + case["room"]), device="cuda")
        return st
    lens = _contexts(case)
    st["lens"] = lens
    st["tables"], st["k_cache"], st["v_cache"] = _pool(case, lens, g, rng)
    st["ctx"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    stride = (max(lens) + 63) // 64 * 64
    live = torch.arange(stride, device="cuda") < st["ctx"][:, None, None]
    # accumulated weights are heavy-tailed: a few tokens hold most of the attention
    st["weights"] = (torch.randn((len(lens), hkv, stride), generator=g, device="cuda") * 2).exp() * live
    if op == "decode_weights":
        st["q"] = randn(len(lens), case["heads"], d)
        st["out"] = torch.empty_like(st["q"])
        if case["dtype"] == "fp8":
            st["k_scale"], st["v_scale"] = (torch.full((hkv,), 0.02, device="cuda") for _ in range(2))
        if own:
            import paged_kv_cache_335_b200 as pa
            st["workspace"] = torch.empty(pa.pa_decode_weights_workspace_size(
                len(lens), case["heads"], max(lens), st["k_cache"]), dtype=torch.uint8, device="cuda")
        return st
    st["weights_out"] = torch.empty_like(st["weights"])
    st["kept"] = torch.empty((len(lens), hkv, case["budget"]), dtype=torch.int32, device="cuda")
    st["new_ctx"] = torch.empty_like(st["ctx"])
    return st


def _spans(lens):
    at = np.concatenate([[0], np.cumsum(lens)])
    return [(int(a), int(b)) for a, b in zip(at[:-1], at[1:])]


def _lse(q, k, scale):
    """Natural log-sum-exp of one prompt's causal scores, [H][n], 1024 rows at a time."""
    n, h, _ = q.shape
    hkv = k.shape[1]
    kf = k.float().permute(1, 2, 0)
    out = []
    for a in range(0, n, 1024):
        b = min(n, a + 1024)
        x = q[a:b].float().reshape(b - a, hkv, h // hkv, -1).permute(1, 2, 0, 3).flatten(1, 2) @ kf[:, :, :b] * scale
        x = x.reshape(h, b - a, b)
        x.masked_fill_(torch.arange(b, device="cuda") > torch.arange(a, b, device="cuda")[:, None], -math.inf)
        out.append(torch.logsumexp(x, -1))
    return torch.cat(out, 1)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


# ---- the library's calls
def _own_rope(st):
    import paged_kv_cache_335_b200 as pa
    args = (st["q_out"], st["q"], st["k"], st["v"], st["positions"], st["slots"], st["k_cache"], st["v_cache"])
    if st["case"]["dtype"] == "fp8":
        pa.pa_rope_append_quant(*args, st["k_scale"], st["v_scale"], st["rope"])
    else:
        pa.pa_rope_append(*args, st["rope"])
    return st["q_out"], st["k_cache"], st["v_cache"]


def _own_prefill(st):
    import paged_kv_cache_335_b200 as pa
    pa.pa_prefill(st["out"], st["q"], st["k"], st["v"], st["cu"], st["scale"], max_seq_len=max(st["lens"]),
                  lse=st["lse"])
    return st["out"], st["lse"]


def _own_prefill_weights(st):
    import paged_kv_cache_335_b200 as pa
    pa.pa_prefill_weights(st["weights"], st["q"], st["k"], st["lse"], st["cu"], st["scale"],
                          max_seq_len=max(st["lens"]), last_queries=st["case"]["last"])
    return st["weights"]


def _own_decode_weights(st):
    import paged_kv_cache_335_b200 as pa
    args = (st["out"], st["weights"], st["q"], st["k_cache"], st["v_cache"])
    rest = (st["tables"], st["ctx"], st["scale"])
    kw = dict(max_context_len=max(st["lens"]), workspace=st["workspace"])
    if st["case"]["dtype"] == "fp8":
        pa.pa_decode_weights_quant(*args, st["k_scale"], st["v_scale"], *rest, **kw)
    else:
        pa.pa_decode_weights(*args, *rest, **kw)
    return st["out"], st["weights"]


def _own_evict(st):
    import paged_kv_cache_335_b200 as pa
    pa.pa_evict(st["k_cache"], st["v_cache"], st["tables"], st["ctx"], st["weights"], st["weights_out"],
                st["new_ctx"], st["kept"], st["case"]["budget"], st["case"]["recent"], max_context_len=max(st["lens"]))
    return st["k_cache"], st["v_cache"], st["weights_out"], st["new_ctx"], st["kept"]


# ---- the plain forms
def _rotate(x, cos, sin, rotary, pairs):
    """x [T][heads][D] float; cos, sin [T][1][rotary / 2]."""
    r, rest = x[..., :rotary], x[..., rotary:]
    if pairs == "half":
        a, b = r.chunk(2, -1)
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _code(x, scale):
    """FP8 codes of x / scale per kv head, saturated."""
    return (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)


def _plain_rope(st):
    c = st["case"]
    bs = c["block"]
    ang = st["positions"].double()[st["axis"]].T * st["freq"]            # 64 bits: far positions
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    st["q_out"].copy_(_rotate(st["q"].float(), cos, sin, c["rotary"], c["pairs"]))
    k = _rotate(st["k"].float(), cos, sin, c["rotary"], c["pairs"])
    v = st["v"].float()
    if c["dtype"] == "fp8":
        k, v = _code(k, st["k_scale"]), _code(v, st["v_scale"])
    else:
        k, v = k.to(st["k_cache"].dtype), v.to(st["v_cache"].dtype)
    keep = st["slots"] >= 0
    sl = st["slots"][keep]
    for cache, x in ((st["k_cache"], k), (st["v_cache"], v)):
        raw = torch.uint8 if c["dtype"] == "fp8" else x.dtype
        cache.view(raw)[sl // bs, :, sl % bs] = x.view(raw)[keep]
    return st["q_out"], st["k_cache"], st["v_cache"]


def _grouped(q, hkv):
    """[T][H][D] -> [Hkv][group * T][D], the rows that read one kv head."""
    t, h, d = q.shape
    return q.reshape(t, hkv, h // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)


def _plain_prefill(st):
    out, lse = st["out"], st["lse"]
    h, hkv = st["case"]["heads"], st["case"]["kv_heads"]
    for a, b in _spans(st["lens"]):
        step = max(1, min(b - a, (1 << 31) // (h * (b - a))))            # rows at a time: up to 8 GB of scores
        k, v = st["k"][a:b].float().permute(1, 2, 0), st["v"][a:b].float().transpose(0, 1)
        for i in range(a, b, step):
            e = min(b, i + step)
            x = _grouped(st["q"][i:e], hkv).float() @ k[:, :, :e - a]
            x = x.reshape(h, e - i, e - a) * st["scale"]
            x.masked_fill_(torch.arange(a, e, device="cuda") > torch.arange(i, e, device="cuda")[:, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            p = x.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            o = (p.reshape(hkv, -1, e - a) @ v[:, :e - a]).reshape(h, e - i, -1) / l
            out[i:e] = o.transpose(0, 1)
            lse[:, i:e] = (m + l.log())[..., 0]
    return out, lse


def _plain_prefill_weights(st):
    c, w = st["case"], st["weights"]
    h, hkv = c["heads"], c["kv_heads"]
    w.zero_()
    for s, (a, b) in enumerate(_spans(st["lens"])):
        first = a if c["last"] == 0 else max(a, b - c["last"])
        step = max(1, min(b - a, (1 << 31) // (h * (b - a))))
        k = st["k"][a:b].float().permute(1, 2, 0)
        for i in range(first, b, step):
            e = min(b, i + step)
            x = _grouped(st["q"][i:e], hkv).float() @ k[:, :, :e - a]
            x = x.reshape(h, e - i, e - a) * st["scale"] - st["lse"][:, i:e, None]
            x.masked_fill_(torch.arange(a, e, device="cuda") > torch.arange(i, e, device="cuda")[:, None], -math.inf)
            w[s, :, :e - a] += x.exp_().reshape(hkv, -1, e - a).sum(1)
    return w


def _gathered(cache, tables, n):
    """[S][Hkv][n][D] values of the first n positions (dead entries read block 0)."""
    bs = cache.shape[2]
    x = cache.view(torch.uint8 if cache.element_size() == 1 else cache.dtype)[tables[:, :-(-n // bs)].clamp(min=0).long()]
    return x.view(cache.dtype).permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :n]


def _plain_decode_weights(st):
    c = st["case"]
    s, hkv, n = c["seqs"], c["kv_heads"], max(st["lens"])
    k = _gathered(st["k_cache"], st["tables"], n).float()
    v = _gathered(st["v_cache"], st["tables"], n).float()
    if c["dtype"] == "fp8":
        k, v = k * st["k_scale"][:, None, None], v * st["v_scale"][:, None, None]
    q = st["q"].float().reshape(s, hkv, c["heads"] // hkv, -1)
    x = (q @ k.transpose(-1, -2)) * st["scale"]
    x.masked_fill_(torch.arange(n, device="cuda") >= st["ctx"][:, None, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp_()
    p = p / p.sum(-1, keepdim=True)
    st["out"].copy_((p @ v).reshape(s, c["heads"], -1))
    st["weights"][:, :, :n] += p.sum(2)
    return st["out"], st["weights"]


def _plain_evict(st):
    c, w, bs = st["case"], st["weights"], st["case"]["block"]
    budget, recent = c["budget"], c["recent"]
    s, hkv, stride = w.shape
    n = st["ctx"].long()[:, None, None]
    t = torch.arange(stride, device="cuda")
    edge = budget - recent                                               # heavy tokens land in [0, edge)
    # the (budget - recent) largest of the tokens before the recent ones; ties go to the lowest index
    heavy = torch.where(t < n - recent, w.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf), -math.inf)
    order = heavy.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order).contiguous())
    # a masked place ties with a weight of -inf but has a higher index
    chosen = (rank < edge) & (t < n - recent)
    hole, mover = ~chosen & (t < edge), chosen & (t >= edge)
    j = torch.arange(budget, device="cuda").expand(s, hkv, budget)
    kept = torch.where(j < edge, j, n - recent + (j - edge))
    # the i-th hole takes the i-th mover
    nth = (mover.cumsum(-1) - 1).clamp(min=0)
    source = torch.zeros_like(order).scatter_add_(-1, torch.where(mover, nth, stride - 1), torch.where(mover, t, 0))
    which = (hole.cumsum(-1) - 1).clamp(min=0)
    if edge:
        kept[..., :edge] = torch.where(hole, source.gather(-1, which), t)[..., :edge]
    kept = torch.where(n > budget, kept, torch.where(j < n, j, -1))
    new = torch.minimum(n, torch.tensor(budget, device="cuda"))
    live = kept >= 0
    st["weights_out"].zero_()
    st["weights_out"][..., :budget] = torch.where(live, w.gather(-1, kept.clamp(min=0))[..., :stride], 0)[..., :stride]
    # rows move inside each sequence's own blocks
    tab = st["tables"].long()
    src = kept.clamp(min=0)
    head = torch.arange(hkv, device="cuda")[None, :, None].expand_as(src)
    seq = torch.arange(s, device="cuda")[:, None, None].expand_as(src)
    go = live & (kept != j)
    sb, so, db, do = (tab[seq, src // bs][go], (src % bs)[go], tab[seq, j.long() // bs][go], (j % bs)[go])
    for cache in (st["k_cache"], st["v_cache"]):
        raw = cache.view(torch.uint8) if cache.element_size() == 1 else cache
        raw[db, head[go], do] = raw[sb, head[go], so]
    st["kept"].copy_(kept)
    st["new_ctx"].copy_(new[:, 0, 0])
    return st["k_cache"], st["v_cache"], st["weights_out"], st["new_ctx"], st["kept"]


_plain = dict(rope=_plain_rope, prefill=_plain_prefill, prefill_weights=_plain_prefill_weights,
              decode_weights=_plain_decode_weights, evict=_plain_evict)
_own = dict(rope=_own_rope, prefill=_own_prefill, prefill_weights=_own_prefill_weights,
            decode_weights=_own_decode_weights, evict=_own_evict)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _pairs(lens, last=0):
    """(query, key) pairs of causal attention; with `last`, of the last queries alone."""
    return sum(n * (n + 1) // 2 - (max(0, n - last) * (max(0, n - last) + 1) // 2 if last else 0) for n in lens)


def work(case):
    op, d, hkv = case["op"], case["head_dim"], case["kv_heads"]
    e = {"f32": 4, "bf16": 2, "fp8": 1}[case["dtype"]]
    a = max(2, e)                                                        # activations: bf16 beside fp8 caches
    if op == "rope":
        t, h = case["tokens"], case["heads"]
        return {"bytes": t * (2 * h * d * a + 2 * hkv * d * (a + e) + 4 * case["axes"] + 8),
                "flops": 3 * t * (h + hkv) * case["rotary"]}
    if op == "prefill":
        t, h = sum(_lens(case)), case["heads"]
        return {"bytes": t * (2 * (h + hkv) * d * a + 4 * h), "flops": 4 * d * h * _pairs(_lens(case))}
    if op == "prefill_weights":
        lens, h = _lens(case), case["heads"]
        asked = sum(min(n, case["last"]) if case["last"] else n for n in lens)
        return {"bytes": asked * h * (d * a + 4) + sum(lens) * hkv * d * a +
                4 * len(lens) * hkv * (max(lens) + case["room"]),
                "flops": 2 * d * h * _pairs(lens, case["last"])}
    lens = _contexts(case)
    if op == "decode_weights":
        h = case["heads"]
        return {"bytes": sum(lens) * hkv * (2 * d * e + 8) + 2 * len(lens) * h * d * a,
                "flops": 4 * d * h * sum(lens)}
    # evict: weights read, the new row of weights and the kept positions written, and the rows that have to
    # move: the recent ones, and with heavy tokens spread evenly, those that lie behind the first budget - recent
    b, r = case["budget"], case["recent"]
    moved = sum(r + (b - r) * (n - b) // max(1, n - r) for n in lens if n > b)
    stride = (max(lens) + 63) // 64 * 64
    return {"bytes": hkv * (4 * sum(lens) + len(lens) * 4 * (stride + b) + moved * 4 * d * e),
            "flops": hkv * sum(lens)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op, d, hkv = case["op"], case["head_dim"], case["kv_heads"]
    if op == "rope":
        pos = st["positions"].double()
        rot = case["rotary"]
        bounds = np.cumsum(_sections(case))
        new = []
        for x in (st["q"], st["k"]):
            y = x.double().clone()
            for i, f in enumerate(_inv_freq(case)):
                ang = pos[int(np.searchsorted(bounds, i, side="right"))] * f
                z = torch.polar(torch.ones_like(ang), ang)[:, None]
                lo, hi = (i, i + rot // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
                r = torch.complex(x[..., lo].double(), x[..., hi].double()) * z
                y[..., lo], y[..., hi] = r.real, r.imag
            new.append(y)
        if case["dtype"] == "fp8":
            return new[0], None, None
        caches = [torch.zeros(st["k_cache"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
        for cache, x in zip(caches, (new[1], st["v"].double())):
            rows = cache.transpose(1, 2).reshape(-1, hkv, d)
            rows[st["slots"][st["slots"] >= 0]] = x[st["slots"] >= 0]
            cache.copy_(rows.reshape(cache.shape[0], case["block"], hkv, d).transpose(1, 2))
        return new[0], caches[0], caches[1]
    if op in ("prefill", "prefill_weights"):
        lens, h = _lens(case), case["heads"]
        if 4 * d * h * sum(n * n for n in lens) > 4e13:
            return None
        k = st["k"].double()
        out = torch.zeros((sum(lens), h, d), dtype=torch.float64, device="cuda")
        lse = torch.zeros((h, sum(lens)), dtype=torch.float64, device="cuda")
        if op == "prefill_weights":
            w = torch.zeros(st["weights"].shape, dtype=torch.float64, device="cuda")
        for s, n in enumerate(lens):
            a = sum(lens[:s])
            i = torch.arange(n, device="cuda")
            dead = i > i[:, None]
            for hd in range(h):
                x = torch.einsum("id,td->it", st["q"][a:a + n, hd].double() * st["scale"], k[a:a + n, hd * hkv // h])
                x[dead] = -math.inf
                if op == "prefill":
                    lse[hd, a:a + n] = torch.logsumexp(x, 1)
                    out[a:a + n, hd] = torch.softmax(x, 1) @ st["v"][a:a + n, hd * hkv // h].double()
                else:
                    p = torch.exp(x - st["lse"][hd, a:a + n, None].double())
                    w[s, hd * hkv // h, :n] += p[n - min(n, case["last"]) if case["last"] else 0:].sum(0)
        return (out, lse) if op == "prefill" else w
    if op == "decode_weights":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        w = st["weights"].double()
        h, bs = case["heads"], case["block"]
        for s, n in enumerate(st["lens"]):
            rows = st["tables"][s, :-(-n // bs)].long()
            kv = []
            for cache in (st["k_cache"], st["v_cache"]):
                raw = cache.view(torch.uint8)[rows].view(cache.dtype) if case["dtype"] == "fp8" else cache[rows]
                x = raw.double().permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n]
                kv.append(x * st["k_scale"].double()[:, None, None] if case["dtype"] == "fp8" else x)
            x = torch.einsum("kgd,ktd->kgt", st["q"][s].double().reshape(hkv, h // hkv, d) * st["scale"], kv[0])
            p = torch.softmax(x, -1)
            out[s] = torch.einsum("kgt,ktd->kgd", p, kv[1]).reshape(h, d)
            w[s, :, :n] += p.sum(1)
        return out, w
    return None  # evict moves values and computes none
