"""Plain 64-bit forms of the calls around decode, from their formulas, and the error bounds
that the tests of those calls hold them to. Torch tensors on any device, float64 inside."""
import math

import torch

EPS32 = 2.0 ** -24    # half a step of fp32, relative
EPS_BF16 = 2.0 ** -8  # half a step of bf16, relative


def rotate(x, positions, inv_freq, axis, rotary, pairs, mscale=1.0):
    """x [T][heads][D] turned by its positions [axes][T]; returns float64 and, per element, the
    sum of magnitudes of the products behind it."""
    y = x.double().clone()
    mag = y.abs()
    ang = torch.stack([positions[a].double() * f for f, a in zip(inv_freq, axis)], -1)[:, None]
    half = rotary // 2
    if pairs == "half":
        lo, hi = torch.arange(half), torch.arange(half) + half
    else:
        lo, hi = 2 * torch.arange(half), 2 * torch.arange(half) + 1
    lo, hi = lo.to(x.device), hi.to(x.device)
    a, b = x[..., lo].double(), x[..., hi].double()
    y[..., lo] = mscale * (a * ang.cos() - b * ang.sin())
    y[..., hi] = mscale * (b * ang.cos() + a * ang.sin())
    mag[..., lo] = mag[..., hi] = abs(mscale) * (a.abs() + b.abs())
    return y, mag


def prompt_attention(q, k, v, scale):
    """One prompt: q [n][H][D], k, v [n][Hkv][D] -> out [n][H][D], lse [H][n], and the
    magnitudes for the bounds: sum of p |v| [n][H][D], largest sum of |scale q k| [H][n]."""
    n, h, _ = q.shape
    hkv = k.shape[1]
    qd, kd, vd = q.double(), k.double(), v.double()
    out, mag = torch.zeros_like(qd), torch.zeros_like(qd)
    lse = torch.zeros((h, n), dtype=torch.float64, device=q.device)
    sabs = torch.zeros_like(lse)
    dead = torch.ones((n, n), dtype=torch.bool, device=q.device).triu(1)
    for hd in range(h):
        kh = hd // (h // hkv)
        x = (qd[:, hd] @ kd[:, kh].T * scale).masked_fill(dead, -math.inf)
        lse[hd] = torch.logsumexp(x, 1)
        p = torch.softmax(x, 1)
        out[:, hd], mag[:, hd] = p @ vd[:, kh], p @ vd[:, kh].abs()
        sabs[hd] = (qd[:, hd].abs() @ kd[:, kh].abs().T * abs(scale)).masked_fill(dead, 0).amax(1)
    return out, lse, mag, sabs


def prompt_weights(q, k, lse, scale, last=0):
    """weights [Hkv][n] of one prompt, and sum of weight x (1 + the bound's magnitudes)."""
    n, h, _ = q.shape
    hkv = k.shape[1]
    w = torch.zeros((hkv, n), dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(w)
    dead = torch.ones((n, n), dtype=torch.bool, device=q.device).triu(1)
    if last:
        dead[:max(0, n - last)] = True
    for hd in range(h):
        kh = hd // (h // hkv)
        qd, kd = q[:, hd].double(), k[:, kh].double()
        x = (qd @ kd.T * scale - lse[hd].double()[:, None])
        p = x.exp().masked_fill(dead, 0)
        w[kh] += p.sum(0)
        err = qd.abs() @ kd.abs().T * abs(scale) * (q.shape[2] + 4) + 4 * lse[hd].double().abs()[:, None]
        mag[kh] += (p * err.masked_fill(dead, 0)).sum(0)
    return w, mag


def attention_bound(out, mag, sabs, d, n, dtype):
    """Most that the computed out may differ from `out`. A score is a sum of d products: it is
    off by (d + 4) EPS32 sabs, which moves numerator and denominator of the softmax by that
    factor each; sums of n weights add n EPS32 each; bf16 weights are off by EPS_BF16 and the
    bf16 result by EPS_BF16 of itself. Twice EPS32 terms for the exponential's own error."""
    s = sabs.movedim(0, -1)[..., None]
    rel = 2 * ((d + 4) * EPS32 * s + (n + 16) * EPS32)
    tol = mag * rel
    if dtype == torch.bfloat16:
        tol = tol + mag * EPS_BF16 + (out.abs() + tol + mag * EPS_BF16) * EPS_BF16
    else:
        tol = tol + out.abs() * EPS32
    return tol + 1e-37


def lse_bound(lse, sabs, d, n):
    return (d + 4) * EPS32 * sabs + (n + 16) * EPS32 + 4 * EPS32 * lse.abs()


def evict(weights, n, budget, recent):
    """One (sequence, kv head): kept (list of old positions, -1 past the length)."""
    if n <= budget:
        return [j if j < n else -1 for j in range(budget)]
    edge, cand = budget - recent, n - recent
    key = [(-math.inf if math.isnan(x) else x) for x in weights[:cand]]
    heavy = set(sorted(range(cand), key=lambda t: (-key[t], t))[:edge])
    movers = iter(sorted(t for t in heavy if t >= edge))
    return [j if j in heavy else next(movers) for j in range(edge)] + list(range(cand, n))
