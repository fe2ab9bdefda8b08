"""Plain 64-bit forms of the scored router, the RMS norm and the int8 rows and
products, straight from their definitions, for the tests to compare with."""

import numpy as np
import torch


def route_scored(logits, bias, k, score="softmax", n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0,
                 n_shared=0):
    """(ids [T, k+S] int32, w [T, k+S] float64) of fp32 or bf16 logits [T, E]."""
    l = logits.detach().cpu().double().numpy()
    l = np.where(np.isnan(l), -np.inf, l)
    T, E = l.shape
    ids = np.zeros((T, k + n_shared), np.int32)
    w = np.ones((T, k + n_shared))
    b = None if bias is None else bias.detach().cpu().double().numpy()
    size = E // n_group
    for t in range(T):
        x = l[t]
        with np.errstate(invalid="ignore", over="ignore"):
            if score == "softmax":
                m = x.max()
                e = np.zeros(E) if m == -np.inf else np.where(x == m, 1.0, np.exp(x - m))
                s = e / e.sum() if e.sum() > 0 else e
            else:
                s = 1.0 / (1.0 + np.exp(-x))
            c = x if b is None else s + np.where(np.isnan(b), -np.inf, b)
            c = np.where(np.isnan(c), -np.inf, c)
        if n_group > 1:
            v = s if b is None and group_top > 1 else c
            with np.errstate(invalid="ignore"):
                g = np.array([np.sort(v[i * size:(i + 1) * size])[::-1][:group_top].sum() for i in range(n_group)])
            g = np.where(np.isnan(g), -np.inf, g)
            kept = sorted(range(n_group), key=lambda i: (-g[i], i))[:topk_group]
            cand = [e for i in kept for e in range(i * size, (i + 1) * size)]
        else:
            cand = list(range(E))
        pick = sorted(cand, key=lambda e: (-c[e], e))[:k]
        ids[t, :k] = pick
        off = np.array([b is not None and not b[e] > -np.inf for e in pick])
        if renormalize:
            # ratios of scores, formed so that they do not underflow
            lp = np.where(off, -np.inf, x[pick])
            top = lp.max()
            if top == -np.inf:
                v = np.zeros(k)
            elif score == "softmax":
                v = np.where(lp == top, 1.0, np.exp(np.minimum(lp - top, 0.0)))
            elif top < -60:
                v = np.exp(lp - top)
            else:
                v = np.where(off, 0.0, s[pick])
            v = v / v.sum() if v.sum() > 0 else v
        else:
            v = np.where(off, 0.0, s[pick])
        w[t, :k] = v * scale
        ids[t, k:] = np.arange(E, E + n_shared)
    return ids, w


def rmsnorm(x, residual, weight, eps):
    """(h, y) in float64 on x's device."""
    h = x.double()
    if residual is not None:
        h = h + residual.double()
    ms = h.square().mean(1, keepdim=True)
    return h, h / torch.sqrt(ms + eps) * weight.double()


def int8_rows(x):
    """(q [rows, K] int8, scales [rows] fp32) of bf16 rows: exact quotients,
    ties to even; a row with an infinity or a NaN has q = 0 and scale NaN."""
    v = x.double()
    amax = v.abs().amax(1, keepdim=True)                       # NaN where the row has one
    bad = ~torch.isfinite(amax)
    q = torch.round(127.0 * v / torch.where((amax == 0) | bad, torch.ones_like(amax), amax))
    q = torch.where(bad.expand_as(q), torch.zeros_like(q), q)
    scales = (amax / 127.0).float()
    scales[bad] = float("nan")
    return q.to(torch.int8), scales[:, 0]


def _rows_of(a, a_scales, perm, slots):
    if perm is None:
        return a.double(), a_scales.double()
    src = (perm.long() // slots).to(a.device)
    return a[src].double(), a_scales[src].double()


def grouped_int8(a, a_scales, perm, offsets, w, w_scales, slots):
    """v [P, N] float64: every row times its expert's weights, scales applied."""
    x, sx = _rows_of(a, a_scales, perm, slots)
    off = offsets.tolist()
    out = torch.zeros(off[-1], w.shape[1], dtype=torch.float64, device=a.device)
    for e in range(w.shape[0]):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            out[lo:hi] = (x[lo:hi] @ w[e].double().T) * w_scales[e].double() * sx[lo:hi, None]
    return out


def swiglu(v):
    """(act, g, u) of gate/up products [P, 2I]."""
    g, u = v.chunk(2, dim=1)
    return g / (1.0 + torch.exp(-g)) * u, g, u
