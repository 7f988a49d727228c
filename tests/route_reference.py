"""The trainable router and the optimizer's end in plain 64-bit numpy, from their formulas,
for the tests of the kernels."""
import math

import numpy as np


def route(l, k, score="softmax", normalize=True, scale=1.0, n_group=1, topk_group=1, group_topn=2, bias=None,
          mask=None, offsets=None):
    """A dict of every output, and the scores and live tokens, token by token."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    offsets = np.array([0, T]) if offsets is None else np.asarray(offsets)
    S = len(offsets) - 1
    idx = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    s, softs = np.zeros((T, E)), np.zeros((T, E))
    lse = np.zeros(T)
    live = np.zeros(T, bool)
    counts = np.zeros((S, E), np.int64)
    P = np.zeros((S, E))
    n = np.zeros(S, np.int64)
    zsum = 0.0
    for b in range(S):
        for t in range(offsets[b], offsets[b + 1]):
            on = [e for e in range(E) if l[t, e] > -np.inf]
            if (mask is not None and not mask[t]) or not on:
                continue
            live[t] = True
            top = max(l[t, e] for e in on)
            soft = np.zeros(E)
            soft[on] = np.exp(l[t, on] - top)
            lse[t] = top + math.log(soft.sum())
            soft /= soft.sum()
            softs[t] = soft
            if score == "softmax":
                s[t] = soft
            else:
                s[t, on] = 1.0 / (1.0 + np.exp(-l[t, on]))
            sel = s[t] + (0.0 if bias is None else np.asarray(bias, np.float64))
            rank = l[t] if bias is None else sel
            on = [e for e in on if sel[e] > -np.inf]     # a bias of -inf keeps an expert from being chosen
            allowed = set(on)
            if n_group > 1:
                size = E // n_group
                sums = []
                for g in range(n_group):
                    inside = sorted((sel[e] for e in on if e // size == g), reverse=True)[:group_topn]
                    sums.append(sum(inside) if inside else -np.inf)
                kept = sorted(range(n_group), key=lambda g: (-sums[g], g))[:topk_group]
                allowed = {e for e in on if e // size in kept}
            best = sorted(allowed, key=lambda e: (-rank[e], e))[:k]
            total = sum(s[t, e] for e in best) + 1e-20
            for j, e in enumerate(best):
                idx[t, j] = e
                w[t, j] = s[t, e] * scale / (total if normalize else 1.0)
                counts[b, e] += 1
            P[b] += s[t] / (s[t].sum() + 1e-20)
            n[b] += 1
            zsum += lse[t] ** 2
    used, N = max(1, int((n > 0).sum())), max(1, int(n.sum()))
    nn = np.maximum(n, 1)[:, None].astype(np.float64)
    balance = (E * counts / (k * nn) * P / nn).sum() / used
    return dict(idx=idx, w=w, s=s, soft=softs, lse=lse, live=live, counts=counts, seq_tokens=np.concatenate([n, [n.sum(), (n > 0).sum()]]),
                losses=np.array([balance, zsum / N]), nn=nn, used=used, N=N)


def chosen_value(l, r, dw, dbal, dz, k, score, normalize, scale, offsets=None):
    """sum dw w + dbal balance + dz z with the selection and counts of `r` held fixed: what the
    backward is the gradient of."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    offsets = np.array([0, T]) if offsets is None else np.asarray(offsets)
    total = 0.0
    for b in range(len(offsets) - 1):
        for t in range(offsets[b], offsets[b + 1]):
            if not r["live"][t]:
                continue
            on = l[t] > -np.inf
            top = l[t][on].max()
            ex = np.where(on, np.exp(np.where(on, l[t], 0.0) - top), 0.0)
            lse = top + math.log(ex.sum())
            s = ex / ex.sum() if score == "softmax" else np.where(on, 1.0 / (1.0 + np.exp(-np.where(on, l[t], 0.0))), 0.0)
            pick = r["idx"][t][r["idx"][t] >= 0]
            base = s[pick].sum() + 1e-20 if normalize else 1.0
            total += (dw[t][: len(pick)] * s[pick] / base * scale).sum()
            share = s / (s.sum() + 1e-20)
            total += dbal * (E * r["counts"][b] / (k * r["nn"][b, 0] ** 2) * share).sum() / r["used"]
            total += dz * lse ** 2 / r["N"]
    return total


def route_backward(l, r, dw, dbal, dz, k, score, normalize, scale, offsets=None):
    """(gradient, the sum of the magnitudes that make it up) of chosen_value, by the formulas."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    offsets = np.array([0, T]) if offsets is None else np.asarray(offsets)
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    for b in range(len(offsets) - 1):
        a = dbal * E * r["counts"][b] / (k * r["nn"][b, 0] ** 2) / r["used"]
        for t in range(offsets[b], offsets[b + 1]):
            if not r["live"][t]:
                continue
            on = l[t] > -np.inf
            s = r["s"][t]
            soft = r["soft"][t]
            pick = r["idx"][t][r["idx"][t] >= 0]
            g, gm = np.zeros(E), np.zeros(E)
            d = dw[t][: len(pick)]
            if normalize:
                base = s[pick].sum() + 1e-20
                g[pick] = scale / base * (d - (d * s[pick]).sum() / base)
                gm[pick] = scale / base * (np.abs(d) + (np.abs(d) * s[pick]).sum() / base)
            else:
                g[pick] = scale * d
                gm[pick] = np.abs(g[pick])
            if score == "softmax":
                g = g + a
                gm = gm + np.abs(a)
                dl = s * (g - (s * g).sum())
                mag = s * (gm + (s * gm).sum())
            else:
                Z = s.sum() + 1e-20
                g = g + (a - (s * a).sum() / Z) / Z
                gm = gm + (np.abs(a) + (s * np.abs(a)).sum() / Z) / Z
                dl = s * (1.0 - s) * g
                mag = s * gm                         # 1 - s carries an absolute error of s's
            z = dz * 2.0 / r["N"] * r["lse"][t] * soft
            grad[t] = np.where(on, dl + z, 0.0)
            # lse = max + log(sum) may cancel: its error is that of its parts
            size[t] = np.where(on, mag + np.abs(dz) * 2.0 / r["N"] * (np.abs(r["lse"][t]) + 2.0 * np.abs(l[t][on]).max() + 1.0) * soft, 0.0)
    return grad, size


def norm(arrays, p):
    flat = np.concatenate([np.asarray(a, np.float64).ravel() for a in arrays]) if arrays else np.zeros(0)
    if p == 2:
        top = np.abs(flat).max() if flat.size else 0.0
        return 0.0 if top == 0 else top * math.sqrt(((flat / top) ** 2).sum()) if np.isfinite(top) else top
    if p == 1:
        return np.abs(flat).sum()
    return np.abs(flat).max() if flat.size else 0.0


def adamw(p, g, m, v, t, lr, b1, b2, eps, wd, f):
    g = g * f
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p - lr * (wd * p + m / (1 - b1 ** t) / (np.sqrt(v / (1 - b2 ** t)) + eps))
    return p, m, v
