"""64-bit references of the tree, sampling and distillation calls, from their
formulas (numpy, on the CPU)."""
import math

import numpy as np


def attention(q, k_new, v_new, k_cache, v_cache, table, ctx, sees, tree_len, scale):
    """All arrays float64 numpy, k_cache [pages, page, H, D]; sees bool [N, T, T].
    -> out, lse, and per output the weighted mean of |v| and the largest sum of |q||k| scale seen."""
    N, T, HQ, D = q.shape
    H, page = k_cache.shape[2], k_cache.shape[1]
    g = HQ // H
    out, mag = np.zeros((N, T, HQ, D)), np.zeros((N, T, HQ, D))
    lse, reach, flat = np.full((N, T, HQ), -np.inf), np.zeros((N, T, HQ)), np.zeros((N, T, HQ, D))
    for n in range(N):
        pos = np.arange(ctx[n])
        kc, vc = k_cache[table[n, pos // page], pos % page], v_cache[table[n, pos // page], pos % page]
        for t in range(min(T, tree_len[n])):
            nodes = np.flatnonzero(sees[n, t, :tree_len[n]])
            for hq in range(HQ):
                h = hq // g
                k = np.concatenate([kc[:, h], k_new[n, nodes, h]])
                v = np.concatenate([vc[:, h], v_new[n, nodes, h]])
                if len(k) == 0:
                    continue
                s = k @ q[n, t, hq] * scale
                m = s.max()
                w = np.exp(s - m)
                out[n, t, hq] = w @ v / w.sum()
                mag[n, t, hq] = w @ np.abs(v) / w.sum()
                flat[n, t, hq] = np.abs(v).sum(0) / w.sum()
                lse[n, t, hq] = m + math.log(w.sum())
                reach[n, t, hq] = (np.abs(k) @ np.abs(q[n, t, hq])).max() * abs(scale)
    return out, lse, mag, reach, flat


def walk(tokens, parents, sampled, length):
    if length == 0:
        return [], -1
    path = [0]
    while True:
        cur = path[-1]
        nxt = [t for t in range(cur + 1, length) if parents[t] == cur and tokens[t] == sampled[cur]]
        if not nxt:
            return path, sampled[cur]
        path.append(nxt[0])


def sample_row(x, u, t=None, k=0, p=1.0, q=0.0):
    """-> (token, logprob, how near the draw or a border is to another outcome, as a share of the mass)."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    m = x.max()
    if m == -np.inf:
        return -1, -np.inf, 1.0
    t = 1.0 if t is None or np.isnan(t) else float(t)
    if t <= 0:
        return int(np.argmax(x)), 0.0, 1.0
    with np.errstate(invalid="ignore"):
        z = np.where(x == m, 0.0, (x - m) / t)
    by = np.argsort(-x, kind="stable")
    w = np.exp(z)
    near = 1.0
    if k > 0:
        by = by[:k]
    if not np.isnan(p) and p < 1:
        mass = np.cumsum(w[by])
        before = np.concatenate([[0.0], mass[:-1]])
        near = min(near, float(np.abs(mass - p * mass[-1]).min() / mass[-1])) if p > 0 else near
        n = max(1, int((before < max(p, 0.0) * mass[-1]).sum()))
        by = by[:n]
    if not np.isnan(q) and q > 0:
        keep = z[by] >= math.log(min(q, 1.0))
        with np.errstate(invalid="ignore"):
            edge = np.abs(z[by] - math.log(min(q, 1.0)))
        if q < 1:
            near = min(near, float(edge.min()))
        by = by[keep]
    kept = np.zeros_like(w)
    kept[by] = w[by]
    cum = np.cumsum(kept)
    target = (0.0 if np.isnan(u) else float(u)) * cum[-1]
    tok = int(np.searchsorted(cum, target, side="right"))
    tok = min(tok, int(np.flatnonzero(kept)[-1]))
    if target > 0:
        near = min(near, float(np.abs(cum - target).min() / cum[-1]))
    return tok, z[tok] - math.log(cum[-1]), near


def distill_row(x, ids, teacher, T, teacher_lse=None):
    """-> loss, lse, gradient (of this row's loss)."""
    x = x.astype(np.float64)
    z = x / T
    m = z.max()
    lse = m + math.log(np.exp(z - m).sum())
    ok = (ids >= 0) & (ids < len(x))
    ids, t = ids[ok], teacher[ok].astype(np.float64) / T
    grad = np.zeros_like(z)
    if len(ids) == 0 or t.max() == -np.inf:
        return 0.0, lse, grad
    t_lse = t.max() + math.log(np.exp(t - t.max()).sum()) if teacher_lse is None else float(teacher_lse)
    p = np.exp(t - t_lse)
    on = p > 0
    loss = T * T * float((p[on] * (t[on] - t_lse - z[ids[on]] + lse)).sum())
    grad = p.sum() * np.exp(z - lse)
    np.subtract.at(grad, ids, p)
    return loss, lse, grad * T
