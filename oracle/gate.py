"""Oracle: routing of given logits and its gradient, float64, one token at a
time.

Test infrastructure only; see the package docstring.

Launch post ("Introducing Beam"), section "Mixture of Experts", and the
transformers model doc "Beam", section "Overview", for sigmoid scores, the
selection bias and the groups; softmax scores, groups ranked by their best
key and weights without renormalisation are the other usual forms.
Readings: a logit of -inf or NaN masks its expert (score 0, key -inf); a key of
-inf or NaN is -inf; equal keys and equal group scores go to the lower index;
where every chosen score is 0 the weights are 0.
"""

import numpy as np


def scores(z, kind):
    z = np.asarray(z, dtype=np.float64)
    on = z > -np.inf  # False for NaN
    f = np.zeros_like(z)
    if kind == "sigmoid":
        e = np.exp(-np.abs(z[on]))
        f[on] = np.where(z[on] >= 0, 1.0, e) / (1.0 + e)
    elif on.any():
        m = z[on].max()
        with np.errstate(invalid="ignore"):
            e = np.where(z[on] == m, 1.0, np.exp(z[on] - m))
        f[on] = e / e.sum()
    return f, on


def gate(z, top_k, bias=None, kind="sigmoid", n_group=1, topk_group=1, group_score="top2",
         renormalise=True, rsf=1.0, valid=None):
    """(idx [T, k] int32, w [T, k], counts [E])."""
    z = np.asarray(z, dtype=np.float64)
    T, E = z.shape
    idx = np.full((T, top_k), -1, dtype=np.int32)
    w = np.zeros((T, top_k))
    counts = np.zeros(E, dtype=np.int64)
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        f, on = scores(z[t], kind)
        key = f if bias is None else f + np.asarray(bias, dtype=np.float64)
        key = np.where(on & (key > -np.inf), key, -np.inf)
        cand = np.arange(E)
        if n_group > 1:
            g = key.reshape(n_group, -1)
            top = -np.sort(-g, axis=1)
            gs = top[:, :2].sum(axis=1) if group_score == "top2" else top[:, 0]
            kept = np.sort(np.argsort(-gs, kind="stable")[:topk_group])
            cand = np.concatenate([np.arange(E).reshape(n_group, -1)[i] for i in kept])
        pick = cand[np.argsort(-key[cand], kind="stable")[:top_k]]
        p = f[pick]
        if renormalise:
            p = p / p.sum() if p.sum() > 0 else 0.0 * p
        idx[t], w[t] = pick, rsf * p
        counts[pick] += 1
    return idx, w, counts


def gate_backward(dw, z, idx, kind="sigmoid", renormalise=True, rsf=1.0):
    """Gradient of the logits [T, E]; slots with an index outside [0, E) are empty,
    and so are a masked expert's, whatever arrives there."""
    z, dw = np.asarray(z, dtype=np.float64), np.asarray(dw, dtype=np.float64)
    T, E = z.shape
    dz = np.zeros((T, E))
    for t in range(T):
        f, on = scores(z[t], kind)
        slots = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E and on[idx[t, j]]]
        e = idx[t, slots]
        p, d = f[e], dw[t, slots]
        if renormalise:
            S = p.sum()
            df = rsf / S * (d - (d * p).sum() / S) if S > 0 else 0.0 * d
        else:
            df = rsf * d
        dfull = np.zeros(E)
        np.add.at(dfull, e, df)
        if kind == "sigmoid":
            dz[t] = dfull * f * (1.0 - f)
        else:
            dz[t] = f * (dfull - (dfull * f).sum())
    return dz
