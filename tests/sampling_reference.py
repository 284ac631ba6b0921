"""The sampling operators in 64 bits, row by row, from their definitions: what the GPU tests compare
with.  Besides each answer the functions say how far it is from another one (margin): the distance
of the nearest filter border, or of the uniform from the nearest step of the running sum, as a share
of the mass it is measured against.  Kernels hold weights as integers good to 2^-39 of themselves and
2^-44 of the largest: sums of V of them are off by 2^-39 of themselves and, with V <= 2^18 roundings
that are as good as independent, by 2^-44 * 2^9 of the largest weight: both below 1e-10.  A float32
row's sums take weights with y = e^z - 1, |z| < 2^-8.5, in one float: four roundings of 2^-33 of the
weight, 4.7e-10 if all of them agree.  Answers with a larger margin than MARGIN have to be equal."""
import numpy as np

MARGIN = 1e-9


def row_truth(l, T, top_k=0, top_p=1.0, min_p=0.0, u=None):
    """One row of float64 logits (exact values of the stored ones)."""
    l = np.asarray(l, np.float64)
    V = len(l)
    T = float(np.float32(T))
    if np.isnan(l).any() or (l == np.inf).any() or (l == -np.inf).all():
        return {"status": 5}
    if not (T >= 0 and np.isfinite(T)) or 0 < T < 1.17549435e-38 or not top_p > 0 or not min_p < 1:
        return {"status": 1}
    if u is not None and not 0 <= u < 1:
        return {"status": 7}
    m = l.max()
    margin = np.inf
    if T == 0:
        keep = np.zeros(V, bool)
        keep[int(np.argmax(l))] = True
        w = keep.astype(np.float64)
        S = 1.0
    else:
        w = np.exp((l - m) / T)
        S = w.sum()
        order = np.lexsort((np.arange(V), -l))
        ls, ws = l[order], w[order]
        start = np.r_[True, ls[1:] != ls[:-1]]
        first = np.maximum.accumulate(np.where(start, np.arange(V), 0))
        above = np.r_[0.0, np.cumsum(ws)[:-1]][first]
        ok = ls > -np.inf
        if top_k > 0:
            ok &= first < top_k
        if top_p < 1:
            ok &= above < top_p * S
            # the first group is kept whatever its border
            if (first > 0).any():
                margin = min(margin, np.min(np.abs(above[first > 0] / S - top_p)))
        if min_p > 0:
            ok &= ws >= min_p
            fin = ls > -np.inf
            margin = min(margin, np.min(np.abs((ls[fin] - m) / T - np.log(min_p))))
        keep = np.zeros(V, bool)
        keep[order[ok]] = True
    E = w[keep].sum()
    out = {"status": 0, "kept": int(keep.sum()), "keep": keep, "mass": E / S,
           "probs": np.where(keep, w, 0.0) / E, "cut_margin": margin}
    if u is not None:
        at = np.flatnonzero(keep)
        at = at[np.lexsort((at, -l[at]))]
        run = np.cumsum(w[at])
        i = min(int(np.searchsorted(run, u * E, side="right")), len(at) - 1)
        while w[at[i]] == 0:
            i -= 1
        out["token"] = int(at[i])
        out["draw_margin"] = float(np.min(np.abs(np.r_[run[:-1], np.inf] / E - u)))
        out["p_token"] = out["probs"][at[i]]
    return out


def logprob_truth(l, x, T, top_n=0):
    l = np.asarray(l, np.float64)
    T = float(np.float32(T))
    if not 0 <= x < len(l):
        return {"status": 4}
    if np.isnan(l).any() or (l == np.inf).any() or (l == -np.inf).all():
        return {"status": 5}
    d = (l - l.max()) / T
    lp = d - np.log(np.exp(d).sum())
    order = np.lexsort((np.arange(len(l)), -l))
    order = order[l[order] > -np.inf][:top_n]
    ids, val = np.full(top_n, -1), np.full(top_n, np.nan)
    ids[:len(order)], val[:len(order)] = order, lp[order]
    return {"status": 0, "logprob": lp[x], "rank": 1 + int((l > l[x]).sum()), "top_tokens": ids,
            "top_logprobs": val}
