"""fp64 reference of expert routing, grouping by expert and the sum of expert outputs, one
token at a time.  numpy only; no code is shared with the HIP path."""
import numpy as np


def ref_scores(logits, scoring):
    """Scores of one token; -inf and NaN logits score 0, infinite ones share a softmax."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, dtype=np.float64))
    out = l == -np.inf
    with np.errstate(all="ignore"):
        if scoring == "sigmoid":
            return np.where(out, 0.0, 1.0 / (1.0 + np.exp(-l)))
        if out.all():
            return np.zeros_like(l)
        m = l.max()
        p = np.where(out, 0.0, np.where(l == m, 1.0, np.exp(np.where(l == m, 0.0, l - m))))
    return p / p.sum()


def ref_route_token(logits, top_k, bias=None, scoring="softmax", n_groups=1, top_groups=None, group_score="max",
                    renormalize=True, scale=1.0):
    """(ids, weights) of one token: groups ranked first, then one expert after another."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, dtype=np.float64))
    s = ref_scores(l, scoring)
    with np.errstate(invalid="ignore"):
        c = l if bias is None else s + np.asarray(bias, dtype=np.float64)
    c = np.where((l == -np.inf) | np.isnan(c), -np.inf, c)
    top_groups = n_groups if top_groups is None else top_groups
    per = len(l) // n_groups
    by = np.where(c == -np.inf, -np.inf, s) if bias is None and group_score == "top2" else c
    ranks = []
    for g in range(n_groups):
        v = sorted((x for x in by[g * per:(g + 1) * per] if x != -np.inf), reverse=True)
        ranks.append(-np.inf if not v else v[0] + v[1] if group_score == "top2" and len(v) > 1 else v[0])
    kept = sorted(range(n_groups), key=lambda g: (-ranks[g], g))[:top_groups]
    can = [e for e in range(len(l)) if e // per in kept and c[e] != -np.inf]
    ids = sorted(can, key=lambda e: (-c[e], e))[:top_k]
    w = s[ids]
    if renormalize:
        w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
    pad = top_k - len(ids)
    return np.array(ids + [-1] * pad, dtype=np.int32), np.concatenate([scale * w, np.zeros(pad)])


def ref_route(logits, top_k, **kw):
    got = [ref_route_token(row, top_k, **kw) for row in logits]
    return np.array([g[0] for g in got]).reshape(-1, top_k), np.array([g[1] for g in got]).reshape(-1, top_k)


def ref_group(ids, n_experts):
    """(offsets, row_index, place) by appending every choice to its expert's list."""
    lists = [[] for _ in range(n_experts)]
    tokens, k = ids.shape
    for t in range(tokens):
        for j in range(k):
            if 0 <= ids[t, j] < n_experts:
                lists[ids[t, j]].append((t, j))
    offsets = np.cumsum([0] + [len(x) for x in lists]).astype(np.int64)
    rows, place = np.full(tokens * k, -1, np.int32), np.full((tokens, k), -1, np.int32)
    for p, (t, j) in enumerate(x for l in lists for x in l):
        rows[p], place[t, j] = t, p
    return offsets, rows, place


def ref_combine(y, place, weights):
    """(out, B): sums in fp64 and the sums of magnitudes."""
    y = np.asarray(y, dtype=np.float64)
    out, size = np.zeros((place.shape[0], y.shape[1])), np.zeros((place.shape[0], y.shape[1]))
    for t in range(place.shape[0]):
        for p, w in zip(place[t], weights[t]):
            if 0 <= p < y.shape[0]:
                out[t] += float(w) * y[p]
                size[t] += abs(float(w)) * np.abs(y[p])
    return out, size
