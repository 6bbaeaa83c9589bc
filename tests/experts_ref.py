"""Plain references of the mixture-of-experts operators, in 64 bits and without the library: the
routing and its gradient, the plan of the expert-ordered rows, and the gather."""
import numpy as np


def scores(logits, sigmoid):
    l = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-l))
        e = np.exp(l - l.max(axis=1, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)


def log_scores(logits, sigmoid):
    l = np.asarray(logits, np.float64)
    if sigmoid:
        return np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
    return l - l.max(axis=1, keepdims=True)  # up to a constant of the row


def route(logits, k, bias=None, sigmoid=False, groups=1, top_groups=1, renorm=True, scale=1.0):
    """(experts [T, k], weights [T, k] float64), one row at a time."""
    T, E = logits.shape
    experts = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        l = np.asarray(logits[t], np.float64)
        if np.isnan(l).any() or (l == np.inf).any():
            continue
        open_ = l > -np.inf
        if not open_.any():
            continue
        s = scores(l[None], sigmoid)[0]
        plain = bias is None and groups == 1
        v = l.copy() if plain else s + (0.0 if bias is None else np.asarray(bias, np.float64))
        if not plain and (np.isnan(v[open_]).any() or (v[open_] == np.inf).any()):
            continue
        v[~open_] = -np.inf
        if groups > 1:
            g = np.sort(v.reshape(groups, -1), axis=1)[:, ::-1]
            total = np.array([r[:2][r[:2] > -np.inf].sum() if r[0] > -np.inf else -np.inf for r in g])
            keep = np.argsort(-total, kind="stable")[:top_groups]
            outside = np.ones(groups, bool)
            outside[keep] = False
            v[np.repeat(outside, E // groups)] = -np.inf
        order = [e for e in np.argsort(-v, kind="stable")[:k] if v[e] > -np.inf]
        if not order:
            continue
        experts[t, :len(order)] = order
        if renorm:
            q = log_scores(l[None], sigmoid)[0][order]
            p = np.exp(q - q.max())
            weights[t, :len(order)] = scale * p / p.sum()
        else:
            weights[t, :len(order)] = scale * s[order]
    return experts, weights


def route_backward(logits, experts, dweights, sigmoid, renorm, scale):
    l = np.asarray(logits, np.float64)
    out = np.zeros_like(l)
    for t in range(l.shape[0]):
        pairs = [(e, scale * float(dweights[t, j])) for j, e in enumerate(experts[t]) if e >= 0]
        if not pairs:
            continue
        idx = [e for e, _ in pairs]
        g = np.array([d for _, d in pairs])
        rest = 1.0 / (1.0 + np.exp(l[t])) if sigmoid else np.ones(l.shape[1])
        if renorm:
            q = log_scores(l[t][None], sigmoid)[0][idx]
            p = np.exp(q - q.max())
            p /= p.sum()
            np.add.at(out[t], idx, p * rest[idx] * (g - (g * p).sum()))
        else:
            s = scores(l[t][None], sigmoid)[0]
            np.add.at(out[t], idx, s[idx] * rest[idx] * g)
            if not sigmoid:
                out[t] -= s * (g * s[idx]).sum()
    return out


def expert_rows(T, k, E):
    """Worst case by trial: one pair in as many experts as there are pairs, the rest in one."""
    pairs = T * k
    n = min(E, pairs)
    spread = [1] * (n - 1) + [pairs - (n - 1)]
    best = sum(-(-c // 128) * 128 for c in spread)
    # pushing a region just over a multiple of 128 can cost one more region
    extra = pairs - n
    return max(best, (n + extra // 128) * 128)


def plan(experts, E, rows):
    """(offsets, pair_row, row_token) in int32."""
    experts = np.asarray(experts)
    T, k = experts.shape
    offsets = np.zeros(E + 1, np.int32)
    pair_row = np.full((T, k), -1, np.int32)
    row_token = np.full(rows, -1, np.int32)
    at = 0
    for e in range(E):
        offsets[e] = at
        r = at
        for t, j in zip(*np.nonzero(experts == e)):
            pair_row[t, j] = r
            row_token[r] = t
            r += 1
        at += -(-(r - at) // 128) * 128
    offsets[E] = at
    return offsets, pair_row, row_token


def gather_bits(x_bits, row_token):
    """Rows of x (bf16 bits) in expert order, zeros where there is no token."""
    out = np.zeros((len(row_token), x_bits.shape[1]), np.uint16)
    has = row_token >= 0
    out[has] = x_bits[row_token[has]]
    return out


def routing(rng, T, E, k, pad=0, empty=()):
    """Distinct experts per token, none of the experts in `empty`, none for the last `pad` tokens."""
    allowed = np.array([e for e in range(E) if e not in set(empty)])
    popularity = rng.normal(size=len(allowed))
    noise = rng.gumbel(size=(T, len(allowed)))
    experts = allowed[np.argsort(-(popularity + noise), axis=1)[:, :k]].astype(np.int32)
    if pad:
        experts[T - pad:] = -1
    return experts
