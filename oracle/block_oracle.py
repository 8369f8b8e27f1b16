"""The operators inside a block in fp64, from their definitions: attention over packed sequences
with a relative position bias by buckets, and the tokens' way to the experts and back, each with
its gradients.  Test infrastructure; shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def _spans(offsets, rows):
    """[start, end) of every sequence; bounds outside the rows are taken as the nearest."""
    if offsets is None:
        return [(0, rows)]
    b = [min(max(int(v), 0), rows) for v in offsets]
    return [(a, max(a, c)) for a, c in zip(b, b[1:])]


def attention_pairs(nq, nk, *, causal=False, window=0, mask=None):
    """(seen, distance), queries x keys of one sequence: query i stands at key position i + nk - nq."""
    dist = np.arange(nk)[None, :] - (np.arange(nq)[:, None] + nk - nq)
    seen = np.ones((nq, nk), bool)
    if causal:
        seen &= dist <= 0
    if window:
        seen &= np.abs(dist) < window
    if mask is not None:
        seen &= np.asarray(mask, bool)[None, :]
    return seen, dist


def attention(q, k, v, *, offsets=None, key_offsets=None, mask=None, bias=None, bucket_map=None, scale=1.0, causal=False,
              window=0, grad_out=None):
    """dict(out, lse) and, with grad_out, q, k, v, bias (the gradients); `parts` lists what every sequence and head was formed
    from: (query rows, key rows, head, key head, scores, p, dp, dz, seen, buckets)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    heads, group = q.shape[1], q.shape[1] // k.shape[1]
    out, lse = np.zeros_like(q), np.full(q.shape[:2], -np.inf)
    res = dict(out=out, lse=lse, parts=[])
    if grad_out is not None:
        do = np.asarray(grad_out, np.float64)
        res.update(q=np.zeros_like(q), k=np.zeros_like(k), v=np.zeros_like(v))
    if bias is not None:
        bias = np.asarray(bias, np.float64)
        reach = len(bucket_map) // 2
        if grad_out is not None:
            res["bias"] = np.zeros_like(bias)
    for (q0, q1), (k0, k1) in zip(_spans(offsets, len(q)), _spans(offsets if key_offsets is None else key_offsets, len(k))):
        seen, dist = attention_pairs(q1 - q0, k1 - k0, causal=causal, window=window, mask=None if mask is None else mask[k0:k1])
        bucket = None if bias is None else np.asarray(bucket_map)[np.clip(dist, -reach, reach) + reach]
        alive = seen.any(1)
        if not alive.any():
            continue
        keys = np.nonzero(seen.any(0))[0]                    # what the others hold does not matter
        s, rows, cols = seen[np.ix_(alive, keys)], q0 + np.nonzero(alive)[0], k0 + keys
        b = None if bias is None else bucket[np.ix_(alive, keys)]
        for h in range(heads):
            g = h // group
            qh, kh, vh = q[rows, h], k[cols, g], v[cols, g]
            z = scale * (qh @ kh.T)
            if bias is not None:
                inside = (b >= 0) & (b < len(bias))
                z = z + np.where(inside, bias[np.where(inside, b, 0), h], 0.0)
            z = np.where(s, z, -np.inf)
            top = z.max(1, keepdims=True)
            e = np.exp(z - np.where(np.isfinite(top), top, 0.0))
            total = e.sum(1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[rows, h] = (top + np.log(total))[:, 0]
            p = e / np.where(total == 0, 1.0, total)
            o = p @ vh
            out[rows, h] = o
            part = dict(rows=rows, cols=cols, head=h, kv=g, z=z, p=p, seen=s, bucket=b)
            if grad_out is not None:
                d = do[rows, h]
                dp = d @ vh.T
                dz = p * (dp - (d * o).sum(1, keepdims=True))
                res["q"][rows, h] = scale * (dz @ kh)
                res["k"][cols, g] += scale * (dz.T @ qh)
                res["v"][cols, g] += p.T @ d
                if bias is not None:
                    np.add.at(res["bias"], (b[inside], h), dz[inside])
                part.update(dp=dp, dz=dz)
            res["parts"].append(part)
    return res


def expert_sort(x, experts, num_experts):
    """(sorted rows, slots, offsets): a stable order of the choices by their expert."""
    x, experts = np.asarray(x, np.float64), np.asarray(experts)
    tokens, chosen = experts.shape
    slots = np.full(tokens * chosen, -1, np.int64)
    rows, offsets = [], [0]
    for e in range(num_experts):
        for i in np.nonzero(experts.reshape(-1) == e)[0]:
            slots[i] = len(rows)
            rows.append(i // chosen)
        offsets.append(len(rows))
    out = np.zeros((tokens * chosen, x.shape[1]))
    out[:len(rows)] = x[rows]
    return out, slots.reshape(tokens, chosen), np.array(offsets)


def expert_sort_backward(grad_sorted, slots):
    g, slots = np.asarray(grad_sorted, np.float64), np.asarray(slots)
    return expert_combine(g, slots, np.ones(slots.shape))


def expert_combine(y, slots, weights):
    y, w, slots = np.asarray(y, np.float64), np.asarray(weights, np.float64), np.asarray(slots)
    out = np.zeros((slots.shape[0], y.shape[1]))
    for t, c in zip(*np.nonzero(slots >= 0)):
        out[t] += w[t, c] * y[slots[t, c]]
    return out


def expert_combine_backward(grad_out, y, slots, weights):
    """(gradient of y, gradient of weights)."""
    g, y, w, slots = np.asarray(grad_out, np.float64), np.asarray(y, np.float64), np.asarray(weights, np.float64), np.asarray(slots)
    gy, gw = np.zeros_like(y), np.zeros(slots.shape)
    for t, c in zip(*np.nonzero(slots >= 0)):
        gy[slots[t, c]] = w[t, c] * g[t]
        gw[t, c] = g[t] @ y[slots[t, c]]
    return gy, gw
