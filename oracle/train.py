"""The training and adapter operators beside the layer, on the CPU in float64.

TEST INFRASTRUCTURE ONLY, like the rest of this package: written from the
definitions (include/moe.h states them), sharing no code with the GPU path.
tests/test_oracle_train.py pins the gradients to differences of the forward
functions.
"""
from __future__ import annotations

import numpy as np


def softmax(logits):
    """p and log-sum-exp of each row; NaN as -inf, a row without any logit above
    -inf gives p = 0 and lse = 0."""
    z = np.asarray(logits, np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    m = z.max(axis=1, keepdims=True)
    none = m[:, 0] == -np.inf
    with np.errstate(invalid="ignore"):
        e = np.exp(z - np.where(none[:, None], 0.0, m))
        s = e.sum(axis=1, keepdims=True)
        p = e / np.where(none[:, None], 1.0, s)
        lse = np.where(none, 0.0, m[:, 0] + np.log(np.where(none, 1.0, s[:, 0])))
    return p, lse


def sequences(tokens, offsets, mask):
    """[(sequence, its tokens that count)] and, per token, whether it is in any."""
    offsets = [0, tokens] if offsets is None else list(offsets)
    on = np.ones(tokens, bool) if mask is None else np.asarray(mask) != 0
    spans, inside = [], np.zeros(tokens, bool)
    for s in range(len(offsets) - 1):
        t = np.arange(offsets[s], offsets[s + 1])
        inside[t] = True
        spans.append((s, t[on[t]]))
    return spans, inside


def router_loss(logits, ids, offsets=None, mask=None):
    T, E = logits.shape
    k = ids.shape[1]
    p, lse = softmax(logits)
    spans, _ = sequences(T, offsets, mask)
    S = len(spans)
    counts, mean = np.zeros((S, E), np.int64), np.zeros((S, E))
    n = np.zeros(S, np.int64)
    for s, t in spans:
        n[s] = len(t)
        if len(t):
            counts[s] = np.bincount(ids[t].reshape(-1), minlength=E)
            mean[s] = p[t].mean(axis=0)
    live, total = int((n > 0).sum()), int(n.sum())
    f = E * counts / (k * np.maximum(n, 1))[:, None]
    every = np.concatenate([t for _, t in spans])
    losses = np.array([(f * mean).sum() / max(live, 1), (lse[every] ** 2).sum() / max(total, 1)])
    return dict(losses=losses, counts=counts, mean_probs=mean,
                seq_tokens=np.concatenate([n, [total, live]]))


def router_backward(logits, ids, offsets=None, mask=None, weights=None, dweights=None, dlosses=None,
                    counts=None, seq_tokens=None):
    """(dlogits, magnitude): magnitude is the sum of the absolute terms of each
    element, the scale of its rounding errors.  Rows in no sequence: NaN."""
    T, E = logits.shape
    k = ids.shape[1]
    p, lse = softmax(logits)
    z = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    some = z.max(axis=1) > -np.inf
    spans, inside = sequences(T, offsets, mask)
    g, mag = np.zeros((T, E)), np.zeros((T, E))
    for s, t in spans:
        t = t[some[t]]
        if not len(t):
            continue
        if dlosses is not None:
            f = E * counts[s] / (k * seq_tokens[s])
            c = dlosses[0] / (seq_tokens[-1] * seq_tokens[s])
            dot = (p[t] * f).sum(axis=1, keepdims=True)
            q = 2.0 * dlosses[1] / seq_tokens[-2]
            g[t] += p[t] * ((f - dot) * c + lse[t, None] * q)
            big = np.abs(z[t].max(axis=1, keepdims=True)) + np.log(E) + 1.0
            mag[t] += p[t] * ((f + dot) * abs(c) + big * abs(q))
        if dweights is not None:
            wd = weights[t] * dweights[t]
            term = wd - weights[t] * wd.sum(axis=1, keepdims=True)
            size = np.abs(wd) + weights[t] * np.abs(wd).sum(axis=1, keepdims=True)
            for j in range(k):
                np.add.at(g, (t, ids[t, j]), term[:, j])
                np.add.at(mag, (t, ids[t, j]), size[:, j])
    g[~inside] = np.nan
    return g, mag


def finalize_backward(dout, weights, y2, slot_row):
    """(dweights, sum of |terms| of each dweights, dy2 of each (token, slot))."""
    d = np.asarray(dout, np.float64)[:, None, :]
    y = np.asarray(y2, np.float64)[slot_row]
    return (d * y).sum(axis=2), np.abs(d * y).sum(axis=2), np.asarray(weights, np.float64)[:, :, None] * d


def adapter_apply(x, adapter_ids, a, b, scale, base):
    out = np.array(base, np.float64)
    for i in range(a.shape[0]):
        t = np.nonzero(adapter_ids == i)[0]
        out[t] += scale[i] * (x[t] @ a[i].T) @ b[i]
    return out


def adapter_backward(dout, x, adapter_ids, a, b, scale, dx_base):
    """dx, da, db."""
    dx = np.array(dx_base, np.float64)
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    for i in range(a.shape[0]):
        t = np.nonzero(adapter_ids == i)[0]
        v = scale[i] * dout[t] @ b[i].T
        dx[t] += v @ a[i]
        da[i] = v.T @ x[t]
        db[i] = scale[i] * (x[t] @ a[i].T).T @ dout[t]
    return dx, da, db
