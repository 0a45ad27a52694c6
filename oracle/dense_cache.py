"""Plain fp64 CPU oracle of a densely attended layer's cache: the decode
attention of one new token, the attention weight that queries give every key,
and the choice of the tokens that stay when a cache is cut to a budget.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports, calls or links
this module: only the tests may use it.  It shares no code with the CUDA path.

Readings (the MSA pages describe the sparse method; these are the plain forms
of what a dense layer's cache needs next to it):

* query head h belongs to group g = h // (H / G); scores are scaled by sm_scale
  and softmax runs over every key the query sees;
* the weight of key j for group g is the sum over queries and the group's heads
  of exp(s_j - lse), lse an argument (the attention's log-sum-exp);
* eviction: with L <= budget every token stays.  Otherwise the first n_sink and
  the last n_recent stay, and the best others by score up to budget; ties go to
  the lower index; NaN ranks last.  The score of a token is the group's weight,
  or the sum over the groups in 64 bits, rounded once to 32 bits.
"""
from __future__ import annotations

import numpy as np

__all__ = ["decode_attention", "key_weights", "evict_select"]


def decode_attention(q, k, v, sm_scale: float):
    """q [H, d], k / v [L, G, d] -> out [H, d], lse [H], weights [G, L], and
    mass [H, d] = sum_j p_j |v_j| (for error bounds)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    H, d = q.shape
    L, G, _ = k.shape
    out, mass = np.zeros((H, d)), np.zeros((H, d))
    lse, w = np.full(H, -np.inf), np.zeros((G, L))
    for h in range(H):
        g = h // (H // G)
        s = (k[:, g] @ q[h]) * sm_scale
        top = s.max() if L else -np.inf
        if top == -np.inf:
            continue
        e = np.exp(s - top)
        lse[h] = top + np.log(e.sum())
        p = e / e.sum()
        out[h], mass[h] = p @ v[:, g], p @ np.abs(v[:, g])
        w[g] += p
    return out, lse, w, mass


def key_weights(q, k, lse, sm_scale: float):
    """q [T, H, d]: the last T of the S tokens; k [S, G, d]; lse [T, H].
    Returns [G, S]: sum over queries that see key j and the group's heads of
    exp(s_j - lse); a query whose lse is -inf has seen nothing and adds nothing."""
    q, k, lse = (np.asarray(x, np.float64) for x in (q, k, lse))
    T, H, _ = q.shape
    S, G, _ = k.shape
    w = np.zeros((G, S))
    for t in range(T):
        n = S - T + t + 1
        for h in range(H):
            if lse[t, h] == -np.inf:
                continue
            g = h // (H // G)
            w[g, :n] += np.exp((k[:n, g] @ q[t, h]) * sm_scale - lse[t, h])
    return w


def evict_select(weights, budget: int, n_sink: int, n_recent: int, per_group: bool):
    """weights [G, L] float32 -> kept [R, min(L, budget)] ascending (R = G or 1)."""
    weights = np.asarray(weights, np.float32)
    G, L = weights.shape
    rows = weights if per_group else weights.astype(np.float64).sum(0, keepdims=True).astype(np.float32)
    kept = []
    for row in rows:
        if L <= budget:
            kept.append(np.arange(L))
            continue
        middle = range(n_sink, L - n_recent)
        rank = sorted(middle, key=lambda j: (np.isnan(row[j]), 0.0 if np.isnan(row[j]) else -float(row[j]), j))
        stay = list(range(n_sink)) + rank[:budget - n_sink - n_recent] + list(range(L - n_recent, L))
        kept.append(np.array(sorted(stay)))
    return np.stack(kept)
