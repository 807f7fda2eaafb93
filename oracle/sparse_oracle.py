"""Plain float64 implementation of routing, expert layers and the embedding
table (include/muon.h states the operators).  Written as loops over tokens and
experts; test infrastructure only."""
from __future__ import annotations

import math

import numpy as np


def plan(choice: np.ndarray, experts: int):
    """(offsets, tokens, place) of a choice [tokens, k]."""
    t, k = choice.shape
    offsets = np.zeros(experts + 1, np.int64)
    tokens, place = np.full(t * k, -1), np.full((t, k), -1)
    row = 0
    for e in range(experts):
        offsets[e] = row
        for i in range(t):
            for j in range(k):
                if choice[i, j] == e:
                    tokens[row], place[i, j] = i, row
                    row += 1
    offsets[experts] = row
    return offsets, tokens, place


def route(logits: np.ndarray, k: int, normalize: bool):
    """(gates, chosen) of logits [tokens, experts]."""
    t, n = logits.shape
    gates, chosen = np.zeros((t, k)), np.full((t, k), -1)
    for i in range(t):
        l = [float(v) for v in logits[i]]

        def before(e):   # NaN first, then the largest, then the lowest expert
            return (0 if math.isnan(l[e]) else 1, 0.0 if math.isnan(l[e]) else -l[e], e)
        some = sorted((e for e in range(n) if l[e] != -math.inf), key=before)[:k]
        if not some:
            continue
        over = some if normalize else [e for e in range(n) if l[e] != -math.inf]
        if any(math.isnan(l[e]) or l[e] == math.inf for e in range(n)):
            p = [math.nan] * len(some)
        else:
            top = max(l)
            total = math.fsum(math.exp(l[e] - top) for e in over)
            p = [math.exp(l[e] - top) / total for e in some]
        chosen[i, :len(some)] = some
        gates[i, :len(some)] = p
    return gates, chosen


def route_grad(dgates: np.ndarray, logits: np.ndarray, gates: np.ndarray, chosen: np.ndarray, normalize: bool):
    """Gradient with respect to the logits, from the Jacobian of the softmax."""
    t, n = logits.shape
    out = np.zeros((t, n))
    for i in range(t):
        slots = [j for j in range(chosen.shape[1]) if 0 <= chosen[i, j] < n]
        if not slots:
            continue
        if normalize:
            p = np.zeros(n)
            for j in slots:
                p[chosen[i, j]] = gates[i, j]
        else:
            p = np.exp(logits[i] - logits[i].max())
            p /= p.sum()
        for j in slots:
            c = chosen[i, j]
            out[i] += dgates[i, j] * p[c] * ((np.arange(n) == c) - p)
    return out


def rows_of(x: np.ndarray, tokens: np.ndarray) -> np.ndarray:
    """The tokens' rows in sorted order; NaN behind the last expert's."""
    out = np.full((len(tokens), x.shape[1]), np.nan)
    for r, t in enumerate(tokens):
        if t >= 0:
            out[r] = x[t]
    return out


def linear(x, w, offsets):
    out = np.full((x.shape[0], w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        for r in range(offsets[e], offsets[e + 1]):
            out[r] = w[e] @ x[r]
    return out


def linear_grad(dy, w, x, offsets):
    dx, dw = np.full(x.shape, np.nan), np.zeros(w.shape)
    for e in range(w.shape[0]):
        for r in range(offsets[e], offsets[e + 1]):
            dx[r] = w[e].T @ dy[r]
            dw[e] += np.outer(dy[r], x[r])
    return dx, dw


def combine(y, gates, place):
    out = np.zeros((place.shape[0], y.shape[1]))
    for t in range(place.shape[0]):
        for j in range(place.shape[1]):
            if place[t, j] >= 0:
                out[t] += gates[t, j] * y[place[t, j]]
    return out


def combine_grad(dout, y, gates, place):
    dy, dgates = np.full(y.shape, np.nan), np.zeros(place.shape)
    for t in range(place.shape[0]):
        for j in range(place.shape[1]):
            if place[t, j] >= 0:
                dy[place[t, j]] = gates[t, j] * dout[t]
                dgates[t, j] = dout[t] @ y[place[t, j]]
    return dy, dgates


def embedding(ids, w, scale):
    out = np.zeros((len(ids), w.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < w.shape[0]:
            out[t] = scale * w[i]
    return out


def embedding_grad(dy, ids, rows, scale):
    dw = np.zeros((rows, dy.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < rows:
            dw[i] += scale * dy[t]
    return dw
