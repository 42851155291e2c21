"""Penalties, biases and grammar masks on the verify rows' logits, the greedy
token and the target distribution, and the token table the penalties read.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

[P1] "阶段 3:拒绝采样与 Bitmask": the acceptance sees masked logits; [P2]
"接受判定:greedy 与 rejection sampling": argmax or distribution of every verify
row.  The penalties are the usual ones of sampling: repetition (tokens of the
prompt or the output: positive logits divided, others multiplied), frequency
(per occurrence in the output) and presence (once).  A verify row that follows
i drafts counts those drafts as output.
"""
from __future__ import annotations

import math

import numpy as np

COUNT_MAX = 32767


def token_counts_ld(V: int) -> int:
    return (V + 7) // 8 * 8


def token_counts_build(counts, tokens, offsets, V, n_prompt=None, count_rows=None):
    """The rows of the requests, rebuilt in a copy of counts [n_rows, ld] int16."""
    out = np.array(counts, dtype=np.int16)
    taken = set()
    for b in range(len(offsets) - 1):
        row = b if count_rows is None else int(count_rows[b])
        if row < 0 or row >= len(out) or row in taken:
            continue
        taken.add(row)
        seg = [int(t) for t in tokens[int(offsets[b]):int(offsets[b + 1])]]
        cut = len(seg) if n_prompt is None else int(n_prompt[b])
        n = [0] * out.shape[1]
        seen = [False] * out.shape[1]
        for j, t in enumerate(seg):
            if 0 <= t < V:
                if j < cut:
                    seen[t] = True
                else:
                    n[t] += 1
        out[row] = [min(c, COUNT_MAX) - (32768 if s else 0) for c, s in zip(n, seen)]
    return out


def token_counts_accept(counts, V, draft, num_accepted, next_tokens, count_rows=None):
    out = np.array(counts, dtype=np.int16)
    for b in range(len(next_tokens)):
        row = b if count_rows is None else int(count_rows[b])
        if row < 0 or row >= len(out):
            continue
        K = 0 if draft is None else draft.shape[1]
        n = 0 if K == 0 else max(0, min(int(num_accepted[b]), K))
        for t in [int(draft[b, j]) for j in range(n)] + [int(next_tokens[b])]:
            if 0 <= t < V:
                word = int(out[row, t])
                c = min((word & COUNT_MAX) + 1, COUNT_MAX)
                out[row, t] = c - 32768 if word < 0 else c
    return out


def process_row(x, word=None, drafts=(), repetition=1.0, frequency=0.0, presence=0.0, biases=(), mask=None,
                temperature=1.0):
    """One row: logits x [V], its request's table words [V], the drafts it follows, (token, value) biases, and
    its mask words.  Returns (processed [V], argmax, probs [V]) in float64."""
    x = np.array(x, dtype=np.float64)
    V = len(x)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for t in range(V):
            w = 0 if word is None else int(word[t])
            n = (w & COUNT_MAX) + sum(1 for d in drafts if d == t)
            if w < 0 or n > 0:
                x[t] = x[t] / repetition if x[t] > 0 else x[t] * repetition
            if n > 0:
                x[t] = x[t] - frequency * n - presence
        for t, v in biases:
            if 0 <= t < V:
                x[t] += v
        if mask is not None:
            for t in range(V):
                if not (int(mask[t // 32]) >> (t % 32)) & 1:
                    x[t] = -math.inf
        nan = [t for t in range(V) if math.isnan(x[t])]
        if nan:
            p = np.full(V, math.nan)
            if not temperature > 0:
                p = np.zeros(V)
                p[nan[0]] = 1.0
            return x, nan[0], p
        top = max(x)
        if top == -math.inf:
            return x, -1, np.zeros(V)
        arg = min(t for t in range(V) if x[t] == top)
        if not temperature > 0:
            p = np.zeros(V)
            p[arg] = 1.0
            return x, arg, p
        d = np.where(x == top, 0.0, x - top)      # +inf entries share the mass
        e = np.exp(d / temperature)
        return x, arg, e / e.sum()
