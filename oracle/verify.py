"""Verification of drafted tokens by the target's probabilities, step by step.

TEST INFRASTRUCTURE ONLY, like oracle.sample, whose masses it uses.

Speculative sampling (Leviathan et al. 2023, algorithm 1; Chen et al. 2023): a
draft x drawn from d is kept with probability min(1, p(x) / d(x)); at the first
one that is not, the token is drawn from max(0, p - d), renormalised.  p and d
are nucleus distributions held as integers (oracle.sample, steps 1 to 3), and
the random numbers are inputs.  The largest doubt that a last-bit difference of
the fp64 exponential can make is reported, so that tests can leave such a block
out: every comparison's distance from its border, relative, and the draw's
distance from the ends of its interval, in units.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from .sample import MASS_SCALE, draw_point, greedy, masses, nucleus_need


def nucleus_masses(logits: np.ndarray, temperature: float, top_p: float) -> np.ndarray:
    """int64 masses of one row's nucleus by token id, zero outside it."""
    l = np.asarray(logits, np.float32)
    q = masses(l, temperature).astype(np.int64)
    need = nucleus_need(int(q.sum()), top_p)
    order = np.argsort(-l.astype(np.float64), kind="stable")
    cum = np.cumsum(q[order])
    k = int(np.searchsorted(cum, need, side="left")) + 1
    a = np.zeros_like(q)
    a[order[:k]] = q[order[:k]]
    return a


@dataclass
class Block:
    tokens: list         # accepted drafts, the drawn token, -1 behind it
    accepted: int
    accept_margin: float  # smallest relative distance of an acceptance from its border
    draw_margin: int      # distance of the draw's point from the ends of its interval


def verify_block(logits, draft_logits, tokens, temperature, top_p, uniforms) -> Block:
    """One block: logits [T, V], draft_logits [T - 1, V] or None, tokens [T]."""
    T, V = logits.shape
    margin, draw = float("inf"), 1 << 80
    greedy_row = not float(np.float32(temperature)) > 0
    out = []
    for s in range(T):
        x = int(tokens[s + 1]) if s + 1 < T else -1
        real = 0 <= x < V
        if greedy_row:
            best = greedy(logits[s])
            out.append(best)
            if x != best:
                break
            continue
        a = nucleus_masses(logits[s], temperature, top_p)
        A = int(a.sum())
        rest = a
        if real:
            if draft_logits is None:
                lhs, rhs = float(uniforms[s]) * float(A), float(a[x])
                rest = a.copy()
                rest[x] = 0
            else:
                d = nucleus_masses(draft_logits[s], temperature, top_p)
                D = int(d.sum())
                lhs, rhs = float(uniforms[s]) * (float(d[x]) * float(A)), float(a[x]) * float(D)
                share = np.rint(a.astype(np.float64) * (MASS_SCALE / float(A))).astype(np.int64)
                other = np.rint(d.astype(np.float64) * (MASS_SCALE / float(D))).astype(np.int64)
                rest = np.maximum(0, share - other)
            if max(lhs, rhs) > 0:
                margin = min(margin, abs(lhs - rhs) / max(lhs, rhs))
            if lhs < rhs:
                out.append(x)
                continue
            if rest.sum() == 0:
                rest = a
        R = int(rest.sum())
        y = draw_point(R, float(uniforms[T - 1]))
        cum = np.cumsum(rest)
        token = int(np.searchsorted(cum, y, side="right"))
        before = int(cum[token - 1]) if token else 0
        draw = min(y - before, int(cum[token]) - 1 - y)
        out.append(token)
        break
    return Block(out + [-1] * (T - len(out)), len(out), margin, draw)
