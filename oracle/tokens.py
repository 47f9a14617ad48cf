"""The steps of a pass over several new tokens (oracle; test infrastructure only):
norms of queries and keys per head with the rotation by position, the slots that a
new token sees, and the verification of drafted tokens, in fp64 by plain loops.

"GGUF Inferencer in R", section 5.2: RMSN(v) = norm * v / sqrt(mean(v^2) + eps),
here over one head; section 5.2.1: attend (oracle.serving.attend_f64 over the slots
that visible_slots names). The rotation and the acceptance rule are on no page:
they are the definitions in include/gguf_tokens.h. PARITY UNPINNED.
"""

from __future__ import annotations

import math

import numpy as np


def rope_f64(x, pos, freqs, axes=None, halves=True, magnitude=1.0, norm=None, eps=0.0):
    """x [n_tokens, n_heads, dim]; pos [n_axes, n_tokens]; freqs [n_rot / 2]; axes per pair."""
    x = np.asarray(x, dtype=np.float64)
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(norm, dtype=np.float64)
    out = x.copy()
    half = 0 if freqs is None else len(freqs)
    for i in range(half):
        axis = 0 if axes is None else int(axes[i])
        a, b = (i, i + half) if halves else (2 * i, 2 * i + 1)
        for t in range(len(x)):
            angle = int(pos[axis][t]) * float(freqs[i]) if 0 <= axis < len(pos) else 0.0
            c, s = magnitude * math.cos(angle), magnitude * math.sin(angle)
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
    return out


def visible_slots(held, rows, j, window=0, sinks=0):
    """Slots that row j of the newest `rows` of `held` tokens sees, ascending."""
    p = held - rows + j
    i = np.arange(max(0, p + 1))
    if window:
        i = i[(i > p - window) | (i < sinks)]
    return i


def softmax_f64(x):
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.exp(x - x.max())
        return e / e.sum()


def verify_f64(target, draft, tokens, uniform, uniform_next, starts, temperature=None):
    """(accepted, next, accept_prob) over sequences of rows starts[s] .. starts[s + 1] - 1."""
    accepted, nxt, probs = [], [], np.full(len(target), np.nan)
    for s in range(len(starts) - 1):
        r0, r1 = int(starts[s]), int(starts[s + 1])
        t = 1.0 if temperature is None else float(temperature[s])
        done, drawn = 0, -1
        stopped = False
        for r in range(r0, r1):
            x = np.asarray(target[r], dtype=np.float64)
            last = r == r1 - 1
            token = -1 if last else int(tokens[r])
            known = 0 <= token < len(x)
            valid = np.isfinite(np.max(x))
            if not t > 0:
                best = int(np.argmax(x)) if valid else -1
                ok = not last and valid and best == token
                probs[r] = float((last and valid) or ok)
                draw = best
            else:
                p = softmax_f64(x / t) if valid else None
                q = None
                if not last and draft is not None:
                    y = np.asarray(draft[r], dtype=np.float64)
                    if not np.isfinite(np.max(y)):
                        valid = False
                    else:
                        q = softmax_f64(y / t)
                if last:
                    ok, probs[r], rest = False, float(valid), p
                else:
                    if draft is None:
                        q = np.zeros(len(x))
                        if known:
                            q[token] = 1.0
                    if not valid or not known:
                        ok, probs[r] = False, 0.0
                    else:
                        ok = float(uniform[r]) * q[token] < p[token]
                        probs[r] = 1.0 if p[token] >= q[token] > 0 else float(p[token] > 0) if q[token] == 0 else \
                            p[token] / q[token]
                    rest = None
                    if valid:
                        rest = np.maximum(p - q, 0.0)
                        if not rest.sum() > 0:
                            rest = p
                draw = -1
                if valid and not ok:
                    cdf = np.cumsum(rest)
                    draw = int(np.searchsorted(cdf, float(uniform_next[s]) * cdf[-1], side="right"))
                    draw = min(draw, int(np.nonzero(rest)[0][-1]))
            if not ok and not stopped:
                stopped, done, drawn = True, r - r0, draw
        accepted.append(done)
        nxt.append(drawn)
    return np.array(accepted), np.array(nxt), probs
