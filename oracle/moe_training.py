"""fp64 NumPy oracle of what stands around the experts' products in a training
step: the balance loss, the combine with dropout and the residual, and the
backward passes of both and of the router.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the
formulas with loops and dense Jacobians where those say it most plainly.
"""

from __future__ import annotations

import numpy as np

from .moe_oracle import _f64

__all__ = [
    "philox4x32_10",
    "dropout_keep",
    "dropout_threshold",
    "balance_loss",
    "router_dlogits",
    "route_backward",
    "combine_dropout",
    "combine_dropout_backward",
]

_M0, _M1 = 0xD2511F53, 0xCD9E8D57
_W0, _W1 = 0x9E3779B9, 0xBB67AE85
_LOW = 0xFFFFFFFF


def philox4x32_10(counter, key):
    """Ten rounds of Philox4x32 (Salmon et al., "Parallel random numbers: as
    easy as 1, 2, 3", 2011).  counter: four and key: two integer arrays (or
    ints) of 32-bit values; returns the four output words as uint64 arrays."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    low, s = np.uint64(_LOW), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(_M0), c[2] * np.uint64(_M1)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + _W0) & _LOW, (k[1] + _W1) & _LOW]
    return c


def dropout_threshold(p):
    """The drop probability in units of 2^-16."""
    return min(int(np.floor(float(p) * 65536.0 + 0.5)), 65535)


def dropout_keep(p, seed, offset, T, d, first=0):
    """Boolean [T, d]: which elements of tokens first .. first + T - 1 stay."""
    n = np.uint64(first * (d // 8)) + np.arange(T * (d // 8), dtype=np.uint64)
    words = philox4x32_10((n & np.uint64(_LOW), n >> np.uint64(32), np.uint64(offset & _LOW),
                           np.uint64(offset >> 32)), (seed & _LOW, seed >> 32))
    lanes = []
    for w in words:
        w = np.broadcast_to(w, n.shape)
        lanes += [w & np.uint64(0xFFFF), w >> np.uint64(16)]
    return (np.stack(lanes, 1) >= np.uint64(dropout_threshold(p))).reshape(T, d)


def balance_loss(scores, idx, E, coef, mask=None):
    """(loss, prob_sum [E], counts [E], tokens): coef E sum_e f_e P_e over the
    counted tokens; scores [E, T]."""
    scores, idx = _f64(scores), np.asarray(idx)
    T, k = idx.shape
    counted = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    n = int(counted.sum())
    picks = idx[counted].reshape(-1)
    counts = np.array([(picks == e).sum() for e in range(E)], dtype=np.int64)
    prob_sum = scores[:, counted].sum(1)
    loss = coef * E * float((counts / (n * k) * prob_sum / n).sum()) if n else 0.0
    return loss, prob_sum, counts, n


def router_dlogits(T, E, idx=None, gate=None, dgate=None, scores=None, counts=None, tokens=0,
                   coef=0.0, dloss=1.0, mask=None, gating="topk_softmax", gate_scale=1.0):
    """dz [T, E] by the Jacobians of the softmaxes, token by token."""
    dz = np.zeros((T, E))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        if dgate is not None:
            g, dg = _f64(gate[t]), _f64(dgate[t])
            k = g.size
            if gating == "topk_softmax":
                q = g / gate_scale
                jac = gate_scale * (np.diag(q) - np.outer(q, q))     # d gate_j / d z_{idx i}
                dsel = jac.T @ dg
                for j in range(k):
                    if 0 <= idx[t, j] < E:
                        dz[t, idx[t, j]] += dsel[j]
            else:
                p = _f64(scores[:, t])
                for j in range(k):
                    row = -g[j] * p                                   # d gate_j / d z
                    if 0 <= idx[t, j] < E:
                        row[idx[t, j]] += g[j]
                    dz[t] += dg[j] * row
        if counts is not None and tokens > 0:
            p = _f64(scores[:, t])
            k = idx.shape[1]
            up = dloss * coef * E / tokens * _f64(counts) / (tokens * k)  # d loss / d p_te
            dz[t] += p * (up - np.dot(up, p))
    return dz


def route_backward(x, Wg, dz, dx_acc=None, mask=None):
    """(dx, dWg, dbias) from dz; a padding token's x is not looked at."""
    x, Wg, dz = _f64(x), _f64(Wg), _f64(dz)
    if mask is not None:
        x = np.where(np.asarray(mask).astype(bool)[:, None], x, 0.0)
    dx = dz @ Wg.T
    if dx_acc is not None:
        dx = dx + _f64(dx_acc)
    return dx, x.T @ dz, dz.sum(0)


def _scale(p):
    return 65536.0 / (65536.0 - dropout_threshold(p))


def combine_dropout(o, pos, gate, keep=None, p=0.0, residual=None):
    """y [T, d]; keep [T, d] from dropout_keep (None: nothing is dropped)."""
    o, pos, gate = _f64(o), np.asarray(pos), _f64(gate)
    T, k = pos.shape
    y = np.zeros((T, o.shape[1]))
    with np.errstate(invalid="ignore"):
        for t in range(T):
            for j in range(k):
                if pos[t, j] >= 0:
                    y[t] += gate[t, j] * o[pos[t, j]]
        if keep is not None:
            y = np.where(keep, y * _scale(p), 0.0)
    return y if residual is None else y + _f64(residual)


def combine_dropout_backward(dy, o, pos, gate, keep=None, p=0.0):
    """(d_o [rows, d] with zeros where no kept slot points, dgate [T, k])."""
    dy, o, pos, gate = _f64(dy), _f64(o), np.asarray(pos), _f64(gate)
    T, k = pos.shape
    a = dy if keep is None else np.where(keep, dy * _scale(p), 0.0)
    d_o, dgate = np.zeros_like(o), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = pos[t, j]
            if r < 0:
                continue
            d_o[r] = gate[t, j] * a[t]
            stay = slice(None) if keep is None else keep[t]
            dgate[t, j] = np.dot(a[t][stay], o[r][stay])
    return d_o, dgate
