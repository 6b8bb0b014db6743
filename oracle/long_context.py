"""The operators for long contexts, restated plainly in float64 (test
infrastructure): attention over a shared prefix and own tokens, the attention
weight of each key, and the rule of eviction.  Keys are rows of 576 values, the
first 512 of which are the values."""
from __future__ import annotations

import numpy as np


def visible(n: int, T: int, t: int, causal: bool) -> int:
    """Own keys that query token t of T sees."""
    return min(max(n - T + t + 1, 0), n) if causal else n


def attention(q: np.ndarray, prefix: np.ndarray, own: np.ndarray, scale: float, causal: bool):
    """One sequence: q [T, H, 576], prefix [P, 576], own [n, 576] -> dict of out
    [T, H, 512], lse [T, H], spread (sum of weights times |value|), top (largest
    |score| of a row) and mag (largest scale * sum |q k| of a row)."""
    T, H, _ = q.shape
    out, spread = np.zeros((T, H, 512)), np.zeros((T, H, 512))
    lse, top, mag = np.full((T, H), -np.inf), np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        k = np.concatenate([prefix, own[:visible(len(own), T, t, causal)]])
        if not len(k):
            continue
        s = scale * (q[t] @ k.T)
        m = s.max(1, keepdims=True)
        w = np.exp(s - m)
        z = w.sum(1, keepdims=True)
        lse[t] = (m + np.log(z))[:, 0]
        w /= z
        out[t], spread[t] = w @ k[:, :512], w @ np.abs(k[:, :512])
        top[t], mag[t] = np.abs(s).max(1), scale * (np.abs(q[t]) @ np.abs(k).T).max(1)
    return dict(out=out, lse=lse, spread=spread, top=top, mag=mag)


def mass(q: np.ndarray, own: np.ndarray, lse: np.ndarray, scale: float, causal: bool):
    """One sequence: q [T, H, 576], own [n, 576], lse [T, H] -> (weights summed
    over rows [n], the sum of weights times what bounds the error of their
    exponent [n]: 576 products of one step each, and the roundings of score,
    log-sum-exp and their difference)."""
    T, H, _ = q.shape
    n = len(own)
    total, bound = np.zeros(n), np.zeros(n)
    for t in range(T):
        sees = visible(n, T, t, causal)
        live = ~np.isneginf(lse[t])
        k = own[:sees]
        s = scale * (k @ q[t].T)
        with np.errstate(invalid="ignore"):
            w = np.where(live, np.exp(s - lse[t]), 0.0)
        mag = scale * (np.abs(k) @ np.abs(q[t]).T)
        step = 2.0 ** -23
        d = 576 * step * mag + 3 * step * (np.abs(s) + np.abs(np.where(live, lse[t], 0.0))) + 2.0 ** -21
        total[:sees] += w.sum(1)
        bound[:sees] += (w * np.expm1(d)).sum(1)
    return total, bound


def evict(mass: np.ndarray, positions: np.ndarray, n: int, keep: int, sinks: int, recent: int):
    """One sequence -> (slots that are filled, slots they are filled from), both
    ascending: the rule token by token."""
    if n <= keep:
        return [], []
    newest = int(positions[:n].max())

    def rank(i):
        forced = positions[i] < sinks or int(positions[i]) > newest - recent
        m = float(mass[i])
        return (not forced, 0.0 if forced else (np.inf if np.isnan(m) else -m), bool(np.isnan(m)) and not forced, i)

    stays = set(sorted(range(n), key=rank)[:keep])
    return [i for i in range(keep) if i not in stays], [i for i in range(keep, n) if i in stays]
