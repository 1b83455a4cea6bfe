"""64-bit restatement of rotary positions, of attention over packed prompts, and of a paged cache's bookkeeping.

Plain loops over rows, pairs, sequences and blocks, from the definitions that the C header gives.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot: int, theta: float, rule=None):
    """(angles per position [rot / 2], factor) of a rule: None or a dict as api.Rope's `scaling`."""
    out, factor = np.empty(rot // 2), 1.0
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        kind = None if rule is None else rule["kind"]
        if kind == "linear":
            f /= rule["factor"]
        elif kind == "ntk":
            f = (theta * rule["factor"] ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif kind == "llama3":
            wave = 2 * math.pi / f
            longest, shortest = rule["original"] / rule["low_freq_factor"], rule["original"] / rule["high_freq_factor"]
            if wave > longest:
                f /= rule["factor"]
            elif wave >= shortest:
                mix = (rule["original"] / wave - rule["low_freq_factor"]) / (rule["high_freq_factor"] - rule["low_freq_factor"])
                f = (1 - mix) * f / rule["factor"] + mix * f
        elif kind == "yarn":
            pair = lambda turns: rot * math.log(rule["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
            lo = max(math.floor(pair(rule.get("beta_fast", 32.0))), 0)
            hi = min(math.ceil(pair(rule.get("beta_slow", 1.0))), rot - 1)
            slow = 0.0 if i <= lo else (1.0 if i >= hi else (i - lo) / (hi - lo))
            f = f * (1 - slow) + f / rule["factor"] * slow
            factor = rule.get("attention") or 0.1 * math.log(rule["factor"]) + 1
        out[i] = f
    return out, factor


def rotate(x: np.ndarray, pos: np.ndarray, freq: np.ndarray, factor: float, interleaved: bool, inverse: bool = False):
    """x [R, heads, d] turned to positions pos [R]; returns (values, slack): slack [R, heads, d] bounds |a| + |b| of the pair
    that an entry comes from (0 where it is copied)."""
    y, slack = x.astype(np.float64).copy(), np.zeros(x.shape)
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freq))
        angle = pos.astype(np.float64) * (-f if inverse else f)
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        y[:, :, a] = factor * (x[:, :, a] * c - x[:, :, b] * s)
        y[:, :, b] = factor * (x[:, :, b] * c + x[:, :, a] * s)
        slack[:, :, a] = slack[:, :, b] = abs(factor) * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
    return y, slack


def attend_packed(q, k, v, start, kstart, scale):
    """(out [R, nq, d], lse [R, nq], weight, reach): rows of no sequence are NaN. weight = sum p |v| / sum p of each row,
    reach [R, nq] = the largest sum |q_i k_i| scale of a key that it sees. Hidden keys take no part."""
    R, nq, d = q.shape
    nkv = k.shape[1]
    out, weight = np.full((R, nq, d), np.nan), np.full((R, nq, d), np.nan)
    lse, reach = np.full((R, nq), np.nan), np.full((R, nq), np.nan)
    for b in range(len(start) - 1):
        n, m = start[b + 1] - start[b], kstart[b + 1] - kstart[b]
        for i in range(n):
            row, sees = start[b] + i, m - n + i + 1
            for h in range(nq):
                if sees <= 0:
                    out[row, h], weight[row, h], lse[row, h], reach[row, h] = 0, 0, -np.inf, 0
                    continue
                K, V = (t[kstart[b]:kstart[b] + sees, h * nkv // nq] for t in (k, v))
                with np.errstate(invalid="ignore", over="ignore"):
                    s = K @ q[row, h] * scale
                    top = s.max()
                    p = np.exp(s - top)
                    out[row, h], weight[row, h] = p @ V / p.sum(), p @ np.abs(V) / p.sum()
                    lse[row, h] = top + np.log(p.sum())
                    reach[row, h] = (np.abs(K) @ np.abs(q[row, h])).max() * scale
    return out, lse, weight, reach


def resize(table, refs, length, block, parent=None):
    """The bookkeeping of one call, in place on lists: (copies, short): [(from, to, slots)], whether blocks ran out. Sequences
    of a call are expected to be valid."""
    B = len(length)
    forks = [b for b in range(B) if parent is not None and parent[b] >= 0 and length[b] >= 0]
    wants = [-(-n // block) if n >= 0 else -1 for n in length]
    for b in range(B):
        for j in range(len(table[b])):
            if wants[b] >= 0 and table[b][j] >= 0 and (b in forks or j >= wants[b]):
                refs[table[b][j]] -= 1
                table[b][j] = -1
    for b in forks:
        for j in range(wants[b]):
            table[b][j] = table[parent[b]][j]
            refs[table[b][j]] += 1
    held = list(refs)
    free = [i for i, n in enumerate(refs) if n == 0]
    copies, short = [], False
    for b in range(B):
        for j in range(max(0, wants[b])):
            missing = table[b][j] < 0
            other = not missing and j == wants[b] - 1 and length[b] % block != 0 and held[table[b][j]] > 1
            if not missing and not other:
                continue
            if not free:
                short = True
                continue
            new = free.pop(0)
            if other:
                copies.append((table[b][j], new, length[b] % block))
                refs[table[b][j]] -= 1
            table[b][j], refs[new] = new, 1
    return copies, short
