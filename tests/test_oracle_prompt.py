"""Pins of the 64-bit restatements around a prompt: rotations are rotations and compose, the rules' limits, packed attention
against a dense softmax, the bookkeeping's invariants."""
import math

import numpy as np
import pytest
import torch

from oracle import prompt as O

RULES = [None, dict(kind="linear", factor=4.0), dict(kind="ntk", factor=4.0),
         dict(kind="llama3", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original=8192),
         dict(kind="yarn", factor=16.0, original=4096, beta_fast=32.0, beta_slow=1.0)]


@pytest.mark.parametrize("rule", RULES, ids=lambda r: "plain" if r is None else r["kind"])
def test_rules_keep_fast_pairs_and_slow_the_slow_ones(rule):
    f, factor = O.frequencies(128, 5e5, rule)
    plain = 5e5 ** (-np.arange(64) / 64)
    ratio = plain / f
    assert np.all(ratio >= 1 - 1e-12) and np.all(np.diff(f) < 0)
    if rule is None:
        assert np.allclose(ratio, 1)
        return
    assert ratio.max() <= rule["factor"] * (1 + 1e-12) and math.isclose(ratio[-1], rule["factor"], rel_tol=1e-9)
    if rule["kind"] in ("llama3", "yarn", "ntk"):
        assert math.isclose(ratio[0], 1.0)
    assert factor == (1.0 if rule["kind"] != "yarn" else 0.1 * math.log(16) + 1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations_compose_and_keep_lengths(interleaved):
    g = np.random.default_rng(0)
    x, f = g.normal(size=(9, 3, 48)), O.frequencies(32, 1e4)[0]
    p1, p2 = g.integers(0, 1000, 9), g.integers(0, 1000, 9)
    a = O.rotate(O.rotate(x, p1, f, 1.0, interleaved)[0], p2, f, 1.0, interleaved)[0]
    assert np.allclose(a, O.rotate(x, p1 + p2, f, 1.0, interleaved)[0], atol=1e-11)
    assert np.allclose(O.rotate(a, p1 + p2, f, 1.0, interleaved, inverse=True)[0], x, atol=1e-11)
    assert np.array_equal(a[..., 32:], x[..., 32:])
    # scores depend on the difference of positions alone
    y = g.normal(size=x.shape)
    s = [np.sum(O.rotate(x, p, f, 1.0, interleaved)[0] * O.rotate(y, p + 7, f, 1.0, interleaved)[0]) for p in (p1, p2)]
    assert math.isclose(s[0], s[1], rel_tol=1e-9)
    # as complex numbers
    z = x[..., 0:32:2] + 1j * x[..., 1:32:2] if interleaved else x[..., :16] + 1j * x[..., 16:32]
    z = z * np.exp(1j * p1[:, None, None] * f)
    r = O.rotate(x, p1, f, 1.0, interleaved)[0]
    got = r[..., 0:32:2] + 1j * r[..., 1:32:2] if interleaved else r[..., :16] + 1j * r[..., 16:32]
    assert np.allclose(z, got, atol=1e-12)


def test_packed_attention_against_dense_softmax():
    g = np.random.default_rng(1)
    lens, keys, nq, nkv, d = [3, 0, 5, 2], [3, 4, 9, 1], 4, 2, 8
    start, kstart = np.cumsum([0] + lens), np.cumsum([0] + keys)
    q, k, v = g.normal(size=(12, nq, d)), g.normal(size=(17, nkv, d)), g.normal(size=(17, nkv, d))
    out, lse, _, _ = O.attend_packed(q, k, v, start, kstart, 0.3)
    assert np.isnan(out[10:]).all() and not out[8].any() and lse[8, 0] == -np.inf
    for b, (n, m) in enumerate(zip(lens, keys)):
        if n == 0:
            continue
        Q, K, V = (torch.from_numpy(t[s[b]:s[b + 1]]) for t, s in ((q, start), (k, kstart), (v, kstart)))
        K, V = K.repeat_interleave(2, 1), V.repeat_interleave(2, 1)
        s = torch.einsum("ihd,jhd->hij", Q, K) * 0.3
        s = s.masked_fill(~torch.ones(n, m, dtype=torch.bool).tril(m - n), -np.inf)
        want = torch.einsum("hij,jhd->ihd", torch.nan_to_num(torch.softmax(s, -1)), V)
        assert np.allclose(out[start[b]:start[b + 1]], want.numpy(), atol=1e-13)
        assert np.allclose(lse[start[b]:start[b + 1]].T, torch.logsumexp(s, -1).numpy(), atol=1e-13)


def test_bookkeeping_invariants():
    g = np.random.default_rng(2)
    B, W, n, block = 7, 6, 30, 16
    table, refs = [[-1] * W for _ in range(B)], [0] * n
    for step in range(300):
        length = [int(x) for x in g.integers(-1, W * block // 2, B)]
        parent = None
        if step % 3 == 2:
            have = [sum(e >= 0 for e in t) * block for t in table]
            p = int(np.argmax(have))
            parent = [p if b != p and g.random() < 0.5 and have[p] else -1 for b in range(B)]
            length = [-1 if b == p or parent[b] < 0 else min(max(0, x), have[p]) for b, x in enumerate(length)]
        _, short = O.resize(table, refs, length, block, parent)
        flat = [e for t in table for e in t if e >= 0]
        assert [flat.count(i) for i in range(n)] == refs
        if not short:
            for b, x in enumerate(length):
                if x >= 0:
                    assert all((e >= 0) == (j * block < x) for j, e in enumerate(table[b]))
                    if x % block:      # what it writes next, nobody else sees
                        assert refs[table[b][x // block]] == 1
