"""Rotary positions and packed prompt attention on the GPU against 64 bits.

Tolerances, fixed before any run. Rotary positions: a turned entry is m (a c - b s). The angle's fraction of a turn is off by
its rounding to fp32 (2^-24 of at most half a turn: pi 2^-24) and by the doubles that it comes from, on both sides (p f 2^-51
radians); sincospi is good to 2 units in the last place (2^-22); the factor, two products and a sum lose 2^-24 each of at most m (|a| +
|b|). So m (|a| + |b|) (pi 2^-24 + p f 2^-51 + 2^-22 + 4 2^-24), and the output's rounding: half a step of its type.
Attention: with W = sum p |v| / sum p and A the largest sum_i |q_i k_i| * scale that the row sees, both in 64 bits:
  2^-8 |o|                    the output's rounding to bf16;
  W * 2^-8                    each weight's rounding to bf16;
  W * 2 * (d + 8) * 2^-23 * A the score: d fp32 additions that may each lose a step of the partial sum, and the products
                              around them; an error x of a score moves a weight by x relative, its own and, through the sum,
                              everybody's;
  W * (n + 64) * 2^-23        n fp32 additions of the value product and of the sum, exp2 and the rescaling.
lse: (d + 8) 2^-23 A for the scores, (n + 64) 2^-23 for the sum, and four roundings of a number of its size, 2^-22 |lse|."""
import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from eagle_speculative_decoding_cycle_gb300 import _lib as L, api
from oracle import prompt as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

RULES = {"plain": None, "linear": dict(kind="linear", factor=4.0), "ntk": dict(kind="ntk", factor=4.0),
         "llama3": dict(kind="llama3", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original=8192),
         "yarn": dict(kind="yarn", factor=16.0, original=4096, beta_fast=32.0, beta_slow=1.0),
         "yarn-own": dict(kind="yarn", factor=4.0, original=2048, attention=1.25)}


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).to(DEV)


def host(t):
    return t.detach().double().cpu().numpy()


# ---- rotary positions -----------------------------------------------------------------------------
def check_rope(plan, rule, theta, x, got, pos, interleaved, inverse=False):
    freq, factor = O.frequencies(plan.rot, theta, rule)
    want, slack = O.rotate(host(x), pos, freq, factor, interleaved, inverse)
    far = np.zeros(x.shape[2])
    for i, f in enumerate(freq):
        for e in ((2 * i, 2 * i + 1) if interleaved else (i, i + len(freq))):
            far[e] = f
    off = slack * (math.pi * 2.0 ** -24 + np.abs(pos.astype(float))[:, None, None] * far * 2.0 ** -51 + 2.0 ** -22 + 2.0 ** -22)
    tol = off + torch.finfo(got.dtype).eps / 2 * (np.abs(want) + off)
    tol[..., plan.rot:] = torch.finfo(got.dtype).eps / 2 * np.abs(want[..., plan.rot:]) if got.dtype != x.dtype else 0
    bad = ~(np.abs(host(got) - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("R,nq,nkv,d,rot,interleaved", [(1, 1, 1, 64, 64, False), (7, 5, 5, 128, 128, True),
                                                        (61, 10, 5, 64, 32, True), (333, 28, 4, 128, 64, False),
                                                        (129, 3, 0, 80, 48, False), (5, 64, 8, 256, 256, True),
                                                        (1000, 2, 1, 16, 16, False), (17, 7, 3, 96, 96, False)])
def test_rope_matches_64_bits(rule, R, nq, nkv, d, rot, interleaved):
    g = torch.Generator().manual_seed(R + d)
    plan = api.Rope(d, theta=5e5, rot=rot, interleaved=interleaved, scaling=RULES[rule], device=DEV)
    pos = torch.randint(0, 200000, (R,), generator=g).numpy()
    pos[: min(R, 3)] = [0, 131071, 1][: min(R, 3)]
    for src, dst in ((torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                     (torch.bfloat16, torch.float32)):
        fused = torch.randn(R, nq + 2 * max(nkv, 1), d, generator=g).to(src).to(DEV)
        q, k = fused[:, :nq], fused[:, nq:nq + nkv] if nkv else None
        before = fused.clone()
        qo, ko = api.rope(plan, q, k, i32(pos), dtype=dst)
        assert qo.dtype == dst and torch.equal(fused, before)
        check_rope(plan, RULES[rule], 5e5, q, qo, pos, interleaved)
        if nkv:
            check_rope(plan, RULES[rule], 5e5, k, ko, pos, interleaved)
        if src == dst:      # in place, between columns that stay
            api.rope(plan, q, k, i32(pos), out=(q, k))
            assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))
            assert torch.equal(fused[:, nq + nkv:], before[:, nq + nkv:])


def test_rope_back_far_and_negative_positions():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(64, 4, 128, generator=g).to(DEV)
    pos = torch.randint(-2 ** 31, 2 ** 31, (64,), generator=g).numpy()
    pos[:4] = [2 ** 31 - 1, -2 ** 31, -1, 2 ** 30]
    plan = api.Rope(128, device=DEV)
    y, _ = api.rope(plan, x, None, i32(pos))
    check_rope(plan, None, 1e4, x, y, pos, False)
    z, _ = api.rope(plan, y, None, i32(pos), inverse=True)
    check_rope(plan, None, 1e4, y, z, pos, False, inverse=True)
    assert float((z - x).abs().max()) < 2.0 ** -18      # two turns: each off by at most some 2^-20 of entries below 8


@pytest.mark.parametrize("rule,d,rot,interleaved", [("plain", 128, 128, False), ("yarn", 64, 32, True), ("yarn-own", 96, 48, False)])
def test_rope_back_is_the_gradient(rule, d, rot, interleaved):
    """Of sum(w * rope(x)) with respect to x: against the formula in 64 bits, and against differences along some directions (the
    map is linear: any step will do). An entry is off by at most 2^-20 m (|a| + |b|), by the arithmetic above for these
    positions; a sum of products by the products' own sums of that."""
    g = torch.Generator().manual_seed(d)
    plan = api.Rope(d, rot=rot, interleaved=interleaved, scaling=RULES[rule], device=DEV)
    pos = torch.randint(0, 100000, (50,), generator=g).numpy()
    x, w = (torch.randn(50, 3, d, generator=g).to(DEV) for _ in range(2))
    grad, _ = api.rope(plan, w, None, i32(pos), inverse=True)
    check_rope(plan, RULES[rule], 1e4, w, grad, pos, interleaved, inverse=True)
    slack = lambda t: O.rotate(host(t), pos, np.asarray(plan.freq), plan.factor, interleaved)[1]  # noqa: E731
    for _ in range(4):
        e = torch.randn(50, 3, d, generator=g).to(DEV)
        up, down = x + e, x - e
        step = host(up) - host(down)
        rise = (host(w) * (host(api.rope(plan, up, None, i32(pos))[0]) - host(api.rope(plan, down, None, i32(pos))[0]))).sum()
        off = 2.0 ** -20 * ((np.abs(host(w)) * (slack(up) + slack(down))).sum() + (np.abs(step) * slack(w)).sum())
        assert abs(rise - (host(grad) * step).sum()) <= off


def test_rope_own_frequencies_and_strides():
    g = torch.Generator().manual_seed(2)
    freq = [0.5, -1.25, 7.0, 0.0, 1e-9, 3.0, math.pi, 0.1]
    plan = api.Rope(32, rot=16, freq=freq, factor=0.5, device=DEV)
    x = torch.randn(40, 6, 32, generator=g).to(torch.bfloat16).to(DEV)
    wide = torch.full((40, 9, 32), 3.0, dtype=torch.float32, device=DEV)
    pos = np.arange(40)
    q, k = api.rope(plan, x[:, :4], x[:, 4:], i32(pos), out=(wide[:, 1:5], wide[:, 6:8]))
    want, slack = O.rotate(host(x), pos, np.asarray(freq), 0.5, False)
    off = slack * 2.0 ** -20 + 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(np.concatenate([host(q), host(k)], 1) - want) <= off)
    assert torch.all(wide[:, [0, 5, 8]] == 3)
    e = api.rope(plan, x[:0], None, i32([]))[0]
    assert e.shape == (0, 6, 32)


def test_rope_in_a_graph_and_on_a_side_stream():
    plan = api.Rope(128, scaling=RULES["llama3"], device=DEV)
    x, pos = torch.randn(64, 10, 128, device=DEV).to(torch.bfloat16), i32(np.arange(64))
    out = (torch.empty(64, 8, 128, dtype=torch.bfloat16, device=DEV), torch.empty(64, 2, 128, dtype=torch.bfloat16, device=DEV))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.rope(plan, x[:, :8], x[:, 8:], pos, out=out)
    for step in range(3):
        pos.add_(1)
        g.replay()
    torch.cuda.synchronize()
    want = api.rope(plan, x[:, :8], x[:, 8:], i32(np.arange(64) + 3))
    side = torch.cuda.Stream()
    got = api.rope(plan, x[:, :8], x[:, 8:], i32(np.arange(64) + 3), stream=side)
    torch.cuda.synchronize()
    for a, b, c in zip(out, want, got):
        assert torch.equal(a, b) and torch.equal(a, c)


# ---- packed prompts -------------------------------------------------------------------------------
class Packed:
    def __init__(self, lens, before, nq, nkv, d, seed=0, qscale=1.5, kspread=0.5, vspread=0.7, extra=3):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.keys = list(lens), [n + b for n, b in zip(lens, before)]
        self.nq, self.nkv, self.d = nq, nkv, d
        self.R, self.K = sum(self.lens) + extra, sum(self.keys) + extra
        # q, k and v are columns of wider rows
        q = torch.randn(self.R, nq + 1, d, generator=g) * qscale
        k = torch.randn(self.K, 2 * nkv, d, generator=g) * torch.exp(kspread * torch.randn(2 * nkv, d, generator=g))
        v = torch.randn(self.K, nkv + 1, d, generator=g) * torch.exp(vspread * torch.randn(self.K, 1, 1, generator=g))
        self.q, self.k, self.v = (x.to(torch.bfloat16).to(DEV)[:, n:n + w] for x, n, w in
                                  ((q, 1, nq), (k, 0, nkv), (v, 1, nkv)))
        self.start, self.kstart = np.cumsum([0] + self.lens), np.cumsum([0] + self.keys)

    def run(self, scale=0.0, **kw):
        out = torch.full((self.R, self.nq + 1, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((self.R, self.nq), 7.0, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        api.attention_prompt(self.q, self.k, self.v, i32(self.start), i32(self.kstart), scale=scale, out=out[:, :self.nq],
                             lse=lse, err=err, **kw)
        assert int(err) == 0
        assert torch.all(out[:, self.nq] == 7)
        return out[:, :self.nq], lse

    def check(self, scale=0.0):
        out, lse = self.run(scale)
        want, wlse, W, A = O.attend_packed(host(self.q), host(self.k), host(self.v), self.start, self.kstart,
                                           scale if scale > 0 else self.d ** -0.5)
        rows = self.start[-1]
        assert torch.all(out[rows:] == 7) and torch.all(lse[rows:] == 7)      # rows of no sequence
        n = max([1] + self.keys)
        got, glse = host(out)[:rows], host(lse)[:rows]
        want, wlse, W, A = want[:rows], wlse[:rows], W[:rows], A[:rows]
        tol = 2.0 ** -8 * np.abs(want) + W * (2.0 ** -8 + 2 * (self.d + 8) * 2.0 ** -23 * A[..., None] + (n + 64) * 2.0 ** -23)
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])
        none = np.isinf(wlse)
        assert np.array_equal(none, np.isinf(glse)) and not got[none].any()
        ltol = (self.d + 8) * 2.0 ** -23 * A + (n + 64) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(none, 0, wlse))
        bad = ~(np.abs(np.where(none, 0, glse) - np.where(none, 0, wlse)) <= ltol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())
        return out, lse


@pytest.mark.parametrize("lens,before,nq,nkv,d", [
    ([1], [0], 1, 1, 64), ([1], [0], 32, 8, 128), ([2], [0], 4, 1, 128),
    ([128], [0], 2, 2, 128), ([129], [0], 2, 2, 128), ([127], [0], 2, 1, 64),
    ([256], [0], 1, 1, 128), ([257], [0], 1, 1, 64), ([385], [0], 3, 3, 128),
    ([1, 17, 77], [0, 0, 0], 10, 5, 64),
    ([5, 0, 64, 1, 0, 33], [0, 0, 0, 0, 3, 9], 8, 2, 128),
    ([40, 70], [100, 0], 28, 4, 128),            # seven heads: 18 positions a tile, two vectors idle
    ([31, 200], [0, 128], 6, 1, 64), ([50], [13], 64, 8, 64), ([9, 3], [0, 250], 64, 1, 128),
    ([1, 1, 1, 1], [0, 127, 128, 300], 8, 8, 128),      # single rows behind keys: a decoding step
    ([100], [-30], 4, 2, 128), ([20, 300], [-20, -290], 4, 4, 64),      # more rows than keys
    ([64], [64], 4, 2, 128), ([512], [0], 4, 1, 64), ([300], [5], 5, 1, 64)])
def test_prompt_matches_64_bits(lens, before, nq, nkv, d):
    Packed(lens, before, nq, nkv, d, seed=sum(lens) + nq).check()


@pytest.mark.parametrize("n,before,nq,nkv,d", [(1500, 0, 2, 1, 128), (700, 1300, 4, 4, 64), (33, 3000, 8, 2, 128)])
def test_long_prompts(n, before, nq, nkv, d):
    Packed([n, 7], [before, 0], nq, nkv, d, seed=3).check()


@pytest.mark.parametrize("qscale,kspread,vspread", [(40.0, 0.5, 0.7), (0.01, 0.1, 3.0), (6.0, 1.5, 0.1)])
def test_wide_value_ranges(qscale, kspread, vspread):
    Packed([200, 41], [0, 100], 4, 2, 128, seed=4, qscale=qscale, kspread=kspread, vspread=vspread).check()


def test_scale_argument():
    Packed([150], [0], 2, 1, 64, seed=5).check(scale=0.7)
    p = Packed([150], [0], 2, 1, 64, seed=5)
    assert torch.equal(p.run(0.125)[0], p.run(0.0)[0])


def test_rising_scores_rescale():
    """Scores that rise by more than the lazy bound from tile to tile: each tile's maximum replaces the reference."""
    p = Packed([1024], [0], 2, 1, 128, seed=6, extra=0)
    ramp = torch.linspace(0.2, 12, 1024, device=DEV).to(torch.bfloat16)
    p.q.copy_(p.q.abs())
    p.k.copy_(p.k.abs() * ramp[:, None, None])
    p.check()
    p.k.copy_(p.k.flip(0))
    p.check()


@pytest.mark.parametrize("nq,nkv,d", [(4, 4, 128), (8, 2, 64), (7, 1, 128)])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
def test_hidden_keys_and_values_may_be_anything(nq, nkv, d, fill):
    """What a row does not see, of its own sequence, of others and behind all of them, leaves its bits alone."""
    p = Packed([150, 70, 300], [0, 20, 0], nq, nkv, d, seed=7)
    want, wlse = p.run()
    for at in (0, 3, 100, 149, 150, 170, 239, 240, 400, 539, 541):      # a key row of some sequence, or of none
        k, v = p.k[at].clone(), p.v[at].clone()
        p.v[at, :, ::3] = fill
        p.k[at, :, 5] = fill
        out, lse = p.run()
        p.k[at], p.v[at] = k, v
        sees = torch.zeros(p.R, dtype=torch.bool, device=DEV)
        for b in range(3):
            if p.kstart[b] <= at < p.kstart[b + 1]:
                first = p.start[b + 1] - (p.kstart[b + 1] - at)
                sees[max(first, p.start[b]):p.start[b + 1]] = True
        assert torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], wlse[~sees])
        if sees.any() and math.isnan(fill):
            assert torch.isnan(out[sees]).all()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_reach_who_sees_them(fill):
    """A value column with one such entry: rows that see it get it (an infinite weight's share of it), other columns stay."""
    for lens, nq, nkv, d, at in (([200], 2, 1, 128, 150), ([64], 8, 2, 64, 0), ([130, 300], 1, 1, 64, 400), ([300], 4, 4, 128, 10),
                                 ([40], 7, 1, 128, 39)):
        p = Packed(lens, [0] * len(lens), nq, nkv, d, seed=8)
        want, _ = p.run()
        p.v[at, 0, 17] = fill
        out, _ = p.run()
        b = 0 if at < p.start[1] else 1
        hit = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
        hit[at:p.start[b + 1], :nq // nkv, 17] = True
        assert torch.equal(out[~hit], want[~hit])
        got = out[hit].float()
        ok = torch.isnan(got) if math.isnan(fill) else (got == fill) | torch.isnan(got)   # (a weight may round to zero)
        assert ok.all()
        # in the tile that holds the diagonal every weight counts: exactly the value
        near = out[at:min(at + 3, int(p.start[b + 1])), :nq // nkv, 17].float()
        assert (torch.isnan(near) if math.isnan(fill) else near == fill).all()


def test_both_infinities_in_one_column():
    p = Packed([100], [0], 2, 1, 128, seed=9)
    want, _ = p.run()
    p.v[20, 0, 3], p.v[50, 0, 3] = float("inf"), -float("inf")
    out = p.run()[0].float()
    assert torch.equal(out[:20].bfloat16(), want[:20])
    assert (out[20:50, :, 3] == float("inf")).all() and torch.isnan(out[50:100, :, 3]).all()
    out[:, :, 3] = want[:, :, 3].float()
    assert torch.equal(out.bfloat16(), want)


def test_results_do_not_depend_on_the_batch():
    """A sequence alone and among others, first and last: the same bits (without scratch, so keys are not shared out)."""
    lens, before = [70, 300, 5, 129], [10, 0, 200, 0]
    p = Packed(lens, before, 8, 2, 128, seed=10)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    out, lse = p.run(scratch=none)
    for b in range(4):
        r, c = slice(p.start[b], p.start[b + 1]), slice(p.kstart[b], p.kstart[b + 1])
        s = torch.empty(lens[b], 8, device=DEV)
        o = api.attention_prompt(p.q[r], p.k[c], p.v[c], i32([0, lens[b]]), i32([0, lens[b] + before[b]]), lse=s, scratch=none)
        assert torch.equal(o, out[r]) and torch.equal(s, lse[r])
    for _ in range(3):
        o2, l2 = p.run(scratch=none)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_chunks_of_a_prompt_agree_with_the_whole():
    """A prompt in chunks behind its earlier keys: the rows' results within the tolerance of both."""
    p = Packed([500], [0], 4, 2, 128, seed=11, extra=0)
    whole, _ = p.check()
    for a, b in ((0, 100), (100, 101), (101, 400), (400, 500)):
        o = api.attention_prompt(p.q[a:b], p.k[:b], p.v[:b], i32([0, b - a]), i32([0, b]))
        W = O.attend_packed(host(p.q), host(p.k), host(p.v), p.start, p.kstart, 128 ** -0.5)[2][a:b]
        assert np.all(np.abs(host(o) - host(whole[a:b])) <= 2.0 ** -7 * np.abs(host(o)) + 2.0 ** -6 * W)


def test_joined_by_lse():
    """Results over two ranges of keys joined by their log-sum-exps: those over all keys."""
    p = Packed([60], [140], 4, 2, 64, seed=12, extra=0)
    want, wlse = p.run()
    l1, l2 = torch.empty(60, 4, device=DEV), torch.empty(60, 4, device=DEV)
    # the 140 keys before: seen by every row, one sequence a row
    ks = torch.cat([p.k[:140]] * 60), torch.cat([p.v[:140]] * 60)
    o1 = api.attention_prompt(p.q, *ks, i32(np.arange(61)), i32(140 * np.arange(61)), lse=l1)
    o2 = api.attention_prompt(p.q, p.k[140:], p.v[140:], i32([0, 60]), lse=l2)
    l = torch.logaddexp(l1.double(), l2.double())
    o = o1.double() * torch.exp(l1 - l)[..., None] + o2.double() * torch.exp(l2 - l)[..., None]
    assert float((l - wlse.double()).abs().max()) < 1e-4
    assert float((o - want.double()).abs().max()) <= 2.0 ** -5 * float(p.v.abs().max())


@pytest.mark.parametrize("lens,before,nq,nkv,d", [
    ([1], [2000], 4, 1, 128), ([5, 1], [2800, 900], 28, 4, 128), ([300], [2200], 2, 2, 64), ([40, 2], [1500, 1700], 8, 2, 128),
    ([1, 1], [4000, 0], 1, 1, 128), ([500], [2000], 4, 2, 128), ([0, 40, 0], [2500, 6500, 3], 64, 1, 64), ([3000], [0], 1, 1, 64),
    ([1900], [-300], 1, 1, 128), ([130], [1700], 5, 5, 128), ([1], [20000], 2, 1, 64)])
def test_few_rows_over_many_keys(lens, before, nq, nkv, d):
    """Items cut into ranges of keys and joined; the same calls without scratch within the tolerances of both."""
    p = Packed(lens, before, nq, nkv, d, seed=sum(lens) + nq)
    api_bytes = api.L.lib().eagle_op_attention_prompt_scratch_bytes(p.R, p.K, nq, nkv, d, len(lens))
    assert api_bytes > 0
    out, lse = p.check()
    again, _ = p.run(scratch=torch.full((max(api_bytes, 16),), 0xff, dtype=torch.uint8, device=DEV))
    assert torch.equal(out, again)
    rows = int(p.start[-1])
    whole, wlse = p.run(scratch=torch.empty(0, dtype=torch.uint8, device=DEV))
    assert float((whole[:rows].float() - out[:rows].float()).abs().max()) <= 2.0 ** -6 * float(p.v.abs().max())
    short, _ = p.run(scratch=torch.empty(max(1, api_bytes // 2) // 16 * 16 + 16, dtype=torch.uint8, device=DEV))
    assert torch.equal(short, whole)      # too little scratch: not split


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_hidden_values_between_the_pieces_of_an_item(fill):
    p = Packed([64, 3], [2500, 1500], 4, 2, 128, seed=17)
    assert api.L.lib().eagle_op_attention_prompt_scratch_bytes(p.R, p.K, 4, 2, 128, 2) > 0
    want, _ = p.run()
    for at in (0, 700, 2499, 2500, 2530, 2563, 2564, 3200, 4066, 4068):
        v = p.v[at].clone()
        p.v[at, :, 9] = fill
        out, _ = p.run()
        p.v[at] = v
        sees = torch.zeros(p.R, dtype=torch.bool, device=DEV)
        for b in range(2):
            if p.kstart[b] <= at < p.kstart[b + 1]:
                first = p.start[b + 1] - (p.kstart[b + 1] - at)
                sees[max(first, p.start[b]):p.start[b + 1]] = True
        assert torch.equal(out[~sees], want[~sees])
        rest = [c for c in range(128) if c != 9]
        assert torch.equal(out[:, :, rest], want[:, :, rest])
        if sees.any():
            got = out[sees][:, :, 9].float()
            assert (torch.isnan(got) | (got == fill)).all()


def test_many_short_sequences():
    g = np.random.default_rng(13)
    lens = g.integers(0, 4, 1500)
    before = g.integers(0, 3, 1500)
    Packed(lens.tolist(), before.tolist(), 4, 2, 64, seed=13).check()


def test_bad_starts_are_latched_and_skipped():
    p = Packed([30, 40, 20], [0, 0, 0], 4, 2, 128, seed=14, extra=0)
    want, _ = p.run()
    for qs, ks, fine in (([0, 95, 70, 90], [0, 30, 70, 90], [2]), ([0, 30, 70, 90], [0, 30, 29, 90], [0]), ([0, 30, 70, 91], [0, 30, 70, 90], [0, 1]),
                         ([0, 30, 70, 90], [0, 30, 70, 2 ** 30], [0, 1]), ([-1, 30, 70, 90], [0, 30, 70, 90], [1, 2])):
        out = torch.full_like(want, 7.0)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        api.attention_prompt(p.q, p.k, p.v, i32(qs), i32(ks), out=out, err=err)
        assert int(err) == 2
        api.attention_prompt(p.q, p.k, p.v, i32(qs), i32(ks), out=torch.empty_like(want))      # without a status word
        for b in fine:
            if qs[b] == p.start[b] and qs[b + 1] == p.start[b + 1]:
                assert torch.equal(out[qs[b]:qs[b + 1]], want[qs[b]:qs[b + 1]])


def test_nothing_to_do():
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    assert api.attention_prompt(q, k, k, i32([0, 0])).shape == (0, 4, 64)
    assert api.attention_prompt(q, k, k, i32([0])).shape == (0, 4, 64)
    q = torch.ones(5, 4, 64, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(5, 4, device=DEV)
    out = api.attention_prompt(q, k, k, i32([0, 5]), i32([0, 0]), lse=lse)      # rows without any keys
    assert not out.any() and torch.all(lse == -float("inf"))


def test_graphs_with_other_lengths_and_streams():
    p = Packed([100, 60, 40], [0, 0, 0], 8, 2, 128, seed=15, extra=0)
    qs, ks = i32(p.start), i32(p.kstart)
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        o = torch.zeros(200, 8, 128, dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            api.attention_prompt(p.q, p.k, p.v, qs, ks, out=o)
        outs.append(o), graphs.append(g)
    for lens in ([100, 60, 40], [1, 198, 1], [0, 0, 200], [200, 0, 0]):
        s = i32(np.cumsum([0] + lens))
        qs.copy_(s), ks.copy_(s)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        want = api.attention_prompt(p.q, p.k, p.v, s)
        side = torch.cuda.Stream()
        got = api.attention_prompt(p.q, p.k, p.v, s, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and torch.equal(got, want)


def test_rows_past_four_gigabytes():
    """Row strides that carry offsets past 2^32 bytes, of inputs and results."""
    n, ld = 1100, 1 << 21
    base = torch.empty(n * ld, dtype=torch.bfloat16, device=DEV)
    view = lambda at, w: base.as_strided((n, w, 128), (ld, 128, 1), at)  # noqa: E731
    g = torch.Generator().manual_seed(16)
    q, k, v = (torch.randn(n, w, 128, generator=g).to(torch.bfloat16).to(DEV) for w in (4, 2, 2))
    want = api.attention_prompt(q, k, v, i32([0, 500, n]))
    for t, at in ((q, 0), (k, 4096), (v, 8192)):
        view(at, t.shape[1]).copy_(t)
    out = api.attention_prompt(view(0, 4), view(4096, 2), view(8192, 2), i32([0, 500, n]), out=view(65536, 4))
    assert torch.equal(out, want)
    plan = api.Rope(128, device=DEV)
    a, b = api.rope(plan, q, k, i32(np.arange(n)))
    api.rope(plan, view(0, 4), view(4096, 2), i32(np.arange(n)), out=(view(0, 4), view(4096, 2)))
    assert torch.equal(view(0, 4), a) and torch.equal(view(4096, 2), b)


def _agree_with_64_bits(p, lens, before, out, lse):
    nq, nkv, d = p.q.shape[1], p.k.shape[1], p.q.shape[2]
    for b in range(len(lens)):
        n, m = lens[b], lens[b] + before[b]
        if n == 0:
            continue
        r, c = slice(p.start[b], p.start[b + 1]), slice(p.kstart[b], p.kstart[b + 1])
        q = p.q[r].double().view(n, nkv, nq // nkv, d)
        s = torch.einsum("nhgd,mhd->hgnm", q, p.k[c].double()) * d ** -0.5
        reach = torch.einsum("nhgd,mhd->hgnm", q.abs(), p.k[c].double().abs()) * d ** -0.5
        hidden = torch.ones(n, m, dtype=torch.bool, device=DEV).triu_(m - n + 1)
        s, A = s.masked_fill(hidden, -math.inf), reach.masked_fill(hidden, 0).amax(-1)
        P, v = torch.softmax(s, -1), p.v[c].double()
        want, W = (torch.einsum("hgnm,mhd->nhgd", P, x).reshape(n, nq, d) for x in (v, v.abs()))
        A = A.permute(2, 0, 1).reshape(n, nq)
        tol = 2.0 ** -8 * want.abs() + W * (2.0 ** -8 + 2 * (d + 8) * 2.0 ** -23 * A[..., None] + (m + 64) * 2.0 ** -23)
        assert ((out[r].double() - want).abs() <= tol).all(), b
        wlse = torch.logsumexp(s, -1).permute(2, 0, 1).reshape(n, nq)
        assert ((lse[r].double() - wlse).abs() <= (d + 8) * 2.0 ** -23 * A + (m + 64) * 2.0 ** -23 + 2.0 ** -22 * wlse.abs()).all(), b


@pytest.mark.parametrize("nq,nkv,d,most", [(32, 8, 128, 300), (7, 7, 128, 700), (12, 12, 64, 500), (64, 4, 64, 90)])
def test_several_items_a_cta(nq, nkv, d, most):
    """More items than SMs, whole ones, with and without rows in their second tile: against 64 bits on the device."""
    g = np.random.default_rng(nq)
    lens = [int(x) for x in g.integers(0, most, 90)]
    before = [int(x) if i % 3 == 0 else 0 for i, x in enumerate(g.integers(0, 200, 90))]
    p = Packed(lens, before, nq, nkv, d, seed=18)
    out, lse = p.run()
    _agree_with_64_bits(p, lens, before, out, lse)
    again, _ = p.run()
    assert torch.equal(out, again)


@pytest.mark.parametrize("nq,nkv,d", [(8, 1, 128), (4, 2, 64)])
def test_lengths_far_apart(nq, nkv, d):
    """A few rows behind many keys among many short sequences and empty ones: most levels have no pairs."""
    g = np.random.default_rng(7)
    lens = [int(x) for x in g.integers(0, 4, 1300)]
    before = [0] * 1300
    for i, (n, m) in {100: (70, 20000), 700: (1, 9000), 701: (33, 20000), 1299: (2, 40000)}.items():
        lens[i], before[i] = n, m
    p = Packed(lens, before, nq, nkv, d, seed=20)
    out, lse = p.run()
    _agree_with_64_bits(p, lens, before, out, lse)


def test_starts_that_rise_and_fall_over_many_keys():
    """Sequences that overlap seem to have more pairs than the rows do: latched, and nothing past the lists is touched."""
    B, R, Rk, d = 100, 3840, 480000, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn(R, 1, d, device=DEV, generator=g).bfloat16()
    k = torch.randn(Rk, 1, d, device=DEV, generator=g).bfloat16()
    assert L.lib().eagle_op_attention_prompt_scratch_bytes(R, Rk, 1, 1, d, B) > 0
    qs = torch.tensor([0, R] * (B // 2) + [0], dtype=torch.int32, device=DEV)
    ks = torch.arange(0, Rk + 1, Rk // B, dtype=torch.int32, device=DEV)
    for scratch in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.zeros(R + 8, 1, d, dtype=torch.bfloat16, device=DEV)
        api.attention_prompt(q, k, k, qs, ks, out=out[:R], err=err, scratch=scratch)
        torch.cuda.synchronize()
        assert err.item() == 2 and torch.isfinite(out.float()).all() and not out[R:].any()


def test_values_that_are_not_finite_among_many_items():
    """The second pass over a CTA's items: results elsewhere keep their bits."""
    g = np.random.default_rng(3)
    lens = [int(x) for x in g.integers(1, 260, 80)]
    p = Packed(lens, [0] * 80, 8, 8, 128, seed=19)
    want, wlse = p.run()
    at = [int(p.kstart[b]) + lens[b] // 2 for b in range(0, 80, 7)]
    for i, x in enumerate(at):
        p.v[x, i % 8, i] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    out, lse = p.run()
    hit = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
    for i, (x, b) in enumerate(zip(at, range(0, 80, 7))):
        hit[x:p.start[b + 1], i % 8, i] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse, wlse)
    assert not torch.isfinite(out[hit].float()).any()


def _on_device(lens, before, nq, nkv, d, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    start, kstart = np.cumsum([0] + list(lens)), np.cumsum([0] + [n + b for n, b in zip(lens, before)])
    new = lambda rows, heads: torch.randn(int(rows), heads, d, device=DEV, dtype=torch.bfloat16, generator=g)  # noqa: E731
    return SimpleNamespace(q=new(start[-1], nq), k=new(kstart[-1], nkv), v=new(kstart[-1], nkv), start=start, kstart=kstart)


@pytest.mark.parametrize("nq,nkv,d", [(64, 1, 64), (8, 2, 128)])
def test_thousands_of_lengths(nq, nkv, d):
    """Sizes that differ from sequence to sequence, more of them than there are levels: each level holds several, of one sequence too."""
    g = np.random.default_rng(nq)
    before = (20000 * g.random(2500) ** 6).astype(int)
    lens = np.where(g.random(2500) < 0.01, g.integers(1, 700, 2500), g.integers(0, 3, 2500))
    p = _on_device(lens, before, nq, nkv, d, 21)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lse = torch.empty(p.q.shape[:2], device=DEV)
    out = api.attention_prompt(p.q, p.k, p.v, i32(p.start), i32(p.kstart), lse=lse, err=err)
    assert int(err) == 0
    _agree_with_64_bits(p, [int(x) for x in lens], [int(x) for x in before], out, lse)


def test_a_million_sequences():
    """As many sequences as are taken, nearly all empty, the others of as many sizes as there are of them. What a CTA goes through to
    find its next item stays far below the limit of a wait: (levels + 2) passes, 32768 rounds each, of which one level at most
    is taken here."""
    B, n = 1 << 20, 2000
    g = np.random.default_rng(22)
    lens, before = np.zeros(B, dtype=int), np.zeros(B, dtype=int)
    at = np.sort(g.choice(B, n, replace=False))
    lens[at], before[at] = 1, 4 * g.permutation(n)
    p = _on_device(lens, before, 64, 1, 64, 22)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lse = torch.full((n, 64), math.nan, device=DEV)
    out = torch.full((n, 64, 64), math.nan, dtype=torch.bfloat16, device=DEV)
    api.attention_prompt(p.q, p.k, p.v, i32(p.start), i32(p.kstart), out=out, lse=lse, err=err)
    assert int(err) == 0
    few = SimpleNamespace(q=p.q, k=p.k, v=p.v, start=np.arange(n + 1), kstart=np.append(p.kstart[at], p.kstart[-1]))
    _agree_with_64_bits(few, [1] * n, [int(x) for x in before[at]], out, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_the_most_keys(d):
    """One row behind 2^27 keys, not shared out: one CTA's item of a second or two, for which other warps wait. All keys are zero, so
    weights are equal; a few values are 2^20, the others zero: their sum is exact and the result within its one rounding."""
    n = 1 << 27
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros(n, 1, d, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(d)
    at = torch.randint(0, n, (3000,), device=DEV, generator=g)
    at[:4] = torch.tensor([0, 1, n - 2, n - 1], device=DEV)
    v[at, 0, torch.randint(0, d, (3000,), device=DEV, generator=g)] = 2.0 ** 20
    q = torch.randn(1, 1, d, device=DEV, generator=g).bfloat16()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lse = torch.zeros(1, 1, device=DEV)
    out = api.attention_prompt(q, k, v, i32([0, 1]), i32([0, n]), lse=lse, err=err, scratch=torch.empty(0, dtype=torch.uint8, device=DEV))
    assert int(err) == 0
    want = (v[:, 0] != 0).sum(0).double() * 2.0 ** 20 / n
    assert want.sum() > 0 and torch.all((out[0, 0].double() - want).abs() <= 2.0 ** -8 * want)
    assert abs(float(lse) - math.log(n)) <= 2.0 ** -22 * math.log(n)


def test_rows_of_skipped_sequences_are_left_alone():
    """Starts that fall or lie outside, no two sequences over the same rows: only rows of the valid ones are written, sums too."""
    p = Packed([30, 40, 20, 50], [0, 0, 0, 0], 4, 2, 128, seed=23, extra=0)
    want, wlse = p.run()
    s = p.start.tolist()
    for qs, ks in ((s, s[:2] + [29] + s[3:]), (s, s[:4] + [141]), (s[:4] + [2 ** 31 - 1], s), ([-1] + s[1:], s), (s, [-2 ** 31] + s[1:]),
                   (s, s[:2] + [-1] + s[3:])):
        fine = [b for b in range(4) if 0 <= qs[b] <= qs[b + 1] <= p.R and 0 <= ks[b] <= ks[b + 1] <= p.K]
        assert 2 <= len(fine) < 4
        for scratch in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
            out, lse = torch.full_like(want, 7.0), torch.full_like(wlse, 7.0)
            err = torch.zeros(1, dtype=torch.int32, device=DEV)
            api.attention_prompt(p.q, p.k, p.v, i32(qs), i32(ks), out=out, lse=lse, err=err, scratch=scratch)
            assert int(err) == 2
            valid = torch.zeros(p.R, dtype=torch.bool, device=DEV)
            for b in fine:
                valid[s[b]:s[b + 1]] = True
            same = [b for b in fine if ks[b] == s[b] and ks[b + 1] == s[b + 1]]
            assert torch.all(out[~valid] == 7) and torch.all(lse[~valid] == 7), (qs, ks)
            for b in same:
                assert torch.equal(out[s[b]:s[b + 1]], want[s[b]:s[b + 1]]) and torch.equal(lse[s[b]:s[b + 1]], wlse[s[b]:s[b + 1]])


def test_a_captured_call_of_few_rows_over_many_keys():
    """Keys shared out, its scratch memory made during the capture: replayed for other lengths, beside a second graph with scratch
    memory of its own, it gives what a call gives."""
    p = Packed([60, 3], [2500, 3500], 8, 2, 128, seed=24, extra=0)
    assert L.lib().eagle_op_attention_prompt_scratch_bytes(p.R, p.K, 8, 2, 128, 2) > 0
    qs, ks = i32(p.start), i32(p.kstart)
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        o, s = torch.zeros(63, 8, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(63, 8, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            api.attention_prompt(p.q, p.k, p.v, qs, ks, out=o, lse=s)
        outs.append((o, s)), graphs.append(g)
    for rows, keys in (([60, 3], [2560, 3503]), ([0, 63], [0, 6063]), ([62, 1], [63, 6000]), ([63, 0], [40, 6000]), ([1, 62], [6001, 62])):
        a, b = i32(np.cumsum([0] + rows)), i32(np.cumsum([0] + keys))
        qs.copy_(a), ks.copy_(b)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        lse = torch.zeros(63, 8, device=DEV)
        want = api.attention_prompt(p.q, p.k, p.v, a, b, lse=lse)
        for o, s in outs:
            assert torch.equal(o, want) and torch.equal(s, lse)
