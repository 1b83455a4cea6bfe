"""The 8-bit KV cache on the GPU: writing and reading bit for bit, attention against 64 bits.

Tolerance of an attention output, fixed before any run. With u the half step of a type (bf16 2^-8, fp16 2^-11),
W = sum p |v| / sum p and A the largest sum_i |q_i k_i| * scale that the row sees, both in 64 bits:
  2^-8 |o|                    the output's rounding;
  W * 2^-11 (own slots),      each weight's rounding before the value product: fp16, or bf16 for
  W * 2^-8 (prefix)           the prefix;
  W * 2 * (d + 8) * 2^-23 * A the score: d fp32 additions that may each lose a step of the partial sum, and
                              the products around them; an error x of a score moves a weight by x relative,
                              its own and, through the sum, everybody's;
  W * (n + 64) * 2^-23        n fp32 additions of the value product and of the sum, exp2 and the joins.
fp16 weights below 2^-14 round to a step of 2^-24, against a largest weight of at least 1 a row: n * 2^-25 * max|v|.
With head_dim 128 and more than 16 query vectors a block (rows x query heads of a KV head) q is held in 8-bit parts:
  W * 2 * 2^-17 * Q           q as two e4m3 parts, its largest entry in [2^7, 2^8): each entry is off by at most half of
                              their smallest step, 2^-10, so 2^-17 of the largest entry; Q = max|q| sum_i |k_i| * scale.
"""
import numpy as np
import pytest
import torch

from eagle_speculative_decoding_cycle_gb300 import _lib as L
from eagle_speculative_decoding_cycle_gb300 import api
from oracle import kv8 as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make_cache(B, nkv, cap, d, block=0, seed=0, fill=None):
    """A cache whose unused bytes hold `fill` (default: 0xa5), its blocks in a mixed order, two spare."""
    g = torch.Generator().manual_seed(seed)
    if block:
        per = -(-cap // block)
        n = B * per + 2
        table = (torch.randperm(n, generator=g)[:B * per]).to(torch.int32).view(B, per).to(DEV)
        shape = (n, nkv, block, d)
    else:
        table, shape = None, (B, nkv, -(-cap // 16) * 16, d)
    new = lambda s: torch.full(s, 0xa5 if fill is None else fill, dtype=torch.uint8, device=DEV)
    return api.KV8Cache(new(shape), new(shape), new(shape[:3]), new(shape[:3]), table)


def places(c, seq, slot):
    if c.table is None:
        return seq, slot
    return c.table.cpu().numpy()[seq, slot // c.block], slot % c.block


def host(t):
    return t.detach().cpu().numpy()


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).to(DEV)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---- writing and reading --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,nkv,d,block", [(1, 1, 64, 0), (7, 3, 128, 16), (61, 5, 64, 32), (333, 8, 128, 0),
                                           (129, 2, 64, 256)])
def test_write_and_read_bit_exact(dtype, R, nkv, d, block):
    g = torch.Generator().manual_seed(R + d)
    B, cap = 3, 352
    c = make_cache(B, nkv, cap, d, block)
    # strided rows: the middle columns of a fused projection, sizes from 2^-60 to 2^60, ties, zeros, both signs
    fused = torch.randn(R, 4, nkv, d, generator=g) * torch.exp2(torch.randint(-8, 8, (R, 4, nkv, 1), generator=g).float())
    fused[0, 1] *= 2.0 ** 60
    fused[R // 2, 1] = 0
    fused[R // 3, 2] = torch.round(fused[R // 3, 2] * 16) / 16
    fused[R - 1, 2] *= 2.0 ** -60
    fused = fused.to(dtype).to(DEV)
    k, v = fused[:, 1], fused[:, 2]
    pick = torch.randperm(B * cap, generator=g)[:R].numpy()
    seq, slot = pick // cap, pick % cap
    pad = np.zeros(R, bool)
    pad[1::5] = True
    err = err_word()
    before = [host(t).copy() for t in (c.k, c.v, c.k_exp, c.v_exp)]
    api.kv8_write(c, k, v, i32(np.where(pad, -1, seq)), i32(slot), err=err)
    assert int(err) == 0
    a, b = places(c, seq, slot)
    for x, codes, exps, cb, eb in ((k, c.k, c.k_exp, before[0], before[2]), (v, c.v, c.v_exp, before[1], before[3])):
        wc, we = O.quantise(x.double().cpu().numpy())
        for r in np.nonzero(~pad)[0]:
            cb[a[r], :, b[r]], eb[a[r], :, b[r]] = wc[r], we[r]
        assert np.array_equal(host(codes), cb) and np.array_equal(host(exps), eb)
    for out_t in (torch.float32, torch.bfloat16):
        wide = torch.full((R, 3, nkv, d), 7.0, dtype=out_t, device=DEV)   # gaps between the rows stay
        api.kv8_read(c, i32(np.where(pad, -1, seq)), i32(slot), out=(wide[:, 0], wide[:, 2]), err=err)
        assert int(err) == 0 and torch.all(wide[:, 1] == 7)
        for got, x in ((wide[:, 0], k), (wide[:, 2], v)):
            want = O.dequantise(*O.quantise(x.double().cpu().numpy()))
            want[pad] = 0
            assert np.array_equal(got.double().cpu().numpy(), want)


def test_write_special_values():
    d = 64
    x = torch.zeros(8, 1, d)
    x[1, 0, 5], x[2, 0, 6], x[3, 0, 0] = float("inf"), float("nan"), -float("inf")
    x[4] = torch.finfo(torch.float32).tiny * 2.0 ** -20       # subnormal inputs
    x[5] = 3e38                                              # past 448 * 2^40: saturates
    x[6, 0, :] = torch.linspace(-448, 448, d)
    x[7, 0, :] = -448.0001                                   # just past a border of the exponent
    c = make_cache(1, 1, 16, d)
    api.kv8_write(c, x.to(DEV), x.to(DEV), i32(np.zeros(8)), i32(np.arange(8)))
    wc, we = O.quantise(x.double().numpy())
    assert np.array_equal(host(c.k)[0, 0, :8], wc[:, 0]) and np.array_equal(host(c.k_exp)[0, 0, :8], we[:, 0])
    assert list(we[1:4, 0]) == [255, 255, 255] and we[5, 0] == 167 and we[0, 0] == 87
    k, _ = api.kv8_read(c, i32(np.zeros(8)), i32(np.arange(8)), dtype=torch.float32)
    want = O.dequantise(wc, we)
    assert np.array_equal(k.double().cpu().numpy(), want, equal_nan=True)


def test_rows_out_of_range_are_skipped_and_latched():
    c = make_cache(2, 2, 32, 64, block=16)
    c.table[1, 1] = -1
    before = [host(t).copy() for t in (c.k, c.v, c.k_exp, c.v_exp)]
    x = torch.ones(1, 2, 64, device=DEV)
    for seq, slot in ((2, 0), (0, 32), (0, -1), (1, 16), (2 ** 30, 3)):
        err = err_word()
        api.kv8_write(c, x, x, i32([seq]), i32([slot]), err=err)
        assert int(err) == 2, (seq, slot)
        k, v = api.kv8_read(c, i32([seq]), i32([slot]), err=err_word())
        assert not k.any() and not v.any()
        api.kv8_write(c, x, x, i32([seq]), i32([slot]))      # without a status word: skipped all the same
    for t, b in zip((c.k, c.v, c.k_exp, c.v_exp), before):
        assert np.array_equal(host(t), b)
    api.kv8_write(c, x[:0], x[:0], i32([]), i32([]))          # no rows
    assert api.kv8_read(c, i32([]), i32([]))[0].shape == (0, 2, 64)


def test_moving_entries_keeps_their_values():
    """Reading an accepted path and writing it at the committed slots stores the same values."""
    g = torch.Generator().manual_seed(5)
    c = make_cache(2, 4, 64, 128)
    x = torch.randn(80, 4, 128, generator=g).to(torch.bfloat16).to(DEV)
    seq, slot = i32(np.repeat([0, 1], 40)), i32(np.tile(np.arange(40), 2))
    api.kv8_write(c, x, 2 * x, seq, slot)
    src, dst = i32([20, 23, 31, 22, 29, 30]), i32([20, 21, 22, 20, 21, 22])
    who = i32([0, 0, 0, 1, 1, 1])
    k, v = api.kv8_read(c, who, src)
    api.kv8_write(c, k, v, who, dst)
    k2, v2 = api.kv8_read(c, who, dst)
    assert torch.equal(k, k2) and torch.equal(v, v2)


# ---- attention ------------------------------------------------------------------------------------
def bits_of(rows, T):
    """[R][words] int64 masks from boolean rows [R, T]."""
    words = (T + 63) // 64
    out = np.zeros((len(rows), words), np.uint64)
    for r, row in enumerate(rows):
        for t in np.nonzero(row)[0]:
            out[r, t // 64] |= np.uint64(1) << np.uint64(t % 64)
    return torch.from_numpy(out.view(np.int64)).to(DEV)


def random_tree(T, g):
    see = np.zeros((T, T), bool)
    for i in range(T):
        if i:
            see[i] = see[int(g.integers(0, i))]
        see[i, i] = True
    return see


class Case:
    """A filled cache, rows and what they see; check() compares the GPU's rows with 64 bits."""

    def __init__(self, B, T, nq, nkv, d, ctx, mode, block=0, P=0, seed=0, qscale=2.0, vspread=0.7, cap=None, fill=None,
                 kspread=0.0):
        g = np.random.default_rng(seed)
        self.g, self.B, self.T, self.nq, self.nkv, self.d, self.mode, self.P = g, B, T, nq, nkv, d, mode, P
        self.ctx = np.asarray(ctx if np.ndim(ctx) else [ctx] * B)
        cap = cap or int(max(self.ctx)) + T
        self.c = make_cache(B, nkv, cap, d, block, seed, fill)
        n = int(max(self.ctx)) + T
        seq = np.repeat(np.arange(B), n)
        slot = np.tile(np.arange(n), B)
        on = slot < self.ctx[seq] + T
        self.k = g.normal(size=(B, n, nkv, d)) * np.exp(0.5 * g.normal(size=(nkv, d))) * \
            np.exp(kspread * g.normal(size=(B, n, nkv, 1)))
        self.v = g.normal(size=(B, n, nkv, d)) * np.exp(vspread * g.normal(size=(B, n, nkv, 1)))
        flat = lambda x: torch.from_numpy(x.reshape(B * n, nkv, d)[on]).float().to(DEV)
        api.kv8_write(self.c, flat(self.k), flat(self.v), i32(seq[on]), i32(slot[on]))
        self.K, self.V = (O.dequantise(*O.quantise(x.astype(np.float32).astype(np.float64))) for x in (self.k, self.v))
        self.q = torch.from_numpy(qscale * g.normal(size=(B * T, nq, d))).to(torch.bfloat16).to(DEV)
        self.pk = torch.from_numpy(g.normal(size=(nkv, P, d))).to(torch.bfloat16).to(DEV) if P else None
        self.pv = torch.from_numpy(g.normal(size=(nkv, P, d))).to(torch.bfloat16).to(DEV) if P else None
        self.row_seq = np.repeat(np.arange(B), T)
        self.row_slot = (self.ctx[:, None] + np.arange(T)).reshape(-1)
        self.trees = np.stack([random_tree(T, g) for _ in range(B)]).reshape(B * T, T) if mode == 1 else None
        self.scale = 0.0

    def run(self, **kw):
        mask = bits_of(self.trees, self.T) if self.mode == 1 else None
        self.err = err_word()
        out = api.attention_shared_kv8(self.q, self.pk, self.pv, self.c, i32(self.row_seq), i32(self.row_slot), i32(self.ctx),
                                       self.T, self.mode, self.T if self.mode == 1 else 0, mask, self.scale, err=self.err, **kw)
        return out

    def want(self, rows=None):
        B, T, nq, nkv, d, P = self.B, self.T, self.nq, self.nkv, self.d, self.P
        G, n = nq // nkv, self.K.shape[1]
        scale = self.scale or d ** -0.5
        q = self.q.double().cpu().numpy()
        out, tol = np.zeros((B * T, nq, d)), np.zeros((B * T, nq, d))
        for r in (range(B * T) if rows is None else rows):
            b = self.row_seq[r]
            if b < 0:
                continue
            see = np.zeros(n, bool)
            if self.mode == 0:
                see[:self.row_slot[r] + 1] = True
            else:
                see[:self.ctx[b]] = True
                see[self.ctx[b]:self.ctx[b] + T] = self.trees[r]
            for h in range(nkv):
                K, V, s = self.K[b, :, h], self.V[b, :, h], see
                if P:
                    K = np.concatenate([self.pk[h].double().cpu().numpy(), K])
                    V = np.concatenate([self.pv[h].double().cpu().numpy(), V])
                    s = np.concatenate([np.ones(P, bool), see])
                o, W, A = O.attend(q[r, h * G:(h + 1) * G], K, V, np.broadcast_to(s, (G, len(s))), scale)
                out[r, h * G:(h + 1) * G] = o
                count = int(s.sum())
                top = np.abs(V[s]).max() if count else 0.0
                nb = -(-T // (128 // G))
                parts = d == 128 and -(-T // nb) * G > 16
                Q = np.abs(q[r, h * G:(h + 1) * G]).max(-1) * np.abs(K[s]).sum(-1).max(initial=0.0) * scale
                tol[r, h * G:(h + 1) * G] = 2.0 ** -8 * np.abs(o) + count * 2.0 ** -25 * top + \
                    W * ((2.0 ** -8 if P else 2.0 ** -11) + 2 * (d + 8) * 2.0 ** -23 * A[:, None] +
                         (count + 64) * 2.0 ** -23 + parts * 2 * 2.0 ** -17 * Q[:, None])
        return out, tol

    def check(self, out=None, rows=None):
        out = self.run() if out is None else out
        assert int(self.err) == 0
        want, tol = self.want(rows)
        got = out.double().cpu().numpy()
        at = slice(None) if rows is None else rows
        bad = np.abs(got[at] - want[at]) - tol[at]
        assert not np.isnan(got[at]).any() and bad.max() <= 0, f"off by {np.abs(got[at] - want[at]).max()}, {bad.max()} too much"
        return out


@pytest.mark.parametrize("P", [0, 1, 130])
@pytest.mark.parametrize("B,T,nq,nkv,d,ctx,mode,block", [
    (1, 1, 1, 1, 64, 0, 0, 0),                      # one row that sees itself
    (1, 1, 32, 8, 128, 700, 0, 0),                  # a decoding step
    (3, 1, 8, 2, 128, [0, 31, 32], 0, 16),          # lengths around a tile
    (5, 1, 5, 5, 64, [1, 15, 16, 63, 257], 0, 32),  # odd head count, one query head per KV head
    (4, 17, 32, 8, 128, [0, 5, 130, 333], 1, 16),   # a batch's verify pass
    (1, 61, 8, 2, 128, 300, 1, 0),                  # two row blocks
    (2, 7, 28, 4, 64, [9, 200], 1, 64),             # seven query heads a KV head
    (2, 100, 10, 5, 64, [3, 77], 1, 0),             # masks of two words, a prompt-sized row count
    (1, 70, 4, 4, 128, 13, 0, 0),                   # a causal chunk
    (2, 2, 64, 1, 128, [40, 90], 1, 256),           # 64 query heads on one KV head
    (1, 3, 48, 1, 64, 129, 0, 16),                  # 48
])
def test_attention_matches_64_bits(B, T, nq, nkv, d, ctx, mode, block, P):
    Case(B, T, nq, nkv, d, ctx, mode, block, P, seed=B + T).check()


@pytest.mark.parametrize("P", [0, 77])
def test_rows_that_see_nothing_and_padding(P):
    k = Case(3, 5, 8, 2, 128, [0, 40, 0], 1, P=P, seed=3)
    k.trees[1] = False                        # sees nothing of its own: no context, empty mask
    k.trees[5 + 2] = False                    # sees its context only
    k.row_seq[[2, 3, 4]] = -1                 # padding behind real rows
    k.row_seq[10] = -1                        # and in front of them
    out = k.check()
    assert not out[[2, 3, 4, 10]].any()
    if not P:
        assert not out[1].any()
    k.row_seq[:] = -1
    assert not k.run().any() and int(k.err) == 0


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("fill", [0x7f, 0xff])
def test_hidden_slots_may_hold_anything(mode, fill):
    """Unwritten bytes that read as NaN, a written NaN and an infinity in slots that a row does not see."""
    k = Case(2, 6, 8, 2, 128, [45, 70], mode, seed=4, fill=fill, cap=112)
    bad = torch.full((2, 2, 128), float("nan"), device=DEV)
    bad[1] = float("inf")
    if mode == 1:
        k.trees[:, 3] = False                 # tree slot 3 seen by no row (its own neither)
        api.kv8_write(k.c, bad, bad, i32([0, 1]), i32(k.ctx + 3))
    else:
        k.row_slot -= 2                       # the last two slots are past every row
        api.kv8_write(k.c, bad, bad, i32([0, 1]), i32(k.ctx + 4))
    k.K[[0, 1], k.ctx + (3 if mode else 4)] = np.nan
    k.V[[0, 1], k.ctx + (3 if mode else 4)] = np.nan
    k.check()


def test_a_nan_reaches_the_rows_that_see_it_and_no_other():
    k = Case(2, 6, 8, 2, 128, [45, 70], 1, seed=5)
    nan = torch.full((1, 2, 128), float("nan"), device=DEV)
    one = torch.ones(1, 2, 128, device=DEV)
    api.kv8_write(k.c, nan, one, i32([0]), i32(k.ctx[:1] + 5))       # key of tree slot 5 of sequence 0
    api.kv8_write(k.c, one, nan, i32([1]), i32(k.ctx[1:] + 5))       # value of tree slot 5 of sequence 1
    out = k.run()
    for b in range(2):
        for t in range(6):
            got = out[b * 6 + t]
            assert torch.isnan(got).all() if k.trees[b * 6 + t, 5] else torch.isfinite(got).all()
    q0 = k.q.clone()
    k.q[7, 3, 9] = float("nan")
    k.q[8, 1, 0] = float("inf")
    other = k.run()
    assert torch.isnan(other[7, 3]).all() and torch.isnan(other[8, 1]).all()
    keep = torch.ones(12, 8, dtype=torch.bool, device=DEV)
    keep[7, 3] = keep[8, 1] = False
    assert torch.equal(other[keep].view(torch.int16), out[keep].view(torch.int16))
    k.q.copy_(q0)


@pytest.mark.parametrize("qscale,vspread,kspread", [(0.0, 0.7, 0.0), (1e-30, 0.7, 0.0), (40.0, 0.7, 0.0), (2.0, 6.0, 0.0),
                                                    (2.0, 0.0, 3.0)])
def test_wide_value_ranges(qscale, vspread, kspread):
    """Zero and tiny queries, peaked rows, values and keys whose sizes differ by many powers of two."""
    Case(2, 9, 8, 2, 128, [200, 513], 1, seed=6, qscale=qscale, vspread=vspread, kspread=kspread).check()


def test_values_far_apart_in_one_tile():
    """A row that looks at a small value beside a huge one it hardly sees keeps the small one's digits."""
    k = Case(1, 1, 4, 1, 128, 63, 0, seed=7)
    big = np.zeros((1, 1, 128))
    kk = np.zeros((1, 1, 128))
    for s, size in ((10, 2.0 ** 30), (11, 2.0 ** -30), (40, 2.0 ** 12)):
        big[...] = size * k.g.normal(size=128)
        kk[...] = -60.0 if s == 10 else (60.0 if s == 11 else -60.0)
        api.kv8_write(k.c, torch.from_numpy(kk).float().to(DEV), torch.from_numpy(big).float().to(DEV), i32([0]), i32([s]))
        k.K[0, s] = O.dequantise(*O.quantise(kk[0]))
        k.V[0, s] = O.dequantise(*O.quantise(big[0].astype(np.float32).astype(np.float64)))
    k.q.fill_(1.0)
    want, _ = k.want()
    got = k.run().double().cpu().numpy()
    assert np.max(np.abs(got - want)) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want).max()


@pytest.mark.parametrize("ctx,block,P", [(20000, 0, 0), (9000, 64, 0), (50, 16, 5000)])
def test_long_contexts(ctx, block, P):
    k = Case(1, 2, 8, 2, 64, ctx, 0, block, P, seed=8)
    k.check()


def test_scale_and_out_arguments():
    k = Case(2, 3, 8, 2, 64, [20, 50], 1, seed=9)
    k.scale = 0.05
    out = torch.empty_like(k.q)
    assert k.check(k.run(out=out)) is out
    big = torch.full((9, 8, 64), 5.0, dtype=torch.bfloat16, device=DEV)     # rows behind the last are left as they were
    k.run(out=big[:6])
    assert torch.equal(big[:6], out) and torch.all(big[6:] == 5)


def test_slots_past_the_capacity_are_left_out_and_latched():
    k = Case(2, 4, 8, 2, 64, [10, 28], 1, seed=10, cap=32)      # sequence 1 fills its 32 slots
    k.check()
    k.ctx = np.asarray([10, 30])                                # two of its tree slots are past the end
    k.K = np.concatenate([k.K, np.zeros((2, 2, 2, 64))], 1)
    k.V = np.concatenate([k.V, np.zeros((2, 2, 2, 64))], 1)
    k.trees[4:, 2:] = False
    want, tol = k.want()
    k.trees[4:, 2:] = True
    out = k.run().double().cpu().numpy()
    assert int(k.err) == 2 and np.all(np.abs(out - want) <= tol)
    k.ctx = np.asarray([10, 28])
    k.row_seq[1], k.row_seq[5] = 1, 9                           # a row of another sequence; one outside the cache
    out = k.run()
    assert int(k.err) == 2 and not out[[1, 5]].any()


@pytest.mark.parametrize("P", [0, 150])
def test_rows_do_not_depend_on_other_rows_values(P):
    k = Case(3, 9, 16, 4, 128, [64, 200, 31], 1, 16, P, seed=11)
    a = k.run()
    k.q[:9] = 3
    k.q[20] = -1
    b = k.run()
    keep = [r for r in range(27) if r >= 9 and r != 20]
    assert torch.equal(a[keep], b[keep])
    assert torch.equal(k.run(), b)                              # and a second call gives the same bits


@pytest.mark.parametrize("P", [0, 300])
def test_graphs_streams_and_reused_scratch(P):
    """Captured calls replayed on new inputs, two graphs with a scratch each on two streams, a scratch that held
    another call's sums."""
    k = Case(4, 5, 32, 8, 128, [100, 3, 250, 31], 1, 16, P, seed=12)
    want = k.run()
    mask = bits_of(k.trees, 5)
    rs, sl, cx = i32(k.row_seq), i32(k.row_slot), i32(k.ctx)
    outs, graphs, streams, scratch = [], [], [], []
    for i in range(2):
        st = torch.cuda.Stream()
        s = api.attention_kv8_scratch(k.c, 20, 32, 5, P)
        s.fill_(0xff)
        o = torch.empty_like(k.q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            api.attention_shared_kv8(k.q, k.pk, k.pv, k.c, rs, sl, cx, 5, 1, 5, mask, out=o, scratch=s)
        outs.append(o), graphs.append(g), streams.append(st), scratch.append(s)
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    k.q.mul_(-1)
    cx.copy_(i32([90, 0, 251, 17]))
    k.ctx = np.asarray([90, 0, 251, 17])
    k2 = k.run(scratch=scratch[1])
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], k2)


def test_a_serving_run():
    """A run as a batch would have it: prompts behind a shared prefix written, verify passes over trees, accepted
    paths moved to their committed slots by read and write, decoding steps - against 64 bits at every step."""
    g = np.random.default_rng(20)
    B, T, nq, nkv, d, P, cap = 3, 8, 8, 2, 128, 200, 96
    c = api.KV8Cache.empty(B, nkv, cap, d, device=DEV, block=16)
    c.table.copy_(torch.randperm(c.n_blocks).to(torch.int32).view(B, -1))
    pk, pv = (torch.from_numpy(g.normal(size=(nkv, P, d))).to(torch.bfloat16).to(DEV) for _ in range(2))
    scratch = api.attention_kv8_scratch(c, B * T, nq, T, P)
    step_scratch = api.attention_kv8_scratch(c, B, nq, 1, P)
    hist = [[] for _ in range(B)]                    # the committed (K, V) rows of each sequence, dequantised
    new = lambda n: torch.from_numpy(g.normal(size=(n, nkv, d))).to(torch.bfloat16).to(DEV)
    deq = lambda x: O.dequantise(*O.quantise(x.double().cpu().numpy()))

    def expect(q, b, extra):
        K = np.concatenate([pk.double().cpu().numpy()] + [k[:, None] for k, _ in hist[b] + extra], 1)
        V = np.concatenate([pv.double().cpu().numpy()] + [v[:, None] for _, v in hist[b] + extra], 1)
        out, tol = np.zeros((nq, d)), np.zeros((nq, d))
        for h in range(nkv):
            qs = slice(h * nq // nkv, (h + 1) * nq // nkv)
            o, W, A = O.attend(q[qs], K[h], V[h], np.ones((nq // nkv, K.shape[1]), bool), d ** -0.5)
            out[qs] = o
            tol[qs] = 2.0 ** -8 * np.abs(o) + W * (2.0 ** -8 + 2 * (d + 8) * 2.0 ** -23 * A[:, None] + 2.0 ** -14)
        return out, tol

    n0 = [0, 5, 17]
    for b in range(B):
        if n0[b]:
            k, v = new(n0[b]), new(n0[b])
            api.kv8_write(c, k, v, i32([b] * n0[b]), i32(np.arange(n0[b])))
            hist[b] = list(zip(deq(k), deq(v)))
    for cycle in range(3):
        ctx = np.asarray([len(h) for h in hist])
        trees = np.stack([random_tree(T, g) for _ in range(B)])
        k, v, q = new(B * T), new(B * T), torch.from_numpy(2 * g.normal(size=(B * T, nq, d))).to(torch.bfloat16).to(DEV)
        seq, slot = np.repeat(np.arange(B), T), (ctx[:, None] + np.arange(T)).reshape(-1)
        api.kv8_write(c, k, v, i32(seq), i32(slot))
        out = api.attention_shared_kv8(q, pk, pv, c, i32(seq), None, i32(ctx), T, 1, T, bits_of(trees.reshape(B * T, T), T),
                                       scratch=scratch).double().cpu().numpy()
        kd, vd = deq(k).reshape(B, T, nkv, d), deq(v).reshape(B, T, nkv, d)
        take_s, take_from, take_to = [], [], []
        for b in range(B):
            for t in range(T):
                path = [(kd[b, a], vd[b, a]) for a in np.nonzero(trees[b, t])[0]]
                want, tol = expect(q[b * T + t].double().cpu().numpy(), b, path)
                assert np.all(np.abs(out[b * T + t] - want) <= tol)
            leaf = int(g.integers(0, T))
            path = list(np.nonzero(trees[b, leaf])[0])
            take_s += [b] * len(path)
            take_from += [ctx[b] + a for a in path]
            take_to += [ctx[b] + j for j in range(len(path))]
            hist[b] = hist[b] + [(kd[b, a], vd[b, a]) for a in path]
        ak, av = api.kv8_read(c, i32(take_s), i32(take_from))
        api.kv8_write(c, ak, av, i32(take_s), i32(take_to))
        # one plain decoding step of every sequence
        k, v, q = new(B), new(B), torch.from_numpy(2 * g.normal(size=(B, nq, d))).to(torch.bfloat16).to(DEV)
        at = np.asarray([len(h) for h in hist])
        api.kv8_write(c, k, v, i32(np.arange(B)), i32(at))
        out = api.attention_shared_kv8(q, pk, pv, c, i32(np.arange(B)), i32(at), None, 1, 0,
                                       scratch=step_scratch).double().cpu().numpy()
        for b in range(B):
            hist[b] = hist[b] + [(deq(k)[b], deq(v)[b])]
            want, tol = expect(q[b].double().cpu().numpy(), b, [])
            assert np.all(np.abs(out[b] - want) <= tol)


# ---- more shapes of work --------------------------------------------------------------------------
@pytest.mark.parametrize("B,T,nq,nkv,d,most,mode,block,P", [
    (600, 1, 4, 2, 64, 40, 0, 16, 0),        # more row blocks than one launch takes
    (600, 1, 4, 2, 64, 40, 0, 0, 50),        # the same behind a prefix
    (530, 9, 8, 1, 128, 70, 1, 16, 130),     # 72 query vectors a block
    (64, 1, 16, 8, 128, 200, 0, 16, 0),      # more (block, head) items than CTAs
    (64, 12, 32, 8, 128, 150, 1, 32, 0),     # the same with 48 query vectors
])
def test_many_sequences(B, T, nq, nkv, d, most, mode, block, P):
    ctx = np.random.default_rng(B + T).integers(0, most, size=B)
    k = Case(B, T, nq, nkv, d, ctx, mode, block, P, seed=30)
    pick = sorted({0, B * T - 1, 511 * T % (B * T), 512 * T % (B * T)} | set(k.g.integers(0, B * T, 25).tolist()))
    a = k.check(rows=pick)
    assert torch.equal(k.run(), a)


@pytest.mark.parametrize("B,T,nq,nkv,d,ctx,mode,block,vspread,P", [
    (1, 9, 4, 1, 128, 3, 1, 0, 0.7, 0),             # a cache shorter than a tile, 36 query vectors
    (2, 200, 4, 2, 128, [5, 60], 0, 16, 0.7, 0),    # a causal chunk in four row blocks
    (2, 60, 4, 2, 64, [131, 20], 0, 0, 0.7, 90),    # 120 query vectors of 64
    (2, 9, 8, 2, 64, [100, 300], 1, 16, 6.0, 0),    # values of many sizes in one tile
    (1, 30, 8, 2, 128, [250], 0, 64, 6.0, 0),
    (2, 12, 16, 2, 128, [0, 140], 1, 0, 6.0, 200),
])
def test_row_blocks_of_many_query_vectors(B, T, nq, nkv, d, ctx, mode, block, vspread, P):
    Case(B, T, nq, nkv, d, ctx, mode, block, P, seed=31, vspread=vspread).check()


@pytest.mark.parametrize("T,P", [(1, 0), (12, 0), (12, 140)])
def test_results_over_the_queries(T, P):
    """out = q is allowed: the same bits as into a tensor of its own."""
    k = Case(5, T, 16, 4, 128, [300, 0, 77, 128, 3], 1, 16, P, seed=32)
    want = k.run()
    assert k.run(out=k.q) is k.q and torch.equal(k.q, want) and int(k.err) == 0


@pytest.mark.parametrize("T,d,P", [(1, 64, 0), (12, 128, 0), (12, 128, 140)])
def test_two_graphs_and_a_side_stream(T, d, P):
    k = Case(6, T, 16, 4, d, [300, 0, 77, 128, 3, 64], 1, 16, P, seed=33)
    want = k.run()
    mask, rs, cx = bits_of(k.trees, T), i32(k.row_seq), i32(k.ctx)
    call = lambda **kw: api.attention_shared_kv8(k.q, k.pk, k.pv, k.c, rs, None, cx, T, 1, T, mask, **kw)
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        s = api.attention_kv8_scratch(k.c, 6 * T, 16, T, P)
        s.fill_(0xff)
        o = torch.empty_like(k.q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call(out=o, scratch=s)
        outs.append((o, s)), graphs.append(g)
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o, _ in outs)
    side = torch.cuda.Stream()
    got = [call(stream=side) for _ in range(8)]       # results and scratch are made for the side stream
    kk = api.kv8_read(k.c, rs, rs, stream=side)
    side.synchronize()
    assert all(torch.equal(o, want) for o in got)
    assert all(torch.equal(a, b) for a, b in zip(kk, api.kv8_read(k.c, rs, rs)))


@pytest.mark.parametrize("P", [0, 33])
def test_a_negative_context_hides_its_sequence(P):
    k = Case(3, 12, 8, 2, 128, [40, 25, 9], 1, P=P, seed=34)
    k.ctx = np.asarray([40, -5, 9])
    out = k.run()
    assert int(k.err) == 2
    k.ctx = np.asarray([40, 0, 9])
    k.trees[12:24] = False                             # the prefix alone, or nothing
    want, tol = k.want()
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("T,P", [(1, 200), (12, 200), (12, 0)])
def test_inputs_changed_between_calls(T, P):
    """Queries, lengths, masks and cache entries rewritten in place on the stream just before each call."""
    k = Case(6, T, 16, 4, 128, [300, 0, 77, 128, 3, 64], 1, 16, P, seed=35)
    rs, qs = i32(k.row_seq), [k.q.roll(j, 0).clone() for j in range(6)]
    cs = [i32((k.ctx + 37 * j) % 290) for j in range(6)]
    ms = [bits_of(np.roll(k.trees, j * T, 0), T) for j in range(6)]
    ks = [torch.randn(6, 4, 128, device=DEV) for _ in range(6)]
    slot = i32(np.zeros(6))
    seqs = i32(np.arange(6))
    q, cx, mask = k.q.clone(), cs[0].clone(), ms[0].clone()

    def step(j):
        q.copy_(qs[j]), mask.copy_(ms[j])
        api.kv8_write(k.c, ks[j], ks[j], seqs, slot)
        cx.copy_(cs[j])
        return api.attention_shared_kv8(q, k.pk, k.pv, k.c, rs, None, cx, T, 1, T, mask)

    alone = []
    for j in range(6):
        alone.append(step(j))
        torch.cuda.synchronize()
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(alone, [step(j) for j in range(6)]))


@pytest.mark.parametrize("T,R,d,P", [(9, 24, 128, 0), (9, 19, 128, 60), (3, 7, 64, 0), (40, 95, 128, 0)])
def test_a_last_sequence_with_fewer_rows(T, R, d, P):
    k = Case(3, T, 16, 4, d, [50, 200, 7], 1, 16, P, seed=36)
    k.err = err_word()
    mask = bits_of(k.trees, T)
    big = torch.full_like(k.q, 9.0)
    out = api.attention_shared_kv8(k.q[:R], k.pk, k.pv, k.c, i32(k.row_seq[:R]), None, i32(k.ctx), T, 1, T, mask[:R],
                                   out=big[:R], err=k.err)
    want, tol = k.want(range(R))
    assert int(k.err) == 0 and torch.all(big[R:] == 9)
    assert np.all(np.abs(out.double().cpu().numpy() - want[:R]) <= tol[:R])


def test_one_sequence_of_more_rows_than_there_are():
    k = Case(1, 5, 8, 2, 128, 90, 0, 16, seed=37)
    a = k.check()
    k.T = 1 << 20
    b = k.run()
    assert int(k.err) == 0 and torch.equal(a, b)


@pytest.mark.parametrize("T,block", [(1, 0), (12, 0), (1, 256), (12, 256)])
def test_a_cache_of_more_than_four_gigabytes(T, block):
    """Codes past 2^32 bytes: the last heads of a long contiguous cache, blocks from all over a large pool."""
    k = Case(1, T, 16, 4, 128, 600, 1, block, seed=38, cap=1 << 24)
    assert k.c.k.numel() > 2 ** 32
    k.check()
    n = 600 + T
    got, _ = api.kv8_read(k.c, i32(np.zeros(n)), i32(np.arange(n)), dtype=torch.float32)
    assert np.array_equal(got.double().cpu().numpy(), k.K[0])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 12])
@pytest.mark.parametrize("block", [16, 32, 64, 256])
@pytest.mark.parametrize("P", [0, 40])
def test_blocks_that_are_not_assigned(block, T, d, P):
    """Table entries below a sequence's length that are -1 or past the pool, one or all of them: latched, and the other
    sequences' rows keep their bits."""
    k = Case(3, T, 16, 4, d, [150, 300, 77], 1, block, P, seed=40)
    want = k.check()
    good = k.c.table.clone()
    others = [r for r in range(3 * T) if r // T != 1]
    for at, entry in ((0, -1), (299 // block, k.c.n_blocks), (100 // block, -2 ** 31), (64 // block, 2 ** 31 - 1),
                      (slice(None), -1)):
        k.c.table.copy_(good)
        k.c.table[1, at] = entry
        out = k.run()
        assert int(k.err) == 2, (at, entry)
        assert torch.equal(out[others], want[others]), (at, entry)
    k.c.table.copy_(good)
    assert torch.equal(k.run(), want) and int(k.err) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 12])
@pytest.mark.parametrize("P", [0, 40])
def test_slots_that_were_never_written(T, d, P):
    """Cleared memory (KV8Cache.empty) in slots that rows see, between written ones and before them: zero keys and
    values, as kv8_read gives them."""
    k = Case(3, T, 16, 4, d, [300, 290, 70], 1, 0, P, seed=41)
    for b, lo, hi in ((0, 100, 200), (0, 17, 18), (1, 0, 45), (1, 60, 64), (1, 289, 290), (2, 0, 70 + T)):
        for t in (k.c.k, k.c.v, k.c.k_exp, k.c.v_exp):
            t[b, :, lo:hi] = 0
        k.K[b, lo:hi] = 0
        k.V[b, lo:hi] = 0
    kk, vv = api.kv8_read(k.c, i32([0] * 100), i32(np.arange(100, 200)))
    assert not kk.any() and not vv.any()
    out = k.check()
    if not P:
        assert not out[2 * T:].any()
    assert torch.equal(k.run(), out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 12])
def test_written_and_cleared_bands(T, d):
    """Long ranges a CTA in which written and cleared bands of 128 slots take turns."""
    k = Case(12, T, 16, 8, d, 2000, 1, seed=42)
    off = np.nonzero(np.arange(2000) // 128 % 2)[0]
    for t in (k.c.k, k.c.v, k.c.k_exp, k.c.v_exp):
        t[:, :, torch.from_numpy(off).to(DEV)] = 0
    k.K[:, off] = 0
    k.V[:, off] = 0
    k.check(rows=[0, T, 12 * T - 1])


@pytest.mark.parametrize("T,d", [(1, 64), (12, 64), (1, 128), (12, 128)])
@pytest.mark.parametrize("P", [0, 40])
def test_many_small_weights_beside_large_values(T, d, P):
    """Thousands of keys of weight 2^-16 next to one of weight 1, and in every tile a value 2^12 times the others' size
    whose weight is nothing: the small ones' sum counts. Tolerance: as above, but a weight's absolute step is at most
    2^-24 of a largest one of at least 2^7 (each product p |v| against the row's largest), so n * 2^-31 * max p |v| / sum p
    in the place of n * 2^-25 * max|V|."""
    k = Case(1, T, 16, 4, d, 6000, 1, 16, P, seed=43)
    n, g = 6000 + T, k.g
    x = np.full(n, -16.3)                                # scores in log2 units
    x[::32] = -200.0
    x[5] = 0.0
    V = 1 + 0.1 * g.normal(size=(n, 4, d))
    V[::32] = 6000.0
    V[5] = g.normal(size=(4, d))
    K = np.broadcast_to((x * d ** -0.5 * np.log(2))[:, None, None], (n, 4, d))
    k.q.fill_(1.0)
    if P:                                                # a prefix that weighs 2^-20 at most in all
        k.pk.fill_(-4.0)
    rows = lambda y: torch.from_numpy(np.ascontiguousarray(y)).float().to(DEV)
    api.kv8_write(k.c, rows(K), rows(V), i32(np.zeros(n)), i32(np.arange(n)))
    k.K, k.V = (O.dequantise(*O.quantise(y.astype(np.float32).astype(np.float64)))[None] for y in (K, V))
    B = 40                                               # as many sequences over the same blocks: long ranges a CTA
    c = api.KV8Cache(k.c.k, k.c.v, k.c.k_exp, k.c.v_exp, k.c.table.expand(B, -1).contiguous())
    err = err_word()
    got = api.attention_shared_kv8(k.q.repeat(B, 1, 1), k.pk, k.pv, c, i32(np.repeat(np.arange(B), T)), None, i32([6000] * B),
                                   T, 1, T, bits_of(k.trees, T).repeat(B, 1), err=err).double().cpu().numpy()
    assert int(err) == 0
    got = got.reshape(B, T, 4, 4, d)
    for r in range(T):
        see = np.concatenate([np.ones(6000, bool), k.trees[r]])
        for h in range(4):
            Kh, Vh = k.K[0, see, h], k.V[0, see, h]
            if P:
                Kh = np.concatenate([k.pk[h].double().cpu().numpy(), Kh])
                Vh = np.concatenate([k.pv[h].double().cpu().numpy(), Vh])
            count = len(Kh)
            s = Kh.sum(-1) * d ** -0.5
            p = np.exp(s - s.max())
            o, W = p @ Vh / p.sum(), p @ np.abs(Vh) / p.sum()
            A = np.abs(s).max()
            tol = 2.0 ** -8 * np.abs(o) + W * ((2.0 ** -8 if P else 2.0 ** -11) + 2 * (d + 8) * 2.0 ** -23 * A +
                                               (count + 64) * 2.0 ** -23 + (d == 128) * 2 * 2.0 ** -17 * A) + \
                count * 2.0 ** -31 * (p * np.abs(Vh).max(-1)).max() / p.sum()
            off = np.abs(got[:, r, h] - o) / tol
            assert off.max() <= 1, f"row {r} head {h}: {off.max()} times the tolerance"


@pytest.mark.parametrize("T,d", [(2, 64), (12, 64), (2, 128), (12, 128)])
def test_rows_do_not_depend_on_values_that_others_see(T, d):
    """A value of 2^14 times the others' size in a tree slot: rows that do not see it keep their bits."""
    k = Case(2, T, 16, 4, d, [500, 77], 1, 16, seed=44)
    k.trees[:, T - 1] = False
    k.trees[T - 1, T - 1] = k.trees[2 * T - 1, T - 1] = True
    a = k.run()
    x = k.g.normal(size=(2, 4, d))
    api.kv8_write(k.c, torch.from_numpy(x).float().to(DEV), torch.from_numpy(2.0 ** 14 * x).float().to(DEV), i32([0, 1]),
                  i32(k.ctx + T - 1))
    b = k.run()
    keep = [r for r in range(2 * T) if r % T != T - 1]
    same = torch.equal(a[keep], b[keep])
    assert same


@pytest.mark.parametrize("T,d,P", [(300, 64, 0), (300, 128, 0), (70, 128, 40)])
def test_padding_in_front_of_long_chunks(T, d, P):
    """Chunks whose first rows are padding, up to all but the last and all, in several row blocks."""
    k = Case(5, T, 8, 4, d, [40, 0, 9, 77, 130], 0, 16, P, seed=45)
    rows = k.row_seq.reshape(5, T)
    for b, n in enumerate((1, T - 1, T, 2 * T // 3, 0)):
        rows[b, :n] = -1
    rows[4, T // 2:] = -1                         # and behind
    out = k.check(rows=[0, 1, T - 1, 2 * T - 2, 2 * T - 1, 2 * T, 3 * T - 1, 3 * T + 2 * T // 3 - 1, 3 * T + 2 * T // 3,
                        4 * T - 1, 4 * T, 4 * T + T // 2 - 1, 4 * T + T // 2, 5 * T - 1])
    assert not out[torch.from_numpy(k.row_seq < 0).to(DEV)].any()


def test_padding_costs_no_more_than_rows():
    """A chunk that is padding throughout, or nearly so, beside one that is not: no slower than two that are not."""
    k = Case(2, 4096, 8, 4, 64, [10, 20], 0, seed=46)
    full = i32(k.row_seq)
    slot, ctx, out = i32(k.row_slot), i32(k.ctx), torch.empty_like(k.q)
    scratch = api.attention_kv8_scratch(k.c, 8192, 8, 4096)

    def best(row_seq):
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                api.attention_kv8(k.q, k.c, row_seq, slot, ctx, 4096, 0, out=out, scratch=scratch)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    for n in (4096, 4095):
        padded = full.clone()
        padded[:n] = -1
        assert best(padded) < 1.3 * best(full), n


@pytest.mark.parametrize("qscale", [1e6, 1e12, 1e25])
@pytest.mark.parametrize("T,d,P", [(1, 64, 0), (12, 64, 0), (1, 128, 0), (12, 128, 0), (1, 128, 20), (12, 128, 20)])
def test_scores_of_any_size(T, d, P, qscale):
    """Scores so large that a row is its best key's value, far past where fp32 holds a score and an exponent apart. Rows
    whose two best scores are closer than 2^-10 of the largest one's terms are left out: d + 8 fp32 roundings of 2^-24 and
    q's 2^-17 (twice: both keys) are less."""
    k = Case(3, T, 16, 4, d, [1, 40, 300], 1, 16, P, seed=47, qscale=qscale)
    out = k.run().double().cpu().numpy()
    assert int(k.err) == 0 and np.isfinite(out).all()
    q, some = k.q.double().cpu().numpy(), 0
    for r in range(3 * T):
        b = r // T
        see = np.concatenate([np.ones(k.ctx[b], bool), k.trees[r]])
        at = np.nonzero(see)[0]
        for h in range(16):
            K, V = k.K[b, at, h // 4], k.V[b, at, h // 4]
            if P:
                K = np.concatenate([k.pk[h // 4].double().cpu().numpy(), K])
                V = np.concatenate([k.pv[h // 4].double().cpu().numpy(), V])
            s = K @ q[r, h]
            order = np.argsort(s)
            if len(s) > 1 and s[order[-1]] - s[order[-2]] < 2.0 ** -10 * np.max(np.abs(K) @ np.abs(q[r, h])):
                continue
            v = V[order[-1]]
            some += 1
            assert np.all(np.abs(out[r, h] - v) <= (2.0 ** -8 + 2.0 ** -8 * (P > 0) + 2.0 ** -11 + 2.0 ** -20) * np.abs(v))
    assert some > 10 * T


def test_small_entries_of_a_query():
    """A query whose scores come from entries 2^-31 of its largest one (that one meets zeros in every key): each entry is
    within 2^-38 of the largest, so a score within sum_i |k_i| * 2^-38 * max|q| * scale; entries of 2^-30 and more are exact."""
    for low, exact in ((2.0 ** -30, True), (2.0 ** -33, False)):
        k = Case(2, 1, 4, 1, 64, [50, 90], 0, seed=48, qscale=1.0)
        q = low * (1 + k.g.integers(0, 128, size=(2, 4, 64)) / 128)
        q[:, :, 0] = 1.0
        k.q.copy_(torch.from_numpy(q).to(torch.bfloat16))
        assert np.array_equal(k.q.double().cpu().numpy(), q)
        n = k.K.shape[1]
        K = k.g.normal(size=(2, n, 1, 64)) / low / 4
        K[..., 0] = 0
        for b in range(2):
            m = k.ctx[b] + 1
            x = torch.from_numpy(K[b, :m]).float().to(DEV)
            v = torch.from_numpy(k.v[b, :m]).float().to(DEV)
            api.kv8_write(k.c, x, v, i32([b] * m), i32(np.arange(m)))
        k.K = O.dequantise(*O.quantise(K.astype(np.float32).astype(np.float64)))
        out = k.run().double().cpu().numpy()
        want, tol = k.want()
        if not exact:
            for r in range(2):
                m = k.ctx[r] + 1
                reach = np.abs(k.K[r, :m, 0]).sum(-1).max() * 2.0 ** -38 * 64 ** -0.5
                tol[r] += 2 * reach * np.abs(k.V[r, :m]).max()
        assert np.all(np.abs(out - want) <= tol)
