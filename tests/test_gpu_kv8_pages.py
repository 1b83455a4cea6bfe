"""Blocks of a paged 8-bit cache and accepted paths in all layers, on the GPU: every result is whole numbers or copied bytes,
compared for equality with the restatement in oracle.prompt."""
import numpy as np
import pytest
import torch

from eagle_speculative_decoding_cycle_gb300 import api
from oracle import kv8 as K8
from oracle import prompt as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).to(DEV)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


class Pool:
    """Layers over one table with their restatement on the host."""

    def __init__(self, B, W, n_blocks, layers=2, nkv=3, d=64, block=16, seed=0):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.B, self.W, self.n, self.block = B, W, n_blocks, block
        shape = (layers, n_blocks, nkv, block, d)
        new = lambda s: torch.randint(0, 255, s, generator=self.g, device=DEV, dtype=torch.uint8)  # noqa: E731
        self.arrays = [new(shape), new(shape), new(shape[:4]), new(shape[:4])]
        self.table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
        self.layers = api.KV8Layers([api.KV8Cache(*x, self.table) for x in zip(*self.arrays)])
        self.t, self.r = [[-1] * W for _ in range(B)], [0] * n_blocks
        self.want = [x.clone() for x in self.arrays]

    def scribble(self):
        """Other contents everywhere, so that copies show."""
        for x, w in zip(self.arrays, self.want):
            x.copy_(torch.randint(0, 255, x.shape, generator=self.g, device=DEV, dtype=torch.uint8))
            w.copy_(x)

    def step(self, length, parent=None, code=0):
        err = err_word()
        if parent is None:
            api.kv8_resize(self.layers, i32(length), err=err)
        else:
            api.kv8_fork(self.layers, i32(parent), i32(length), err=err)
        copies, short = O.resize(self.t, self.r, [int(x) for x in length], self.block,
                                 None if parent is None else [int(x) for x in parent])
        for src, dst, n in copies:
            for w in self.want:
                w[:, dst, :, :n] = w[:, src, :, :n]
        assert int(err) == (3 if short else code)
        self.same()
        return copies

    def same(self):
        assert self.table.tolist() == self.t and self.layers.refs.tolist() == self.r
        for x, w in zip(self.arrays, self.want):
            assert torch.equal(x, w)


@pytest.mark.parametrize("B,W,n_blocks,layers,nkv,d,block", [(1, 1, 1, 1, 1, 64, 16), (7, 6, 30, 2, 3, 64, 16),
                                                             (70, 40, 2500, 1, 1, 64, 32), (5, 9, 50, 67, 2, 128, 16),
                                                             (40, 3, 60, 3, 5, 128, 256)])
def test_random_steps(B, W, n_blocks, layers, nkv, d, block):
    g = np.random.default_rng(B)
    p = Pool(B, W, n_blocks, layers, nkv, d, block, seed=B)
    seen = 0
    for step in range(24):
        length = g.integers(-1, W * block + 1, B)
        if step % 2:
            length = np.where(g.random(B) < 0.5, -1, length // 2)
        parent = None
        if step % 3 == 2:      # forks of the sequence with the most blocks, and of another one
            have = np.asarray([min([j for j, e in enumerate(t) if e < 0] + [W]) for t in p.t]) * block
            order = np.argsort(-have)
            parent = np.full(B, -1)
            for b in range(B):
                x = order[b % min(2, B)]
                if b in order[:2] or g.random() < 0.4:
                    continue
                parent[b], length[b] = x, g.integers(0, have[x] + 1)
            length[order[:2]] = -1
        p.scribble()
        seen += len(p.step(length, parent))
    assert B == 1 or seen > 0
    p.step(np.zeros(B))
    assert not any(p.r) and (p.table == -1).all()


def test_a_shared_last_block_is_copied_when_a_sequence_steps_back():
    p = Pool(3, 8, 20)
    p.step([100, -1, -1])
    p.step([-1, 100, 96], [-1, 0, 0])       # 100: the seventh block copied; 96: six whole blocks shared
    assert len(p.step([-1, 50, -1])) == 1   # back into a shared block: a copy of its first two slots
    assert len(p.step([40, -1, -1])) == 1   # the parent too
    assert len(p.step([-1, -1, 33])) == 1   # the third block: sequence 1, at 50, still holds it
    assert len(p.step([-1, 35, -1])) == 0   # and now alone
    p.step([0, 0, 0])


def test_all_holders_step_back_at_once():
    p = Pool(4, 4, 12)
    p.step([64, -1, -1, -1])
    p.step([-1, 64, 64, 64], [-1, 0, 0, 0])
    assert len(p.step([40, 41, 42, 43])) == 4      # each gets a copy, the block itself is free afterwards
    p.step([64, 64, 64, 64])


def test_running_out_of_blocks():
    p = Pool(3, 4, 5)
    p.step([64, 16, 32])                # seven wanted, five there: the first ones of the order
    p.step([16, 16, 16])
    p.step([-1, 16, 10], [-1, 0, 0])    # two forks share the one block, the second of them is partly filled: copied
    p.step([0, 0, 0])
    p = Pool(2, 2, 1)
    p.step([10, -1])
    p.step([-1, 10], [-1, 0])           # no block for the copy: it stays shared, and the call says so
    assert p.layers.refs.tolist() == [2]


def test_refused_sequences_stay_as_they_were():
    p = Pool(4, 4, 16)
    p.step([64, 30, -1, -1])
    t, r = p.table.clone(), p.layers.refs.clone()
    for length, parent in (([-1, -1, 65, -1], None), ([-1, -1, 2 ** 30, -1], None),
                           ([-1, -1, 20, -1], [-1, -1, 4, -1]), ([-1, -1, 20, -1], [-1, -1, 2, -1]),
                           ([20, -1, 20, -1], [-1, -1, 0, -1]),        # its parent takes part
                           ([-1, -1, 40, -1], [-1, -1, 1, -1]),        # its parent has fewer slots
                           ([-1, -1, 20, 20], [-1, -1, 3, 2])):        # two forks of each other
        err = err_word()
        if parent is None:
            api.kv8_resize(p.layers, i32(length), err=err)
        else:
            api.kv8_fork(p.layers, i32(parent), i32(length), err=err)
        assert int(err) == 2, (length, parent)
        assert torch.equal(p.table[1:], t[1:])
        if length[0] < 0:
            assert torch.equal(p.table, t) and torch.equal(p.layers.refs, r)
        else:
            assert p.table[0].tolist() == t[0].tolist()[:2] + [-1, -1]
            api.kv8_resize(p.layers, i32([64, -1, -1, -1]))
            t, r = p.table.clone(), p.layers.refs.clone()


def test_entries_outside_the_pool_and_wrong_counts():
    p = Pool(2, 3, 6)
    p.step([48, 20])
    p.table[0, 2] = 99
    err = err_word()
    api.kv8_resize(p.layers, i32([10, -1]), err=err)
    assert int(err) == 2 and p.table[0].tolist()[1:] == [-1, -1]
    p.layers.refs[int(p.table[1, 1])] = 0       # a count that misses an entry
    err = err_word()
    api.kv8_resize(p.layers, i32([-1, 0]), err=err)
    assert int(err) == 2 and p.table[1].tolist() == [-1] * 3 and int(p.layers.refs.min()) == 0


def test_fewer_sequences_than_the_table_and_a_parent_behind_them():
    p = Pool(5, 4, 30)
    p.step([20, 20, 20, 20, 50])
    api.kv8_fork(p.layers, i32([4, -1]), i32([40, -1]))
    O.resize(p.t, p.r, [40, -1, -1, -1, -1], 16, [4, -1, -1, -1, -1])
    assert p.table.tolist() == p.t and p.layers.refs.tolist() == p.r
    api.kv8_resize(p.layers, i32([]))
    assert p.table.tolist() == p.t


def test_counts_from_the_table():
    p = Pool(3, 4, 10)
    p.table.copy_(i32([[3, 1, -1, -1], [3, 2, 9, -1], [-1, -1, -1, -1]]))
    l = api.KV8Layers(p.layers.caches)
    assert l.refs.tolist() == [0, 1, 1, 2, 0, 0, 0, 0, 0, 1]


def test_large_pools():
    """More blocks than one pass of the search, free ones far behind, long rows."""
    B, W, n = 130, 500, 90000
    p = Pool(B, W, n, layers=1, nkv=1, d=64, block=16)
    g = np.random.default_rng(5)
    for _ in range(4):
        p.step(g.integers(-1, W * 16 + 1, B))
    p.step(np.where(np.arange(B) % 2 == 0, 0, -1))
    p.step(np.full(B, W * 16))


def test_graphs_and_a_side_stream():
    """A captured cycle of calls (slots for a tree, then only the accepted ones kept) follows the lengths it reads."""
    p = Pool(6, 20, 100)
    length, kept = i32([0] * 6), i32([0] * 6)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        api.kv8_resize(p.layers, length)
        api.kv8_resize(p.layers, kept)
    rng = np.random.default_rng(6)
    ctx = rng.integers(0, 100, 6)
    for _ in range(8):
        took = rng.integers(1, 10, 6)
        length.copy_(i32(ctx + 17)), kept.copy_(i32(ctx + took))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        O.resize(p.t, p.r, (ctx + 17).tolist(), 16)
        O.resize(p.t, p.r, (ctx + took).tolist(), 16)
        p.same()
        ctx = ctx + took
    api.kv8_resize(p.layers, i32(ctx + 3), stream=side)
    side.synchronize()
    O.resize(p.t, p.r, (ctx + 3).tolist(), 16)
    p.same()


# ---- accepted paths ---------------------------------------------------------------------------------
def contiguous(B, layers, nkv, d, cap, g):
    shape = (layers, B, nkv, cap, d)
    new = lambda s: torch.randint(0, 255, s, generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
    arrays = [new(shape), new(shape), new(shape[:4]), new(shape[:4])]
    return arrays, api.KV8Layers([api.KV8Cache(*x) for x in zip(*arrays)])


@pytest.mark.parametrize("B,layers,nkv,d,block,deep", [(1, 1, 1, 64, 0, 1), (3, 2, 3, 128, 16, 5), (5, 40, 2, 64, 32, 8),
                                                       (2, 70, 1, 128, 0, 16), (64, 3, 8, 128, 16, 6), (1, 2, 40, 128, 0, 9)])
def test_compaction_moves_paths_at_once(B, layers, nkv, d, block, deep):
    g = torch.Generator(device=DEV).manual_seed(deep)
    rng = np.random.default_rng(deep)
    cap = 160
    if block:
        p = Pool(B, cap // block, B * (cap // block) + 3, layers, nkv, d, block, seed=1)
        p.step([cap] * B)
        p.table.copy_(p.table[:, torch.randperm(cap // block)])
        arrays, ls, table = p.arrays, p.layers, p.table.tolist()
    else:
        (arrays, ls), table = contiguous(B, layers, nkv, d, cap, g), None
    place = lambda b, s: (b, s) if table is None else (table[b][s // block], s % block)  # noqa: E731
    for kind in range(3):
        n_old = rng.integers(0, cap - 70, B)
        took = rng.integers(0, deep + 1, B)
        path = np.sort(np.stack([rng.permutation(np.arange(1, 61))[:deep] for _ in range(B)]), 1)
        if kind == 1:      # any order, sources that are other moves' places
            path = rng.integers(0, deep + 2, (B, deep))
        if kind == 2:
            took[:] = deep
        want = [x.clone() for x in arrays]
        for b in range(B):
            for x, w in zip(arrays, want):
                for j in range(1, took[b] + 1):
                    (db, ds), (sb, ss) = place(b, n_old[b] + j), place(b, n_old[b] + path[b, j - 1])
                    w[:, db, :, ds] = x[:, sb, :, ss]
        err = err_word()
        api.kv8_compact(ls, i32(n_old), i32(took), i32(path), err=err)
        assert int(err) == 0
        for x, w in zip(arrays, want):
            assert torch.equal(x, w)


def test_compaction_leaves_out_what_is_out_of_range():
    p = Pool(3, 4, 20, layers=2)
    p.step([64, 64, 40])
    for n_old, took, path in (([60, -1, -1], [3, 0, 0], [[1, 2, 9]] * 3), ([-5, 0, 0], [2, 0, 0], [[1, 2, 3]] * 3),
                              ([0, 0, 46], [0, 0, 2], [[1, 3, 0]] * 3), ([0, 0, 0], [3, 0, 0], [[-7, 64, 2 ** 31 - 1]] * 3),
                              ([2 ** 31 - 1, 0, 0], [1, 0, 0], [[2 ** 31 - 1, 0, 0]] * 3)):
        before = [x.clone() for x in p.arrays]
        err = err_word()
        api.kv8_compact(p.layers, i32(n_old), i32(took), i32(path), err=err)
        assert int(err) == 2
        api.kv8_compact(p.layers, i32(n_old), i32(took), i32(path))      # without a status word
        b = int(np.argmax(took))
        ok = [j for j in range(1, took[b] + 1) if 0 <= n_old[b] and n_old[b] + j < 64 and 0 <= n_old[b] + path[b][j - 1] < 64 and
              p.t[b][(n_old[b] + j) // 16] >= 0 and p.t[b][(n_old[b] + path[b][j - 1]) // 16] >= 0]
        for x, w in zip(p.arrays, before):
            for j in ok:
                s, t = n_old[b] + path[b][j - 1], n_old[b] + j
                w[:, p.t[b][t // 16], :, t % 16] = x[:, p.t[b][s // 16], :, s % 16]
        # (twice the same move: sources of these cases are not places of others)
        for x, w in zip(p.arrays, before):
            assert torch.equal(x, w)
    err = err_word()
    api.kv8_compact(p.layers, i32([0, 0, 0]), i32([9, 0, 0]), i32([[1, 2, 3]] * 3), err=err)      # longer than its path: three moves
    assert int(err) == 2
    api.kv8_compact(p.layers, i32([0, 0, 0]), i32([-1, 0, -9]), i32([[1, 2, 3]] * 3), err=err_word())


def test_compaction_equals_reading_and_writing():
    """The same values as kv8_read and kv8_write of the accepted rows, layer by layer."""
    g = torch.Generator().manual_seed(4)
    caches = [api.KV8Cache.empty(2, 4, 96, 128, device=DEV) for _ in range(3)]
    for c in caches:
        x = torch.randn(2 * 90, 4, 128, generator=g).to(torch.bfloat16).to(DEV)
        api.kv8_write(c, x, 3 * x, i32(np.repeat([0, 1], 90)), i32(np.tile(np.arange(90), 2)))
    who, src, dst = i32([0, 0, 0, 1, 1]), i32([22, 25, 40, 51, 60]), i32([21, 22, 23, 51, 52])
    want = [api.kv8_read(c, who, src) for c in caches]
    api.kv8_compact(api.KV8Layers(caches), i32([20, 50]), i32([3, 2]), i32([[2, 5, 20], [1, 10, 0]]))
    for c, (k, v) in zip(caches, want):
        k2, v2 = api.kv8_read(c, who, dst)
        assert torch.equal(k, k2) and torch.equal(v, v2)


def test_a_run_from_prompts_to_cycles():
    """Prompts turned, attended and written, answers forked from them, verify passes over trees, accepted paths moved, blocks
    given back: every attention result against 64 bits over each sequence's own history."""
    rng = np.random.default_rng(20)
    nq, nkv, d, block, layers, T = 8, 2, 128, 16, 2, 7
    B, W = 6, 12
    table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    n = 40
    new = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    caches = [api.KV8Cache(new(n, nkv, block, d), new(n, nkv, block, d), new(n, nkv, block), new(n, nkv, block), table)
              for _ in range(layers)]
    ls = api.KV8Layers(caches)
    rope_rule = dict(kind="llama3", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original=64)
    plan = api.Rope(d, theta=5e5, scaling=rope_rule, device=DEV)
    freq, factor = O.frequencies(d, 5e5, rope_rule)
    deq = lambda t: K8.dequantise(*K8.quantise(t.double().cpu().numpy()))  # noqa: E731
    rows = lambda m: torch.from_numpy(rng.normal(size=(m, nq + 2 * nkv, d))).to(torch.float32).to(DEV)  # noqa: E731

    def turned(x, pos):
        q, k = api.rope(plan, x[:, :nq], x[:, nq:nq + nkv], i32(pos), dtype=torch.bfloat16)
        want = O.rotate(x[:, :nq + nkv].double().cpu().numpy(), np.asarray(pos), freq, factor, False)[0]
        both = torch.cat([q, k], 1).double().cpu().numpy()
        assert np.all(np.abs(both - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * (1 + np.abs(x[:, :nq + nkv].double().cpu().numpy()).max()))
        return q, k, x[:, nq + nkv:].to(torch.bfloat16)

    def close(got, q, K, V, see, weights):
        for h in range(nkv):
            at = slice(h * nq // nkv, (h + 1) * nq // nkv)
            o, Wt, A = K8.attend(q[at], K[:, h], V[:, h], np.repeat(see[None], nq // nkv, 0), d ** -0.5)
            tol = 2.0 ** -8 * np.abs(o) + Wt * (weights + 2 * (d + 8) * 2.0 ** -23 * A[:, None] + 2.0 ** -14 + 2.0 ** -15 * A[:, None])
            assert np.all(np.abs(got[at] - o) <= tol)

    # two prompts of 37 and 20 tokens
    lens = [37, 20]
    pos = np.concatenate([np.arange(m) for m in lens])
    start = i32([0, 37, 57])
    hist = [[[] for _ in range(B)] for _ in range(layers)]      # per layer and sequence: (k, v) rows as the cache holds them
    api.kv8_resize(ls, i32(lens + [0] * 4))
    for l, c in enumerate(caches):
        q, k, v = turned(rows(57), pos)
        out = api.attention_prompt(q, k, v, start).double().cpu().numpy()
        qd, kd, vd = (t.double().cpu().numpy() for t in (q, k, v))
        for r in range(57):
            b, i = (0, r) if r < 37 else (1, r - 37)
            keys = slice(0, i + 1) if b == 0 else slice(37, 37 + i + 1)
            close(out[r], qd[r], kd[keys], vd[keys], np.ones(i + 1, bool), 2.0 ** -8)
        api.kv8_write(c, k, v, i32([0] * 37 + [1] * 20), i32(pos))
        kq, vq = deq(k), deq(v)
        hist[l][0], hist[l][1] = list(zip(kq[:37], vq[:37])), list(zip(kq[37:], vq[37:]))
    # further answers to the prompts
    api.kv8_fork(ls, i32([-1, -1, 0, 0, 1, -1]), i32([-1, -1, 37, 32, 20, -1]))
    for l in range(layers):
        hist[l][2], hist[l][3], hist[l][4] = list(hist[l][0]), list(hist[l][0][:32]), list(hist[l][1])
    live = [0, 1, 2, 3, 4]
    for cycle in range(3):
        ctx = np.asarray([len(hist[0][b]) for b in range(B)])
        api.kv8_resize(ls, i32(np.where(np.isin(np.arange(B), live), ctx + T, -1)))
        trees = np.zeros((B, T, T), bool)
        for b in range(B):
            for i in range(T):
                if i:
                    trees[b, i] = trees[b, rng.integers(0, i)]
                trees[b, i, i] = True
        seq, slot = np.repeat(live, T), (ctx[live][:, None] + np.arange(T)).reshape(-1)
        depth = trees[live].sum(2).reshape(-1) - 1
        bits = np.zeros((len(live) * T, 1), np.uint64)
        for r, row in enumerate(trees[live].reshape(-1, T)):
            bits[r, 0] = sum(1 << int(t) for t in np.nonzero(row)[0])
        mask = torch.from_numpy(bits.view(np.int64)).to(DEV)
        leaf = {b: int(rng.integers(0, T)) for b in live}
        path = {b: list(np.nonzero(trees[b, leaf[b]])[0]) for b in live}
        for l, c in enumerate(caches):
            q, k, v = turned(rows(len(seq)), np.repeat(ctx[live], T) + depth)
            api.kv8_write(c, k, v, i32(seq), i32(slot))
            out = api.attention_kv8(q, c, i32(seq), None, i32(ctx), T, 1, T, mask).double().cpu().numpy()
            kq, vq, qd = deq(k), deq(v), q.double().cpu().numpy()
            for r, b in enumerate(seq):
                i, base = r % T, r - r % T
                hk = np.stack([x for x, _ in hist[l][b]] + [kq[base + a] for a in range(T)])
                hv = np.stack([y for _, y in hist[l][b]] + [vq[base + a] for a in range(T)])
                close(out[r], qd[r], hk, hv, np.concatenate([np.ones(ctx[b], bool), trees[b, i]]), 2.0 ** -11)
            for x, b in enumerate(live):
                hist[l][b] = hist[l][b] + [(kq[x * T + a], vq[x * T + a]) for a in path[b]]
        # row 0 of a tree sits at slot ctx and is always on the path: the others move behind it
        acc = np.asarray([len(path[b]) - 1 if b in live else 0 for b in range(B)])
        moves = np.zeros((B, T), np.int64)
        for b in live:
            moves[b, :acc[b]] = path[b][1:]
        api.kv8_compact(ls, i32(ctx), i32(acc), i32(moves))
        api.kv8_resize(ls, i32(np.where(np.isin(np.arange(B), live), ctx + acc + 1, -1)))
        if cycle == 1:      # one answer ends, its blocks are free for a new one
            api.kv8_resize(ls, i32([-1, -1, -1, 0, -1, -1]))
            live = [0, 1, 2, 4]
    flat = [e for t in table.tolist() for e in t if e >= 0]
    assert [flat.count(i) for i in range(n)] == ls.refs.tolist()


@pytest.mark.parametrize("length,at", [([48, 20], (0, 1)), ([40, 20], (0, 2)), ([40, 20], (0, 0)), ([33, 32], (1, 1)), ([48, -1], (1, 0)),
                                       ([16, 20], (0, 2))])
@pytest.mark.parametrize("entry", [12, 99, 2 ** 31 - 1])
def test_an_entry_outside_the_pool_among_those_that_stay(length, at, entry):
    """It is latched and counts as missing: its slots get a block. (A sequence that takes no part keeps it, unnoticed.)"""
    p = Pool(2, 3, 12)
    p.step([48, 32])
    p.table[at] = entry
    takes_part = length[at[0]] >= 0
    p.t[at[0]][at[1]] = -1 if takes_part else entry
    p.step(length, code=2 if takes_part else 0)
    p.step([48, 48] if takes_part else [48, -1])


def test_an_entry_outside_the_pool_at_a_shared_end():
    """The last entry, partly filled, of a fork that steps back: nothing is copied from it, and its block is a new one."""
    p = Pool(3, 3, 12)
    p.step([48, -1, -1])
    p.step([-1, 48, 48], [-1, 0, 0])
    p.table[1, 1] = 12
    p.t[1][1] = -1
    assert p.step([-1, 20, -1], code=2) == []
    assert len(p.step([-1, -1, 20])) == 1


@pytest.mark.parametrize("B", [2047, 2048, 2049, 5000])
def test_thousands_of_sequences(B):
    """Both sides of what the plan hands on in shared memory: forks, steps back into shared blocks, too few blocks, bad entries."""
    g = np.random.default_rng(B)
    p = Pool(B, 3, 3 * B, layers=2, nkv=1, d=64, block=16, seed=B)
    p.step(g.integers(0, 49, B))
    copies = 0
    for _ in range(3):
        have = np.asarray([sum(e >= 0 for e in t) for t in p.t]) * 16
        forks = g.random(B) < 0.4
        forks[-1] = True
        parent = np.where(forks, g.choice(np.flatnonzero(~forks), B), -1)
        length = np.where(forks, g.integers(0, 49, B) % (have[parent] + 1), -1)
        p.scribble()
        copies += len(p.step(length, parent))
        p.scribble()
        copies += len(p.step(np.where(g.random(B) < 0.5, g.integers(0, 49, B), -1)))
    assert copies > B // 4
    p.table[B - 1, 0] = 3 * B
    p.t[B - 1][0] = -1
    p.step(np.full(B, 40), code=2)
    p.step(np.zeros(B))


def test_captured_forks_and_moves():
    """A captured fork, moves in all layers and resize, replayed for other parents, lengths and paths."""
    p = Pool(5, 6, 40, layers=3)
    p.step([60, 40, -1, -1, -1])
    parent, length, kept = i32([-1] * 5), i32([-1] * 5), i32([-1] * 5)
    n_old, took, path = i32([0] * 5), i32([0] * 5), i32(np.zeros((5, 4)))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        api.kv8_fork(p.layers, parent, length)
        api.kv8_compact(p.layers, n_old, took, path)
        api.kv8_resize(p.layers, kept)
    p.same()
    for par, n, moves in (([-1, -1, 0, 0, 1], [-1, -1, 60, 33, 40], {2: [50, 3, 8], 3: [20], 4: [30, 7]}),
                          ([-1, -1, 1, -1, -1], [-1, -1, 17, 96, 50], {0: [5, 4], 2: [10], 3: [60, 70, 80, 90]})):
        # places inside a sequence's last block, which is its own (sequence 0: a block that nobody holds any more)
        at = [40 if b == 0 else 0 if m < 0 else max((m - 1) // 16 * 16, m - 5) for b, m in enumerate(n)]
        paths = np.zeros((5, 4), dtype=int)
        count = [0] * 5
        for b, slots in moves.items():
            paths[b, :len(slots)] = [s - at[b] for s in slots]
            count[b] = len(slots)
        keep = [-1 if b < 2 else at[b] + count[b] + 1 for b in range(5)]
        for t, x in ((parent, par), (length, n), (kept, keep), (n_old, at), (took, count), (path, paths)):
            t.copy_(i32(x))
        p.scribble()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        place = lambda b, s: (p.t[b][s // 16], s % 16)  # noqa: E731
        copies = [O.resize(p.t, p.r, n, 16, par)[0]]
        for src, dst, m in copies[0]:
            for w in p.want:
                w[:, dst, :, :m] = w[:, src, :, :m]
        for w in p.want:
            old = w.clone()
            for b in range(5):
                for j in range(1, count[b] + 1):
                    (db, ds), (sb, ss) = place(b, at[b] + j), place(b, at[b] + paths[b, j - 1])
                    w[:, db, :, ds] = old[:, sb, :, ss]
        for src, dst, m in O.resize(p.t, p.r, keep, 16)[0]:
            for w in p.want:
                w[:, dst, :, :m] = w[:, src, :, :m]
        p.same()
