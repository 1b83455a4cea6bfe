"""CPU checks of the operators around a prompt: what the C ABI and the binding refuse before any launch, and the host's
frequency tables."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from eagle_speculative_decoding_cycle_gb300 import _lib as L
from eagle_speculative_decoding_cycle_gb300 import api
from oracle import prompt as O

FAKE = 1 << 20      # 16-byte aligned, never dereferenced: every call here returns on the host
BIG = 1 << 30       # another buffer, far enough behind the first


@pytest.fixture(scope="module")
def lib():
    from eagle_speculative_decoding_cycle_gb300 import build
    build.build()
    return L.lib()


# ---- rotary positions -------------------------------------------------------------------------------
RULES = [None, dict(kind="linear", factor=4.0), dict(kind="ntk", factor=2.5),
         dict(kind="llama3", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original=8192),
         dict(kind="yarn", factor=16.0, original=4096, beta_fast=32.0, beta_slow=1.0),
         dict(kind="yarn", factor=40.0, original=4096), dict(kind="yarn", factor=4.0, original=100, attention=1.5)]


@pytest.mark.parametrize("rot,theta", [(128, 5e5), (64, 1e4), (16, 1e4), (96, 1e6), (256, 1e4)])
@pytest.mark.parametrize("rule", RULES, ids=str)
def test_frequencies_and_turns(lib, rot, theta, rule):
    plan = api.Rope(256, theta=theta, rot=rot, scaling=rule, device="cpu")
    want, factor = O.frequencies(rot, theta, rule)
    assert np.allclose(plan.freq, want, rtol=1e-13, atol=0) and math.isclose(plan.factor, factor, rel_tol=1e-7)
    for f, t in zip(plan.freq, plan.turns.tolist()):
        t &= (1 << 64) - 1
        exact = f / (2 * math.pi) * 2.0 ** 64
        assert abs(t - exact) <= exact * 2.0 ** -50 + 1
        # a far position's fraction of a turn, in whole numbers
        p = 2 ** 31 - 1
        part = (p * t) % (1 << 64) / 2.0 ** 64
        back = math.remainder(p * f / (2 * math.pi) - part, 1.0)
        assert abs(back) <= p * (f * 2.0 ** -50 + 2.0 ** -64)      # the angle's doubles; the table's unit, once a position


def test_turns_of_any_angle(lib):
    f = [0.0, -1.0, 2 * math.pi, 7.0, -1e-30, 1e9]
    t = (C.c_uint64 * 6)()
    assert lib.eagle_rope_turns(6, (C.c_double * 6)(*f), t) == L.EAGLE_OK
    assert t[0] == 0 and t[2] == 0 and t[4] in (0, 2 ** 64 - 1)
    assert abs(t[1] / 2.0 ** 64 - (1 - 1 / (2 * math.pi))) < 1e-15 and abs(t[3] / 2.0 ** 64 - (7 / (2 * math.pi) - 1)) < 1e-15
    for bad in (float("nan"), float("inf"), 1e300):
        assert lib.eagle_rope_turns(1, (C.c_double * 1)(bad), t) == L.EAGLE_EINVAL
    assert lib.eagle_rope_turns(0, (C.c_double * 1)(1), t) == L.EAGLE_EINVAL
    assert lib.eagle_rope_turns(1, None, t) == L.EAGLE_EINVAL


def test_frequencies_refuse(lib):
    f, m = (C.c_double * 128)(), C.c_float()

    def call(rot=64, theta=1e4, f=f, m=C.byref(m), **s):
        return lib.eagle_rope_frequencies(rot, theta, C.byref(L.RopeScaling(**s)) if s else None, f, m)

    assert call() == L.EAGLE_OK
    for kw in (dict(rot=0), dict(rot=63), dict(rot=-2), dict(theta=1.0), dict(theta=float("nan")), dict(theta=float("inf")),
               dict(f=None), dict(m=None), dict(kind=5), dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=1, factor=float("nan")),
               dict(kind=3, factor=8.0, low=1.0, high=4.0), dict(kind=3, factor=8.0, original=100.0, low=4.0, high=4.0),
               dict(kind=4, factor=8.0, original=100.0, low=0.0, high=4.0), dict(kind=4, factor=8.0, original=100.0, low=2.0, high=1.0),
               dict(rot=2, kind=2, factor=2.0)):
        assert call(**kw) == L.EAGLE_EINVAL, kw
    for bad in (dict(kind="other", factor=2.0), dict(factor=2.0), dict(kind="llama3", factor=2.0, original=10),
                dict(kind="linear"), dict(kind="yarn", factor=2.0), dict(kind="linear", factor=2.0, beta=1)):
        with pytest.raises(ValueError):
            api.Rope(64, scaling=bad, device="cpu")
    for bad in (dict(rot=0), dict(rot=7), dict(freq=[1.0] * 3), dict(freq=[1.0] * 32, scaling=dict(kind="linear", factor=2.0))):
        with pytest.raises(ValueError):
            api.Rope(64, device="cpu", **bad)


def rope(lib, ti=1, to=1, q=FAKE, ldq=1024, qo=BIG, ldqo=1024, nq=8, k=2 * BIG, ldk=256, ko=3 * BIG, ldko=256, nkv=2, d=128,
         rot=128, R=5, pos=FAKE, turns=FAKE, factor=1.0):
    return lib.eagle_op_rope(None, ti, to, q, ldq, qo, ldqo, nq, k, ldk, ko, ldko, nkv, d, rot, 0, R, pos, turns, factor, 0)


def test_rope_refuses(lib):
    for kw in (dict(ti=2), dict(to=-1), dict(q=None), dict(q=FAKE + 8), dict(qo=None), dict(qo=BIG + 2), dict(k=None),
               dict(ko=3 * BIG + 4), dict(ldq=1016), dict(ldq=1028), dict(ldqo=1000), dict(ldk=128), dict(ldko=250), dict(nq=-1),
               dict(nkv=-1), dict(nq=0, nkv=0), dict(d=8), dict(d=72, rot=64), dict(d=272), dict(rot=0), dict(rot=8),
               dict(rot=144), dict(rot=40), dict(R=-1), dict(pos=None), dict(turns=None), dict(factor=float("nan")),
               dict(ti=0, ldq=1026), dict(to=0, ldqo=1026), dict(ldq=1 << 50)):
        assert rope(lib, **kw) == L.EAGLE_EINVAL, kw
    assert rope(lib, R=0, q=None, pos=None) == L.EAGLE_OK
    # outputs over inputs in any other way than the rows that they come from
    for kw in (dict(qo=FAKE + 256), dict(qo=FAKE, ldqo=1032), dict(qo=FAKE, to=0), dict(qo=2 * BIG), dict(ko=BIG),
               dict(ko=BIG + 4096), dict(ko=FAKE), dict(qo=FAKE + 2048), dict(k=FAKE + 2048, ldk=1024, ldq=1024, ko=FAKE + 2048)):
        assert rope(lib, **kw) == L.EAGLE_EINVAL, kw


def prompt(lib, q=FAKE, ldq=1024, k=BIG, ldk=256, v=2 * BIG, ldv=256, out=3 * BIG, ldo=1024, lse=None, R=9, Rk=9, nq=8, nkv=2,
           d=128, B=2, qs=FAKE, ks=FAKE, work=None, nb=0):
    return lib.eagle_op_attention_prompt(None, q, ldq, k, ldk, v, ldv, out, ldo, lse, R, Rk, nq, nkv, d, B, qs, ks, 0.0, work, nb,
                                         None)


def test_prompt_attention_refuses(lib):
    for kw in (dict(q=None), dict(q=FAKE + 8), dict(k=None), dict(k=BIG + 2), dict(v=None), dict(v=2 * BIG + 4), dict(out=None),
               dict(out=3 * BIG + 8), dict(ldq=1016), dict(ldq=1028), dict(ldk=248), dict(ldk=260), dict(ldv=128), dict(ldo=1000),
               dict(ldo=1 << 40), dict(R=-1), dict(Rk=-1), dict(nq=7), dict(nq=0), dict(nkv=0), dict(nq=130, ldq=1 << 15, ldo=1 << 15),
               dict(d=96), dict(d=256), dict(B=-1), dict(qs=None), dict(ks=None),
               dict(out=FAKE), dict(out=FAKE + 1024), dict(out=BIG), dict(out=2 * BIG - 2048), dict(work=FAKE + 8, nb=1 << 30)):
        assert prompt(lib, **kw) == L.EAGLE_EINVAL, kw
    for at in (FAKE + 1024, BIG + 512, 2 * BIG - 64, 3 * BIG):      # sums or scratch memory in the way
        assert prompt(lib, lse=at) == L.EAGLE_EINVAL and prompt(lib, work=at, nb=4096) == L.EAGLE_EINVAL, at
    assert prompt(lib, lse=5 * BIG, work=5 * BIG + 256, nb=64) == L.EAGLE_EINVAL
    assert prompt(lib, Rk=(1 << 27) + 1) == L.EAGLE_ECAPACITY and prompt(lib, B=(1 << 20) + 1) == L.EAGLE_ECAPACITY
    assert prompt(lib, R=1 << 30, ldq=1024) == L.EAGLE_ECAPACITY and prompt(lib, Rk=2 ** 31 - 100) == L.EAGLE_ECAPACITY
    assert prompt(lib, R=0, q=None, out=None) == L.EAGLE_OK and prompt(lib, B=0) == L.EAGLE_OK


def test_binding_refuses_rows(lib):
    x = torch.zeros(4, 6, 128, dtype=torch.bfloat16)
    s = torch.tensor([0, 4], dtype=torch.int32)
    plan = api.Rope(128, device="cpu")
    with pytest.raises(ValueError):
        api.attention_prompt(x, x[:, :2], x[:, 2:4], s)                       # the CPU's tensors
    with pytest.raises(ValueError):
        api.rope(plan, x, None, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        api.rope(plan, x.half(), None, torch.zeros(4, dtype=torch.int32))


# ---- blocks and paths ---------------------------------------------------------------------------------
def layers(n=2, **kw):
    f = dict(k_code=FAKE, v_code=FAKE, k_exp=FAKE, v_exp=FAKE, table=FAKE, n_kv_heads=2, head_dim=64, max_batch=4, cap=64,
             block=16, n_blocks=20)
    f.update(kw)
    return (L.KV8 * n)(*[L.KV8(**f) for _ in range(n)])


def resize(lib, c, n=2, B=4, refs=FAKE, parent=None, length=FAKE, scratch=FAKE, nb=1 << 30):
    return lib.eagle_op_kv8_resize(None, c, n, B, refs, parent, length, scratch, nb, None)


def compact(lib, c, n=2, B=4, n_old=FAKE, acc=FAKE, path=FAKE, deep=5):
    return lib.eagle_op_kv8_compact(None, c, n, B, n_old, acc, path, deep, None)


def test_block_calls_refuse(lib):
    for bad in (dict(k_code=None), dict(head_dim=96), dict(cap=40), dict(block=8), dict(n_blocks=0), dict(v_exp=FAKE + 1)):
        assert resize(lib, layers(**bad)) == L.EAGLE_EINVAL and compact(lib, layers(**bad)) == L.EAGLE_EINVAL, bad
        assert lib.eagle_op_kv8_resize_scratch_bytes(layers(**bad)) == 0
    flat = layers(table=None, block=0, n_blocks=0)
    assert resize(lib, flat) == L.EAGLE_EINVAL and lib.eagle_op_kv8_resize_scratch_bytes(flat) == 0
    for name, value in (("table", 2 * FAKE), ("n_blocks", 21), ("head_dim", 128), ("cap", 80), ("max_batch", 5), ("n_kv_heads", 3)):
        c = layers()
        setattr(c[1], name, value)
        assert resize(lib, c) == L.EAGLE_EINVAL and compact(lib, c) == L.EAGLE_EINVAL, name
    assert resize(lib, None) == L.EAGLE_EINVAL and compact(lib, None) == L.EAGLE_EINVAL
    for kw in (dict(n=0), dict(n=-1), dict(B=5), dict(B=-1), dict(refs=None), dict(length=None)):
        assert resize(lib, layers(), **kw) == L.EAGLE_EINVAL, kw
    need = lib.eagle_op_kv8_resize_scratch_bytes(layers())
    assert need > 0
    for kw in (dict(scratch=None), dict(scratch=FAKE + 8), dict(nb=need - 1)):
        assert resize(lib, layers(), **kw) == L.EAGLE_ECAPACITY, kw
    for kw in (dict(n=0), dict(B=5), dict(B=-1), dict(n_old=None), dict(acc=None), dict(path=None), dict(deep=0), dict(deep=17)):
        assert compact(lib, layers(), **kw) == L.EAGLE_EINVAL, kw
    assert resize(lib, layers(), B=0, refs=None) == L.EAGLE_OK and compact(lib, layers(), B=0, n_old=None) == L.EAGLE_OK


def test_binding_refuses_layers(lib):
    def cache(table=None, B=2):
        shape = (B, 3, 32, 64)
        z = lambda s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
        return api.KV8Cache(z(shape), z(shape), z(shape[:3]), z(shape[:3]), table)

    t, u = (torch.full((4, 2), -1, dtype=torch.int32) for _ in range(2))
    for bad in ([], [cache(), cache(B=3)], [cache(t), cache(u)], [cache(), cache(t)]):
        with pytest.raises(ValueError):
            api.KV8Layers(bad)
    with pytest.raises(ValueError):
        api.KV8Layers([cache()], refs=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        api.KV8Layers([cache(t)], refs=torch.zeros(3, dtype=torch.int32))
    flat, paged = api.KV8Layers([cache()]), api.KV8Layers([cache(t)])
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.kv8_resize(flat, n)
    for bad in (n.long(), n.view(1, 2), torch.zeros(5, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)[::4]):
        with pytest.raises(ValueError):
            api.kv8_resize(paged, bad)
    with pytest.raises(ValueError):
        api.kv8_fork(paged, torch.zeros(3, dtype=torch.int32), n)
    with pytest.raises(ValueError):
        api.kv8_resize(paged, n)                                # the CPU's tensors
    for path in (torch.zeros(2, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(2, 2)):
        with pytest.raises(ValueError):
            api.kv8_compact(paged, n, n, path)


@pytest.mark.parametrize("kind,own", [("linear", {}), ("ntk", {}), ("llama3", dict(low_freq_factor=1.0, high_freq_factor=4.0, original=8192)),
                                      ("yarn", dict(original=4096, beta_fast=32.0, beta_slow=1.0, attention=1.25))])
@pytest.mark.parametrize("name", ["original", "attention", "low_freq_factor", "high_freq_factor", "beta_fast", "beta_slow"])
def test_entries_of_another_rule_are_refused(lib, kind, own, name):
    """A rule takes its own entries and no other rule's: what would be without effect is not taken in silence."""
    rule = dict(kind=kind, factor=4.0, **own)
    api.Rope(64, scaling=rule, device="cpu")
    if name not in own:
        with pytest.raises(ValueError):
            api.Rope(64, scaling={**rule, name: 2.0}, device="cpu")


def test_layers_that_share_memory_are_refused(lib):
    """Given twice, a layer's accepted paths would be moved twice, the second time from what the first one wrote."""
    t = torch.full((2, 2), -1, dtype=torch.int32)
    pool = [torch.zeros(2 * 64 * 48 * 2 * 16, dtype=torch.uint8) for _ in range(2)]
    codes = lambda p, at: p[at:at + 3 * 2 * 16 * 64].view(3, 2, 16, 64)  # noqa: E731
    exps = lambda: torch.zeros(3, 2, 16, dtype=torch.uint8)  # noqa: E731
    one = api.KV8Cache(codes(pool[0], 0), codes(pool[1], 0), exps(), exps(), t)
    beside = api.KV8Cache(codes(pool[0], 6144), codes(pool[1], 6144), exps(), exps(), t)
    assert api.KV8Layers([beside, one]).n == 2
    for bad in ([one, one], [beside, one, beside], [one, api.KV8Cache(codes(pool[0], 4096), codes(pool[1], 6144), exps(), exps(), t)],
                [one, api.KV8Cache(codes(pool[0], 6144), codes(pool[1], 6144), exps(), one.v_exp, t)],
                [api.KV8Cache(one.k, one.k, exps(), exps(), t)]):
        with pytest.raises(ValueError):
            api.KV8Layers(bad)


def test_tables_of_too_many_entries_are_refused(lib):
    """Missing entries are counted in 32 bits: a count that passed them would have assigned nothing and said nothing."""
    wide = 2 ** 31 - 16      # slots of a sequence: 2^27 - 1 blocks of 16
    for most, cap, fits in ((16, wide, True), (17, wide, False), (2 ** 27, 16 * 16, False), (2 ** 27 - 1, 16 * 16, True), (2 ** 20, wide, False)):
        c = layers(max_batch=most, cap=cap)
        assert (lib.eagle_op_kv8_resize_scratch_bytes(c) > 0) == fits, (most, cap)
        if not fits:
            assert resize(lib, c, nb=1 << 60) == L.EAGLE_ECAPACITY
