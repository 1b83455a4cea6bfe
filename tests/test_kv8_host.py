"""CPU checks of the 8-bit cache entry points: what the C ABI and the binding refuse before any launch."""
import ctypes as C

import pytest
import torch

from eagle_speculative_decoding_cycle_gb300 import _lib as L
from eagle_speculative_decoding_cycle_gb300 import api

FAKE = 4096   # 16-byte aligned, never dereferenced: every call here returns on the host


@pytest.fixture(scope="module")
def lib():
    from eagle_speculative_decoding_cycle_gb300 import build
    build.build()
    return L.lib()


def cache(**kw):
    f = dict(k_code=FAKE, v_code=FAKE, k_exp=FAKE, v_exp=FAKE, table=None, n_kv_heads=8, head_dim=128, max_batch=4,
             cap=256, block=0, n_blocks=0)
    f.update(kw)
    return C.byref(L.KV8(**f))


BAD_CACHES = [dict(k_code=None), dict(v_exp=None), dict(k_code=FAKE + 8), dict(k_exp=FAKE + 4), dict(n_kv_heads=0),
              dict(head_dim=96), dict(head_dim=256), dict(max_batch=0), dict(cap=0), dict(cap=250),
              dict(table=FAKE, block=8, n_blocks=9), dict(table=FAKE, block=24, n_blocks=9),
              dict(table=FAKE, block=512, cap=512, n_blocks=9), dict(table=FAKE, block=16, n_blocks=0),
              dict(table=FAKE, block=64, cap=272, n_blocks=9)]


def rows(lib, fn, c, dtype=1, k=FAKE, ldk=1024, v=FAKE, ldv=1024, R=3, seq=FAKE, slot=FAKE):
    return getattr(lib, fn)(None, c, dtype, k, ldk, v, ldv, R, seq, slot, None)


@pytest.mark.parametrize("fn", ["eagle_op_kv8_write", "eagle_op_kv8_read"])
def test_row_calls_refuse(lib, fn):
    assert getattr(lib, fn)(None, None, 1, FAKE, 1024, FAKE, 1024, 3, FAKE, FAKE, None) == L.EAGLE_EINVAL
    for bad in BAD_CACHES:
        assert rows(lib, fn, cache(**bad)) == L.EAGLE_EINVAL, bad
    assert rows(lib, fn, cache(max_batch=1 << 15, cap=1 << 16)) == L.EAGLE_ECAPACITY
    for kw in (dict(dtype=2), dict(R=-1), dict(k=None), dict(v=FAKE + 2), dict(ldk=1016), dict(ldv=1028), dict(seq=None),
               dict(slot=None), dict(dtype=0, ldk=1026)):
        assert rows(lib, fn, cache(), **kw) == L.EAGLE_EINVAL, kw
    assert rows(lib, fn, cache(), R=0, k=None, v=None, seq=None, slot=None) == L.EAGLE_OK   # nothing to do


def attn(lib, c, pk=None, pv=None, P=0, q=FAKE, out=FAKE, R=8, nq=32, rps=4, seq=FAKE, slot=FAKE, ctx=FAKE, mode=0, T=0,
         mask=None, words=0, scratch=FAKE, nb=1 << 40):
    return lib.eagle_op_attention_shared_kv8(None, c, pk, pv, P, q, out, R, nq, rps, seq, slot, ctx, mode, T, mask, words,
                                             0.0, scratch, nb, None)


def test_attention_refuses(lib):
    for bad in BAD_CACHES:
        assert attn(lib, cache(**bad)) == L.EAGLE_EINVAL, bad
        assert lib.eagle_op_attention_kv8_scratch_bytes(cache(**bad), 8, 32, 4, 0) == 0, bad
    for kw in (dict(R=0), dict(R=-3), dict(nq=0), dict(nq=30), dict(nq=8 * 65), dict(rps=0), dict(P=-1), dict(q=None),
               dict(out=None), dict(q=FAKE + 2), dict(out=FAKE + 8), dict(seq=None), dict(slot=None), dict(mode=2),
               dict(mode=1, T=4, mask=None, words=1), dict(mode=1, T=0, mask=FAKE, words=1),
               dict(mode=1, T=257, mask=FAKE, words=5), dict(mode=1, T=65, mask=FAKE, words=1),
               dict(mode=1, T=4, mask=FAKE, words=1, ctx=None), dict(P=9), dict(P=9, pk=FAKE, pv=FAKE + 2)):
        assert attn(lib, cache(), **kw) == L.EAGLE_EINVAL, kw
    need = lib.eagle_op_attention_kv8_scratch_bytes(cache(), 8, 32, 4, 0)
    assert need > 0
    assert attn(lib, cache(), nb=need - 1) == L.EAGLE_ECAPACITY
    assert attn(lib, cache(), scratch=None) == L.EAGLE_ECAPACITY
    assert attn(lib, cache(), scratch=FAKE + 8) == L.EAGLE_ECAPACITY
    assert attn(lib, cache(), R=1 << 24) == L.EAGLE_ECAPACITY
    assert lib.eagle_op_attention_kv8_scratch_bytes(cache(), 0, 32, 4, 0) == 0
    assert lib.eagle_op_attention_kv8(None, cache(), None, FAKE, 8, 32, 4, FAKE, FAKE, FAKE, 0, 0, None, 0, 0.0, FAKE,
                                      1 << 40, None) == L.EAGLE_EINVAL


def cpu_cache(table=None, **kw):
    c = dict(k=torch.zeros(2, 3, 32, 64, dtype=torch.uint8), v=torch.zeros(2, 3, 32, 64, dtype=torch.uint8),
             k_exp=torch.zeros(2, 3, 32, dtype=torch.uint8), v_exp=torch.zeros(2, 3, 32, dtype=torch.uint8))
    c.update(kw)
    return api.KV8Cache(c["k"], c["v"], c["k_exp"], c["v_exp"], table)


def test_binding_refuses_wrong_tensors():
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)
    with pytest.raises(ValueError):
        cpu_cache(k=z(2, 3, 32, 64, dt=torch.int8))
    with pytest.raises(ValueError):
        cpu_cache(v=z(2, 3, 32, 128))
    with pytest.raises(ValueError):
        cpu_cache(k_exp=z(2, 3, 16))
    with pytest.raises(ValueError):
        cpu_cache(k=z(2, 3, 64, 64)[:, :, ::2])
    with pytest.raises(ValueError):
        cpu_cache(table=z(2, 4, dt=torch.int64))
    c = cpu_cache()
    assert (c.max_batch, c.nkv, c.cap, c.d) == (2, 3, 32, 64)
    p = api.KV8Cache.empty(3, 3, 70, 64, device="cpu", block=32)
    assert (p.max_batch, p.cap, p.n_blocks, p.block) == (3, 96, 9, 32) and int(p.table.max()) == -1
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    rows = torch.zeros(5, 3, 64)
    for k, v in ((rows.half(), rows.half()), (rows, rows.bfloat16()), (rows[:, :2], rows[:, :2]),
                 (rows, torch.zeros(4, 3, 64)), (torch.zeros(5, 3, 128)[:, :, ::2], rows),
                 (torch.zeros(5, 6, 64)[:, ::2], rows)):
        with pytest.raises(ValueError):
            api.kv8_write(c, k, v, i32(5), i32(5))
    with pytest.raises(ValueError):
        api.kv8_write(c, rows, rows, i32(4), i32(5))
    with pytest.raises(ValueError):
        api.kv8_write(c, rows, rows, i32(5).long(), i32(5))
    with pytest.raises(ValueError):
        api.kv8_read(c, i32(5), i32(5), out=(rows[:4], rows[:4]))
    with pytest.raises(ValueError):
        api.kv8_read(c, i32(5), i32(5), dtype=torch.float16)
    q = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    bad = [dict(q=q.float()), dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1)), dict(out=q.float()),
           dict(prefix_k=torch.zeros(3, 5, 64)), dict(prefix_k=torch.zeros(2, 5, 64, dtype=torch.bfloat16)),
           dict(mask=torch.zeros(4, 1, dtype=torch.int32)), dict(mask=torch.zeros(3, 1, dtype=torch.int64)),
           dict(row_seq=i32(3)), dict(ctx_len=i32(1)), dict(err=torch.zeros(1)), dict(scratch=torch.zeros(64)),
           dict(rows_per_seq=0), dict(q=torch.zeros(4, 7, 64, dtype=torch.bfloat16))]
    for kw in bad:
        a = dict(q=q, prefix_k=None, prefix_v=None, cache=c, row_seq=i32(4), row_slot=i32(4), ctx_len=i32(2),
                 rows_per_seq=2, mode=0)
        a.update(kw)
        if kw.get("prefix_k") is not None:
            a["prefix_v"] = kw["prefix_k"]
        with pytest.raises(ValueError):
            api.attention_shared_kv8(**a)


def test_sizes_at_their_limits(lib):
    size = lambda rps, P=0, **kw: lib.eagle_op_attention_kv8_scratch_bytes(cache(**kw), 8, 32, rps, P)
    assert size((1 << 31) - 1) == size(8) > 0            # more rows a sequence than rows: one sequence
    assert size(4, (1 << 28) - 513) > 0
    assert size(4, (1 << 28) - 512) == 0                 # 8 heads: prefix slots past 32 bits once rounded up
    assert size(4, max_batch=1, cap=(1 << 28) - 528) > 0
    assert size(4, max_batch=1, cap=(1 << 28) - 512) == 0


def test_out_may_be_q_but_not_overlap_it(lib):
    step = 32 * 128 * 2
    for out in (FAKE + step, FAKE + 8 * step - 16, FAKE - 16):
        assert attn(lib, cache(), q=FAKE, out=out) == L.EAGLE_EINVAL


def test_tensors_of_the_cpu_are_refused():
    """Calls whose tensors agree with one another but lie on the CPU: refused before any launch."""
    c = cpu_cache()
    rows, i32 = torch.zeros(4, 3, 64), torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    for call in (lambda: api.kv8_write(c, rows, rows, i32, i32), lambda: api.kv8_read(c, i32, i32),
                 lambda: api.kv8_read(c, i32, i32, out=(rows, rows)),
                 lambda: api.attention_kv8(q, c, i32, i32, i32, 2, 0),
                 lambda: api.attention_shared_kv8(q, torch.zeros(3, 5, 64, dtype=torch.bfloat16),
                                                  torch.zeros(3, 5, 64, dtype=torch.bfloat16), c, i32, i32, i32, 2, 0)):
        with pytest.raises(ValueError, match="GPU"):
            call()
