"""Measured cases of the compressed-cache serving operators: writing an 8-bit KV cache, reading it back,
tree / causal attention over it, and the same attention behind a prefix that the whole batch shares.

The cache holds e4m3 codes and one power-of-two exponent byte per (slot, head) vector:
value = code * 2^(byte - 127), byte 255 = the vector held something that is not finite.
`own` false: each operator in elementary torch operations; true: the package's entry points.
"""
import math

import torch

own = False

E_LO, E_HI = -40, 40          # exponents that the cache stores
E4M3_MAX = 448.0


# ---- the cases --------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a batch of 64 over 16-slot blocks: the smallest write, latency counts
        dict(name="write-step-64", op="write", B=64, T=1, nkv=8, d=128, lo=128, hi=2048, block=16, dtype="bf16", fused=False),
        # a 4096-token prompt of the 40-head long-context model, straight from the fp32 projection [q | k | v]
        dict(name="write-prompt-4096", op="write", B=1, T=4096, nkv=40, d=128, lo=0, hi=0, block=0, dtype="f32", fused=True),
        # 61 tree rows of five 64-wide heads: an odd head count
        dict(name="write-tree-61-d64", op="write", B=1, T=61, nkv=5, d=64, lo=333, hi=333, block=0, dtype="bf16", fused=True),
        # the accepted paths of a batch of 64, fetched before they move to their committed slots
        dict(name="read-accepted-64", op="read", B=64, T=5, nkv=8, d=128, lo=128, hi=2048, block=16, dtype="bf16"),
        # a whole 4096-token sequence handed to a full-precision cache
        dict(name="read-sequence-4096", op="read", B=1, T=4096, nkv=40, d=128, lo=0, hi=0, block=0, dtype="bf16"),
        # one decoding step of a single long conversation
        dict(name="step-1x32768", op="attention", B=1, T=1, nq=32, nkv=8, d=128, lo=32768, hi=32768, block=0, mode="causal", pad=False),
        # one decoding step of a batch of 64 prompts of 128 to 2048 tokens over 16-slot blocks
        dict(name="step-64xragged", op="attention", B=64, T=1, nq=32, nkv=8, d=128, lo=128, hi=2048, block=16, mode="causal", pad=False),
        # the verify pass of the same batch: 17 tree rows a sequence
        dict(name="tree-64xraggedx17", op="attention", B=64, T=17, nq=32, nkv=8, d=128, lo=128, hi=2048, block=16, mode="tree", pad=False),
        # the verify pass of one sequence: 61 tree rows behind a 1024-token prompt, latency counts
        dict(name="tree-1x1024x61", op="attention", B=1, T=61, nq=32, nkv=8, d=128, lo=1024, hi=1024, block=0, mode="tree", pad=False),
        # 64 conversations behind one 8192-token system prompt, one decoding step
        dict(name="shared-8192-step-64", op="shared", B=64, T=1, nq=32, nkv=8, d=128, P=8192, lo=32, hi=512, block=16, mode="causal", pad=False),
        # the same with 17 tree rows a conversation behind 4096 shared tokens: the largest work
        dict(name="shared-4096-tree-64x17", op="shared", B=64, T=17, nq=32, nkv=8, d=128, P=4096, lo=16, hi=256, block=16, mode="tree", pad=False),
        # three short conversations, 64-wide heads, an odd prefix, one of them with nothing of its own yet
        dict(name="shared-333-tree-3x7-d64", op="shared", B=3, T=7, nq=10, nkv=5, d=64, P=333, lo=0, hi=40, block=0, mode="tree", pad=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        top[c["op"]] = max(top.get(c["op"], 0.0), max(w["bytes"], w["flops"] / 50))
    while True:
        op = rng.choice(["write", "read", "attention", "shared", "attention", "shared"])
        d = rng.choice([128, 128, 64])
        nq, nkv = rng.choice([(32, 8), (32, 8), (32, 32), (40, 40), (5, 5), (10, 5), (28, 4), (64, 8)])
        block = rng.choice([0, 16, 32, 64])
        B = _log_int(rng, 1, 64)
        if op in ("write", "read"):
            T = _log_int(rng, 1, 4096) if B <= 4 else _log_int(rng, 1, 61)
            lo = 0 if B == 1 and T > 61 else _log_int(rng, 1, 1024)
            c = dict(op=op, B=B, T=T, nkv=nkv, d=d, lo=lo, hi=lo + rng.randrange(0, lo + 1), block=block,
                     dtype=rng.choice(["bf16", "f32"]))
            if op == "write":
                c["fused"] = rng.random() < 0.5
        else:
            mode = rng.choice(["causal", "tree"])
            T = rng.choice([1, _log_int(rng, 1, 61)])
            lo = _log_int(rng, 1, 32768 if op == "attention" else 1024)
            hi = lo + rng.randrange(0, lo + 1)
            if rng.random() < 0.2:
                lo = 0
            c = dict(op=op, B=B, T=T, nq=nq, nkv=nkv, d=d, lo=lo, hi=hi, block=block, mode=mode, pad=rng.random() < 0.3)
            if op == "shared":
                c["P"] = _log_int(rng, 1, 16384)
        w = work(c)
        # entries of the plain form's fp32 caches and scores: a draw stays below the largest listed case
        S = c["hi"] + c["T"]
        room = c["B"] * c["nkv"] * S * c["d"]
        scores = 0 if op in ("write", "read") else c["B"] * c["nq"] * c["T"] * (S + c.get("P", 0))
        if max(w["bytes"], w["flops"] / 50) <= top[op] and room <= 1.5e8 and scores <= 1.6e8:
            return c


def _lens(c):
    """Context lengths of the case's sequences: evenly spread from lo to hi."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [lo + (i * (hi - lo)) // max(1, B - 1) for i in range(B)]


def work(c):
    d, nkv, T, B = c["d"], c["nkv"], c["T"], c["B"]
    if c["op"] in ("write", "read"):
        n = 2 * B * T * nkv
        return {"bytes": n * (d * (4 if c["dtype"] == "f32" else 2) + d + 1) + 8 * B * T, "flops": 3 * n * d}
    own_keys = sum(_lens(c)) + B * T
    P = c.get("P", 0)
    seen = sum(T * n + (T * (T + 1) // 2 if c["mode"] == "causal" else 4 * T) for n in _lens(c)) + B * T * P
    return {"bytes": own_keys * nkv * 2 * (d + 1) + P * nkv * d * 4 + 2 * B * T * c["nq"] * d * 2 + 8 * B * T,
            "flops": 4 * seen * c["nq"] * d}


def _pow2(e):
    """2^e of whole numbers in fp32's normal range, put together from the exponent's bits: no pow, which may round."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


# ---- inputs -----------------------------------------------------------------------------------
def _quantise(x):
    """(codes, exponent bytes) of vectors x [..., d]: the smallest exponent in [E_LO, E_HI] with
    max |x| <= 448 * 2^e, codes rounded to nearest even."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(top == 0, torch.full_like(e, E_LO), e).clamp(E_LO, E_HI)
    bad = ~torch.isfinite(top)
    e = torch.where(bad, torch.zeros_like(e), e)
    y = (x * _pow2(-e)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    y = torch.where(bad[..., None], torch.zeros_like(y), y)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _tree_masks(B, T, gen):
    """Ancestry bit masks [B * T][words] of random trees, parents before children, at most 8 deep."""
    words = (T + 63) // 64
    out = torch.zeros(B * T, words, dtype=torch.int64)
    pick = torch.rand(B, T, generator=gen).tolist()
    for b in range(B):
        bits, depth = [1], [0]
        for i in range(1, T):
            p = int(pick[b][i] * i)
            while depth[p] >= 8:
                p //= 2
            bits.append(bits[p] | (1 << i))
            depth.append(depth[p] + 1)
        for i, m in enumerate(bits):
            for w in range(words):
                x = (m >> (64 * w)) & (2 ** 64 - 1)
                out[b * T + i, w] = x - 2 ** 64 if x >= 2 ** 63 else x
    return out


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    B, T, nkv, d, block = c["B"], c["T"], c["nkv"], c["d"], c["block"]
    R = B * T
    lens = torch.tensor(_lens(c))[torch.randperm(B, generator=host)]
    cap = (c["hi"] + T + 15) // 16 * 16
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731

    # keys have a few strong channels, values a size of their own per token
    chan = torch.exp(0.5 * randn(nkv, d))
    if block:
        per = (cap + block - 1) // block
        n = B * per
        table = torch.randperm(n, generator=host).to(torch.int32).view(B, per).to(dev)
        shape, sizes = (n, nkv, block, d), (n, nkv, block, 1)
    else:
        table, shape, sizes = None, (B, nkv, cap, d), (B, nkv, cap, 1)
    k, k_exp = _quantise(randn(*shape) * chan[:, None, :])
    v, v_exp = _quantise(randn(*shape) * torch.exp(0.7 * randn(*sizes)))
    st = dict(case=c, k=k, v=v, k_exp=k_exp, v_exp=v_exp, table=table, cap=cap, lens=lens.tolist(),
              row_seq=torch.arange(B).repeat_interleave(T).to(torch.int32).to(dev),
              row_slot=(lens[:, None] + torch.arange(T)).reshape(-1).to(torch.int32).to(dev),
              ctx_len=lens.to(torch.int32).to(dev))
    if c["op"] == "write":
        dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        if c["fused"]:        # the k and v columns of a fused projection [q | k | v] with as many q heads
            rows = randn(R, 3, nkv, d).to(dt)
            st["new_k"], st["new_v"] = rows[:, 1], rows[:, 2]
        else:
            st["new_k"], st["new_v"] = randn(R, nkv, d).to(dt), randn(R, nkv, d).to(dt)
    elif c["op"] == "read":
        st["dtype"] = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    else:
        st["q"] = (2 * randn(R, c["nq"], d)).to(torch.bfloat16)
        st["mask"] = _tree_masks(B, T, host).to(dev) if c["mode"] == "tree" else None
        if c["pad"]:          # the last third of a sequence's rows is padding
            st["row_seq"].view(B, T)[torch.rand(B, generator=host).to(dev) < 0.5, T - T // 3:] = -1
        if c["op"] == "shared":
            st["pk"] = (randn(nkv, c["P"], d) * chan[:, None, :]).to(torch.bfloat16)
            st["pv"] = (randn(nkv, c["P"], d) * torch.exp(0.7 * randn(nkv, c["P"], 1))).to(torch.bfloat16)
    if own:
        from eagle_speculative_decoding_cycle_gb300 import api
        st["cache"] = api.KV8Cache(k, v, k_exp, v_exp, table=table)
        if c["op"] in ("attention", "shared"):   # the scratch that a serving loop keeps
            st["scratch"] = api.attention_kv8_scratch(st["cache"], R, c["nq"], T, prefix_len=c.get("P", 0))
    return st


# ---- one pass -----------------------------------------------------------------------------------
def run(st):
    c = st["case"]
    if own:
        from eagle_speculative_decoding_cycle_gb300 import api
        if c["op"] == "write":
            api.kv8_write(st["cache"], st["new_k"], st["new_v"], st["row_seq"], st["row_slot"])
            return _cache_values(st)
        if c["op"] == "read":
            k, v = api.kv8_read(st["cache"], st["row_seq"], st["row_slot"], dtype=st["dtype"])
            return {"k": k, "v": v}
        tree = c["mode"] == "tree"
        kw = dict(mode=int(tree), tree_T=c["T"] if tree else 0, mask=st["mask"], scratch=st["scratch"])
        if c["op"] == "attention":
            return {"out": api.attention_kv8(st["q"], st["cache"], st["row_seq"], st["row_slot"], st["ctx_len"], c["T"], **kw)}
        return {"out": api.attention_shared_kv8(st["q"], st["pk"], st["pv"], st["cache"], st["row_seq"], st["row_slot"],
                                                st["ctx_len"], c["T"], **kw)}
    if c["op"] == "write":
        at = _places(st)
        for name, x in (("k", st["new_k"]), ("v", st["new_v"])):
            codes, e = _quantise(x)
            st[name][at] = codes
            st[name + "_exp"][at] = e
        return _cache_values(st)
    if c["op"] == "read":
        at = _places(st)
        return {n: _value(st[n][at], st[n + "_exp"][at]).to(st["dtype"]) for n in ("k", "v")}
    return {"out": _attention(st)}


def _cache_values(st):
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn),
            "k_exp": st["k_exp"], "v_exp": st["v_exp"]}


def _places(st):
    """Index of each row's vectors [R, nkv] in the cache tensors."""
    heads = torch.arange(st["case"]["nkv"], device=st["k"].device)[None, :]
    seq, slot = st["row_seq"].long(), st["row_slot"].long()
    if st["table"] is None:
        return seq[:, None], heads, slot[:, None]
    block = st["case"]["block"]
    return st["table"][seq, slot // block].long()[:, None], heads, (slot % block)[:, None]


def _value(codes, e):
    ok = (e != 255)
    x = codes.view(torch.float8_e4m3fn).float() * _pow2(torch.where(ok, e.int() - 127, 0))[..., None]
    return torch.where(~ok[..., None], torch.full_like(x, math.nan), x)


def _own_keys(st, name, S):
    """The sequences' first S slots [B, nkv, S, d] in fp32."""
    x, e = st[name], st[name + "_exp"]
    if st["table"] is not None:
        nb = -(-S // st["case"]["block"])
        t = st["table"][:, :nb].long()
        x, e = x[t].transpose(1, 2).flatten(2, 3), e[t].transpose(1, 2).flatten(2, 3)
    return _value(x[:, :, :S], e[:, :, :S])


def _attention(st):
    c = st["case"]
    B, T, nq, nkv, d = c["B"], c["T"], c["nq"], c["nkv"], c["d"]
    G = nq // nkv
    S = max(st["lens"]) + T
    dev = st["q"].device
    slot = torch.arange(S, device=dev)
    live = (st["row_seq"] >= 0).view(B, T, 1)
    if c["mode"] == "causal":
        see = (slot <= st["row_slot"].view(B, T, 1)) & live
    else:
        t = slot - st["ctx_len"][:, None]                                        # [B, S]
        inside = (t >= 0) & (t < T)
        tc = t.clamp(0, T - 1)[:, None, :]
        word = torch.gather(st["mask"].view(B, T, -1), 2, (tc // 64).expand(B, T, S))
        see = ((t < 0)[:, None, :] | (inside[:, None, :] & ((word >> (tc % 64)) & 1).bool())) & live
    used = see.any(1)[:, None, :, None]                                          # [B, 1, S, 1]
    K, V = _own_keys(st, "k", S), _own_keys(st, "v", S)
    K, V = torch.where(used, K, torch.zeros_like(K)), torch.where(used, V, torch.zeros_like(V))
    q = st["q"].float().view(B, T, nkv, G, d).permute(0, 2, 1, 3, 4)             # [B, nkv, T, G, d]
    scale = 1.0 / math.sqrt(d)
    s = torch.matmul(q.reshape(B, nkv, T * G, d), K.transpose(2, 3)).view(B, nkv, T, G, S) * scale
    s = s.masked_fill(~see[:, None, :, None, :], -math.inf)
    top = s.amax(-1)
    if c["op"] == "shared":
        qp = q.permute(1, 0, 2, 3, 4).reshape(nkv, B * T * G, d)
        sp = torch.matmul(qp, st["pk"].float().transpose(1, 2)) * scale          # [nkv, B T G, P]
        top = torch.maximum(top, sp.amax(-1).view(nkv, B, T, G).transpose(0, 1))
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - top[..., None])
    total = p.sum(-1)
    o = torch.matmul(p.view(B, nkv, T * G, S), V).view(B, nkv, T, G, d)
    if c["op"] == "shared":
        pp = torch.exp(sp - top.transpose(0, 1).reshape(nkv, B * T * G, 1))
        total = total + pp.sum(-1).view(nkv, B, T, G).transpose(0, 1)
        o = o + torch.matmul(pp, st["pv"].float()).view(nkv, B, T, G, d).transpose(0, 1)
    o = torch.where((total > 0)[..., None], o / total[..., None], torch.zeros_like(o))
    o = torch.where(live.view(B, 1, T, 1, 1), o, torch.zeros_like(o))
    return o.permute(0, 2, 1, 3, 4).reshape(B * T, nq, d).to(torch.bfloat16)


# ---- the definition in 64 bits ------------------------------------------------------------------
def _table64(dev):
    """The 256 e4m3 codes' values: sign, four exponent bits of bias 7, three fraction bits, no infinities."""
    v = []
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v.append(math.nan if e == 15 and f == 7 else (-x if code & 128 else x))
    return torch.tensor(v, dtype=torch.float64, device=dev)


def _two64(e):
    """2^e of whole numbers in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _rows64(st, name, b, slots):
    """Cache vectors [nkv, n, d] of sequence b at `slots` in 64 bits."""
    if st["table"] is None:
        x, e = st[name][b][:, slots], st[name + "_exp"][b][:, slots]
    else:
        block = st["case"]["block"]
        blk = st["table"][b].long()[slots // block]
        x, e = st[name][blk, :, slots % block].transpose(0, 1), st[name + "_exp"][blk, :, slots % block].transpose(0, 1)
    return _table64(x.device)[x.long()] * _two64(e.long() - 127)[..., None]


def exact(case, seed):
    c, st = case, prepare(case, seed)
    B, T, nkv, d = c["B"], c["T"], c["nkv"], c["d"]
    dev = st["k"].device
    if c["op"] == "write":
        out = {n: _table64(dev)[st[n].long()] for n in ("k", "v")}
        out.update({n + "_exp": st[n + "_exp"].clone() for n in ("k", "v")})
        for n in ("k", "v"):
            x = st["new_" + n].double()
            top = x.abs().amax(-1)
            e = torch.ceil(torch.log2(top.clamp_min(1e-300) / E4M3_MAX))
            e = torch.where(_two64(e - 1) * E4M3_MAX >= top, e - 1, e)   # log2 of a power of two may round up
            e = torch.where(_two64(e) * E4M3_MAX < top, e + 1, e).clamp(E_LO, E_HI)
            y = x / _two64(e)[..., None]
            step = _two64(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)      # eight steps in each binade
            y = (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
            for b in range(B):
                at = st["row_slot"].view(B, T)[b].long()
                rows, er = y.view(B, T, nkv, d)[b], (e + 127).view(B, T, nkv)[b].to(torch.uint8)
                if st["table"] is None:
                    out[n][b][:, at] = rows.transpose(0, 1)
                    out[n + "_exp"][b][:, at] = er.transpose(0, 1)
                else:
                    blk = st["table"][b].long()[at // c["block"]]
                    out[n][blk, :, at % c["block"]] = rows
                    out[n + "_exp"][blk, :, at % c["block"]] = er
        return out
    if c["op"] == "read":
        return {n: torch.cat([_rows64(st, n, b, st["row_slot"].view(B, T)[b].long()).transpose(0, 1) for b in range(B)])
                for n in ("k", "v")}
    if work(c)["flops"] > 4e11:      # over about 20 seconds at this card's 64-bit rate
        return None
    nq = c["nq"]
    G = nq // nkv
    out = torch.zeros(B, T, nq, d, dtype=torch.float64, device=dev)
    bits = None if st["mask"] is None else st["mask"].view(B, T, -1).cpu().tolist()
    for b in range(B):
        n = st["lens"][b]
        slots = torch.arange(n + T, device=dev)
        K, V = _rows64(st, "k", b, slots), _rows64(st, "v", b, slots)
        if bits is None:
            see = torch.tensor([[s <= n + t for s in range(n, n + T)] for t in range(T)])
        else:
            see = torch.tensor([[(bits[b][t][s // 64] >> (s % 64)) & 1 == 1 for s in range(T)] for t in range(T)])
        hide = torch.cat([torch.zeros(T, n, dtype=torch.bool), ~see], 1).to(dev)
        if c["op"] == "shared":
            K, V = torch.cat([st["pk"].double(), K], 1), torch.cat([st["pv"].double(), V], 1)
            hide = torch.cat([torch.zeros(T, c["P"], dtype=torch.bool, device=dev), hide], 1)
        q = st["q"].view(B, T, nkv, G, d)[b].double()
        s = torch.einsum("thgd,hsd->htgs", q, K) / math.sqrt(d)
        s = s.masked_fill(hide[None, :, None, :], -math.inf)
        out[b] = torch.einsum("htgs,hsd->thgd", torch.softmax(s, -1), V).reshape(T, nq, d)
        out[b][(st["row_seq"].view(B, T)[b] < 0)] = 0
    return {"out": out.view(B * T, nq, d)}
