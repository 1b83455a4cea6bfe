"""Measured cases of the operators that take a prompt into a served batch and keep its cache pages: rotary positions,
attention over whole prompts packed one behind another, moving accepted paths in all layers of an 8-bit cache, and
assigning, forking and releasing its blocks.

`own` false: each operator in elementary torch operations; true: the package's entry points.

Rotary positions: a vector's first `rot` entries are pairs, (x[i], x[i + rot/2]) or, interleaved, (x[2i], x[2i + 1]); pair i of a
row at position p is turned by p * f[i]. f[i] = theta^(-2i / rot), changed for long contexts by one of four published rules.
Prompt attention: rows of sequence b are q[start[b] .. start[b+1]) with keys k[kstart[b] .. kstart[b+1]); the last row sees all of
the sequence's keys, each row before it one fewer. Row results and log-sum-exps.
Pages: a block table [sequence][slots / block] over a pool of blocks, -1 where none, and a count of the table's entries for
each block. After a call sequence b has exactly the blocks of its first length[b] slots: surplus ones are released, missing ones are
the lowest-numbered free ones, in the order of sequences and slots. A block that the sequence could write to and others still
hold (its last one, partly filled) is replaced by a copy. A fork first takes its parent's blocks in place of its own.
"""
import math

import torch

own = False


# ---- the cases --------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a batch of 64 in contexts of up to 131072 tokens: the smallest, latency counts
        dict(name="rope-step-64", op="rope", R=64, far=131072, nq=32, nkv=8, d=128, rot=128, pairs="halves",
             rule="bands", theta=5e5, src="bf16", dst="bf16", back=False),
        # a 4096-token prompt of the 40-head long-context model, from the fp32 projection [q | k | v] to bf16 rows
        dict(name="rope-prompt-4096", op="rope", R=4096, far=0, nq=40, nkv=40, d=128, rot=128, pairs="halves",
             rule="none", theta=1e4, src="f32", dst="bf16", back=False),
        # keys and queries of 61 tree rows turned back to position zero, half of each 64-wide head turned
        dict(name="rope-back-61-d64", op="rope", R=61, far=40000, nq=10, nkv=5, d=64, rot=32, pairs="neighbours",
             rule="ramp", theta=1e4, src="f32", dst="f32", back=True),
        # three short prompts of odd lengths, 64-wide heads: latency counts
        dict(name="prompt-3-short-d64", op="prompt", B=3, lo=1, hi=77, before=0, nq=10, nkv=5, d=64),
        # the batch-1 prompt of 1024 tokens
        dict(name="prompt-1x1024", op="prompt", B=1, lo=1024, hi=1024, before=0, nq=32, nkv=8, d=128),
        # the long-context model's prompt of 4096 tokens, a head of keys for each head of queries
        dict(name="prompt-1x4096", op="prompt", B=1, lo=4096, hi=4096, before=0, nq=40, nkv=40, d=128),
        # its last chunk of 512 rows behind the 3584 before
        dict(name="prompt-chunk-512", op="prompt", B=1, lo=512, hi=512, before=3584, nq=40, nkv=40, d=128),
        # the 64 prompts of 128 to 2048 tokens that a batch starts with, packed: the largest work
        dict(name="prompt-64xragged", op="prompt", B=64, lo=128, hi=2048, before=0, nq=32, nkv=8, d=128),
        # the accepted paths of a batch of 64 in all 32 layers, blocks of 16
        dict(name="compact-64x32", op="compact", B=64, layers=32, nkv=8, d=128, lo=5, hi=100, deep=5, T=17, block=16),
        # the accepted path of one tree of 61 rows in the 40 layers of the long-context model, contiguous
        dict(name="compact-1x40", op="compact", B=1, layers=40, nkv=40, d=128, lo=333, hi=333, deep=6, T=49, block=0),
        # fifteen further answers to one prompt of 1000 tokens: its blocks shared, its last one copied in 32 layers
        dict(name="fork-15-of-1000", op="fork", parents=1, kids=15, n=1000, cut=0, layers=32, nkv=8, d=128, block=16),
        # a cycle of a batch of 64: slots for 17 tree rows, then only those of the accepted path kept
        dict(name="resize-cycle-64", op="resize", B=64, lo=128, hi=2048, T=17, block=16),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_HEADS = [(32, 8), (32, 8), (32, 32), (40, 40), (5, 5), (10, 5), (28, 4), (64, 8), (6, 1)]


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        top[c["op"]] = max(top.get(c["op"], 0.0), max(w["bytes"], w["flops"] / 50))
    while True:
        op = rng.choice(["rope", "prompt", "prompt", "compact", "fork", "resize"])
        nq, nkv = rng.choice(_HEADS)
        d = rng.choice([128, 128, 64])
        if op == "rope":
            src = rng.choice(["bf16", "f32"])
            c = dict(op=op, R=_log_int(rng, 1, 16384), far=rng.choice([0, _log_int(rng, 1, 1000000)]), nq=nq, nkv=nkv, d=d,
                     rot=rng.choice([d, d, d // 2, 16]), pairs=rng.choice(["halves", "neighbours"]),
                     rule=rng.choice(["none", "linear", "base", "bands", "ramp"]), theta=rng.choice([1e4, 5e5]), src=src,
                     dst="bf16" if src == "bf16" else rng.choice(["bf16", "f32"]), back=rng.random() < 0.25)
        elif op == "prompt":
            B = _log_int(rng, 1, 64)
            lo = _log_int(rng, 1, 4096)
            hi = lo + rng.randrange(0, lo + 1)
            if B > 1 and rng.random() < 0.2:
                lo = 0
            c = dict(op=op, B=B, lo=lo, hi=hi, before=0 if rng.random() < 0.6 else _log_int(rng, 1, 4096), nq=nq, nkv=nkv, d=d)
        elif op == "compact":
            lo = _log_int(rng, 1, 1024)
            c = dict(op=op, B=_log_int(rng, 1, 64), layers=_log_int(rng, 1, 40), nkv=nkv, d=d, lo=lo,
                     hi=lo + rng.randrange(0, lo + 1), deep=rng.randrange(1, 9), T=rng.randrange(9, 62),
                     block=rng.choice([0, 16, 32, 128]))
        elif op == "fork":
            n = _log_int(rng, 1, 4096)
            c = dict(op=op, parents=_log_int(rng, 1, 8), kids=_log_int(rng, 1, 16), n=n, cut=rng.choice([0, rng.randrange(0, n)]),
                     layers=_log_int(rng, 1, 32), nkv=nkv, d=d, block=rng.choice([16, 16, 32, 128]))
        else:
            lo = _log_int(rng, 1, 8192)
            c = dict(op=op, B=_log_int(rng, 1, 256), lo=lo, hi=lo + rng.randrange(0, lo + 1), T=_log_int(rng, 1, 61),
                     block=rng.choice([16, 16, 32, 128]))
        w = work(c)
        pool = 0
        if op in ("compact", "fork"):      # codes of the caches: a state stays a fraction of a gigabyte
            pool = _blocks(c) * max(1, c["block"]) * c["layers"] * c["nkv"] * c["d"]
        if max(w["bytes"], w["flops"] / 50) <= top[op] * 1.0001 and pool <= 1.5e8:
            return c


def _spread(B, lo, hi):
    """Lengths of B sequences: evenly spread from lo to hi."""
    return [lo + (i * (hi - lo)) // max(1, B - 1) for i in range(B)]


def _blocks(c):
    """Pool blocks of a case (slots of all sequences where the cache is contiguous)."""
    b = c["block"]
    if c["op"] == "fork":
        return c["parents"] * (c["kids"] + 2 + -(-c["n"] // b)) + 4
    if c["op"] == "resize":
        return sum(-(-(n + c["T"]) // b) for n in _spread(c["B"], c["lo"], c["hi"])) + 16
    cap = -(-(c["hi"] + c["T"]) // (b or 16)) * (b or 16)
    return c["B"] * cap // b if b else c["B"] * cap


def work(c):
    if c["op"] == "rope":
        n = c["R"] * (c["nq"] + c["nkv"])
        es = {"bf16": 2, "f32": 4}
        return {"bytes": n * c["d"] * (es[c["src"]] + es[c["dst"]]) + 4 * c["R"], "flops": 3 * n * c["rot"]}
    if c["op"] == "prompt":
        lens = _spread(c["B"], c["lo"], c["hi"])
        rows, keys = sum(lens), sum(n + c["before"] for n in lens)
        seen = sum(n * c["before"] + n * (n + 1) // 2 for n in lens)
        return {"bytes": 4 * rows * c["nq"] * c["d"] + 4 * keys * c["nkv"] * c["d"] + 4 * rows * c["nq"] + 8 * (c["B"] + 1),
                "flops": 4 * seen * c["nq"] * c["d"] + 1}
    if c["op"] == "compact":      # half of the path on average, read and written
        moved = c["B"] * (c["deep"] + 1) / 2 * c["layers"] * c["nkv"] * 2
        return {"bytes": 2 * moved * (c["d"] + 1) + 4 * c["B"] * (2 + c["deep"]), "flops": 0}
    if c["op"] == "fork":
        kids, n = c["parents"] * c["kids"], max(0, c["n"] - c["cut"])
        copied = kids * (n % c["block"]) * c["layers"] * c["nkv"] * 2
        return {"bytes": 2 * copied * (c["d"] + 1) + 8 * kids * (-(-n // c["block"])) + 8 * _blocks(c), "flops": 0}
    entries = sum(-(-(n + c["T"]) // c["block"]) for n in _spread(c["B"], c["lo"], c["hi"]))
    return {"bytes": 2 * (4 * entries + 4 * _blocks(c) + 4 * c["B"]), "flops": 0}


# ---- inputs -----------------------------------------------------------------------------------
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_RULES = {"none": None, "linear": dict(kind="linear", factor=4.0), "base": dict(kind="ntk", factor=4.0),
          "bands": dict(kind="llama3", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original=8192),
          "ramp": dict(kind="yarn", factor=16.0, original=4096, beta_fast=32.0, beta_slow=1.0)}


def _pool(c, n, g, dev):
    """Codes and exponent bytes of the keys and values of all layers: [layers][n][nkv][slots of one][d]."""
    slots = c["block"] or n // c["B"]
    shape = (c["layers"], n if c["block"] else c["B"], c["nkv"], slots, c["d"])
    out = {}
    for name in ("k", "v"):
        out[name] = (60 * torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        out[name + "_exp"] = torch.randint(112, 124, shape[:4], generator=g, device=dev, dtype=torch.uint8)
    return out


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(dev)  # noqa: E731
    st = dict(case=c)
    if c["op"] == "rope":
        # q and k columns of a fused projection [q | k | v]; a prompt's positions in order, or a batch's, each its own
        rows = randn(c["R"], c["nq"] + 2 * c["nkv"], c["d"]).to(_TYPES[c["src"]])
        st.update(q=rows[:, :c["nq"]], k=rows[:, c["nq"]:c["nq"] + c["nkv"]], dtype=_TYPES[c["dst"]],
                  pos=i32(torch.randint(0, c["far"], (c["R"],), generator=host) if c["far"] else torch.arange(c["R"])))
    elif c["op"] == "prompt":
        lens = torch.tensor(_spread(c["B"], c["lo"], c["hi"]))[torch.randperm(c["B"], generator=host)]
        keys = lens + c["before"]
        ends = lambda n: [0] + torch.cumsum(n, 0).tolist()  # noqa: E731
        R, K, nq, nkv, d = int(lens.sum()), int(keys.sum()), c["nq"], c["nkv"], c["d"]
        # keys have a few strong channels, values a size of their own per token; values are the columns of a fused projection
        k = (randn(K, nkv, d) * torch.exp(0.5 * randn(nkv, d))).to(torch.bfloat16)
        v = (randn(K, 2, nkv, d) * torch.exp(0.7 * randn(K, 1, nkv, 1))).to(torch.bfloat16)[:, 1]
        st.update(q=(1.5 * randn(R, nq, d)).to(torch.bfloat16), k=k, v=v, ends=ends(lens), kends=ends(keys),
                  start=i32(ends(lens)), kstart=i32(ends(keys)))
    elif c["op"] == "compact":
        lens = torch.tensor(_spread(c["B"], c["lo"], c["hi"]))[torch.randperm(c["B"], generator=host)]
        n = _blocks(c)
        st.update(_pool(c, n, g, dev))
        st["table"] = i32(torch.randperm(n, generator=host).view(c["B"], -1)) if c["block"] else None
        # rising tree rows 1 .. T - 1 of each accepted path, of 0 to `deep` nodes
        path = torch.rand(c["B"], c["T"] - 1, generator=host).argsort(1)[:, :c["deep"]].sort(1)[0] + 1
        st.update(n_old=i32(lens), acc_len=i32(torch.randint(1, c["deep"] + 1, (c["B"],), generator=host)), path=i32(path))
    elif c["op"] == "fork":
        n, P, kids, b = _blocks(c), c["parents"], c["kids"], c["block"]
        per = -(-c["n"] // b)
        table = torch.full((P * (1 + kids), per + 1), -1, dtype=torch.int32)
        table[:P, :per] = torch.randperm(n, generator=host)[:P * per].view(P, per).to(torch.int32)
        parent = torch.cat([torch.full((P,), -1), torch.arange(P).repeat_interleave(kids)])
        length = torch.where(parent < 0, -1, max(0, c["n"] - c["cut"]))
        st.update(_pool(c, n, g, dev), table=table.to(dev), parent=i32(parent), length=i32(length))
    else:
        b, n = c["block"], _blocks(c)
        lens = torch.tensor(_spread(c["B"], c["lo"], c["hi"]))[torch.randperm(c["B"], generator=host)]
        j = torch.arange(-(-(c["hi"] + c["T"]) // b))
        held = j[None, :] < (-(-lens // b))[:, None]
        table = torch.full(held.shape, -1, dtype=torch.int32)
        table[held] = torch.randperm(n, generator=host)[:int(held.sum())].to(torch.int32)
        took = torch.randint(1, c["T"] + 1, (c["B"],), generator=host).clamp_max(9)
        st.update(_pool(dict(c, layers=1, nkv=1, d=64), n, g, dev), table=table.to(dev), grown=i32(lens + c["T"]), kept=i32(lens + took))
    if c["op"] in ("fork", "resize"):
        held = st["table"][st["table"] >= 0].long()
        st["ref"] = torch.bincount(held, minlength=_blocks(c)).to(torch.int32)
    if own:      # the handles that a serving program keeps
        from eagle_speculative_decoding_cycle_gb300 import api
        if c["op"] == "rope":
            st["rope"] = api.Rope(c["d"], theta=c["theta"], rot=c["rot"], interleaved=c["pairs"] == "neighbours",
                                  scaling=_RULES[c["rule"]])
        elif c["op"] != "prompt":
            st["layers"] = api.KV8Layers([api.KV8Cache(*x, st["table"]) for x in
                                          zip(st["k"], st["v"], st["k_exp"], st["v_exp"])], refs=st.get("ref"))
    return st


# ---- one pass -----------------------------------------------------------------------------------
def run(st):
    c = st["case"]
    if own:
        from eagle_speculative_decoding_cycle_gb300 import api
        if c["op"] == "rope":
            q, k = api.rope(st["rope"], st["q"], st["k"], st["pos"], dtype=st["dtype"], inverse=c["back"])
            return {"q": q, "k": k}
        if c["op"] == "prompt":
            lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=st["q"].device)
            return {"out": api.attention_prompt(st["q"], st["k"], st["v"], st["start"], st["kstart"], lse=lse), "lse": lse}
        if c["op"] == "compact":
            api.kv8_compact(st["layers"], st["n_old"], st["acc_len"], st["path"])
            return _values(st)
        if c["op"] == "fork":
            api.kv8_fork(st["layers"], st["parent"], st["length"])
            return {"table": st["table"], "ref": st["ref"], **_values(st)}
        api.kv8_resize(st["layers"], st["grown"])
        api.kv8_resize(st["layers"], st["kept"])
        return {"table": st["table"], "ref": st["ref"]}
    if c["op"] == "rope":
        cos, sin = _turns(c, st["pos"])
        return {n: _rotated(c, st[n], cos, sin).to(st["dtype"]) for n in ("q", "k")}
    if c["op"] == "prompt":
        return _prompt(st)
    if c["op"] == "compact":
        return _compact(st)
    if c["op"] == "fork":
        _resize(st, st["length"], st["parent"])
        return {"table": st["table"], "ref": st["ref"], **_values(st)}
    _resize(st, st["grown"])
    _resize(st, st["kept"])
    return {"table": st["table"], "ref": st["ref"]}


def _values(st):
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn),
            "k_exp": st["k_exp"], "v_exp": st["v_exp"]}


def _frequencies(c, dev):
    """(angle per position of each pair, factor of the turned entries), 64 bits."""
    rot, theta, r = c["rot"], c["theta"], _RULES[c["rule"]]
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    if r is None:
        return theta ** (-2 * i / rot), 1.0
    if r["kind"] == "ntk":          # another base, so that the slowest pair turns `factor` times slower
        return (theta * r["factor"] ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0
    f = theta ** (-2 * i / rot)
    if r["kind"] == "linear":
        return f / r["factor"], 1.0
    if r["kind"] == "llama3":       # slow pairs by the factor, fast ones unchanged, a blend between
        turns = r["original"] * f / (2 * math.pi)
        mix = ((turns - r["low_freq_factor"]) / (r["high_freq_factor"] - r["low_freq_factor"])).clamp(0, 1)
        return f * (mix + (1 - mix) / r["factor"]), 1.0
    # a ramp over the pairs between those that make beta_fast and beta_slow turns in the original context
    at = lambda beta: rot * math.log(r["original"] / (beta * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(at(r["beta_fast"])), 0), min(math.ceil(at(r["beta_slow"])), rot - 1)
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f * (1 - ramp + ramp / r["factor"]), 0.1 * math.log(r["factor"]) + 1


def _turns(c, pos):
    """Cosines and sines [R, 1, rot / 2]: angles in 64 bits, far positions lose them in 32."""
    f, factor = _frequencies(c, pos.device)
    a = pos.double()[:, None] * f
    return (torch.cos(a) * factor).float()[:, None], ((-factor if c["back"] else factor) * torch.sin(a)).float()[:, None]


def _rotated(c, x, cos, sin):
    x, rot = x.float(), c["rot"]
    t = x[..., :rot]
    if c["pairs"] == "halves":
        a, b = t[..., :rot // 2], t[..., rot // 2:]
        t = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = t[..., 0::2], t[..., 1::2]
        t = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([t, x[..., rot:]], -1)


def _prompt(st):
    """One sequence after another: padded to the longest, a ragged batch would take twice the products."""
    c = st["case"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    out, lse = torch.empty(st["q"].shape, dtype=torch.bfloat16, device=st["q"].device), []
    for b in range(c["B"]):
        r0, r1, k0, k1 = st["ends"][b], st["ends"][b + 1], st["kends"][b], st["kends"][b + 1]
        n, m = r1 - r0, k1 - k0
        if n == 0:
            continue
        q = st["q"][r0:r1].float().view(n, nkv, nq // nkv, d).permute(1, 2, 0, 3).reshape(nkv, -1, d)   # [nkv, G n, d]
        K, V = st["k"][k0:k1].float().transpose(0, 1), st["v"][k0:k1].float().transpose(0, 1)
        s = torch.matmul(q, K.transpose(1, 2)).mul_(1 / math.sqrt(d)).view(nkv, -1, n, m)
        hidden = torch.ones(n, m, dtype=torch.bool, device=s.device).triu_(m - n + 1)
        s.masked_fill_(hidden, -math.inf)
        top = s.amax(-1, keepdim=True)
        p = s.sub_(top).exp_()
        total = p.sum(-1)
        o = torch.matmul(p.view(nkv, -1, m), V).view(nkv, -1, n, d) / total[..., None]
        out[r0:r1] = o.permute(2, 0, 1, 3).reshape(n, nq, d).to(torch.bfloat16)
        lse.append((top[..., 0] + total.log()).permute(2, 0, 1).reshape(n, nq))
    return {"out": out, "lse": torch.cat(lse) if lse else out.new_empty((0, nq), dtype=torch.float32)}


def _compact(st):
    """Slot n_old + j takes what slot n_old + path[j - 1] held, j = 1 .. acc_len, in every layer and head."""
    c = st["case"]
    j = torch.arange(1, c["deep"] + 1, device=st["path"].device)[None, :]
    seq, at = torch.nonzero((j <= st["acc_len"][:, None]), as_tuple=True)
    src, dst = st["n_old"][seq].long() + st["path"][seq, at].long(), st["n_old"][seq].long() + at + 1
    heads = torch.arange(c["nkv"], device=seq.device)[None, :]

    def place(slot):
        if st["table"] is None:
            return slice(None), seq[:, None], heads, slot[:, None]
        return slice(None), st["table"][seq, slot // c["block"]].long()[:, None], heads, (slot % c["block"])[:, None]

    for name in ("k", "v", "k_exp", "v_exp"):
        st[name][place(dst)] = st[name][place(src)]
    return _values(st)


def _resize(st, length, parent=None):
    c, table, ref = st["case"], st["table"], st["ref"]
    b = c["block"]
    length = length.long()
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    nb = ((length + b - 1) // b)[:, None]
    active = (length >= 0)[:, None]
    drop = active & (table >= 0) & ((j >= nb) if parent is None else ((j >= nb) | (parent >= 0)[:, None]))
    ref -= torch.bincount(table[drop].long(), minlength=ref.numel()).to(torch.int32)
    table[drop] = -1
    if parent is not None:      # the parents' blocks in place of the dropped ones
        share = active & (parent >= 0)[:, None] & (j < nb)
        table.copy_(torch.where(share, table[parent.clamp_min(0).long()], table))
        ref += torch.bincount(table[share].long(), minlength=ref.numel()).to(torch.int32)
    ends = active & (j == nb - 1) & (length % b != 0)[:, None] & (table >= 0)
    copy = ends & (ref[table.clamp_min(0).long()] > 1)
    need = (active & (j < nb) & (table < 0)) | copy
    new = torch.nonzero(ref == 0)[:, 0][:int(need.sum())]
    old = table[need]
    table[need] = new.to(torch.int32)
    ref[new] = 1
    moved = copy[need]
    src, dst = old[moved].long(), new[moved]
    ref -= torch.bincount(src, minlength=ref.numel()).to(torch.int32)
    if src.numel():
        used = torch.arange(b, device=src.device)[None, :] < (length % b)[torch.nonzero(copy)[:, 0]][:, None]   # [n, block]
        for name in ("k", "v", "k_exp", "v_exp"):
            x, u = st[name], used[None, :, None, :]
            u = u[..., None] if x.dim() == 5 else u
            x[:, dst] = torch.where(u, x[:, src], x[:, dst])


# ---- the definition in 64 bits ------------------------------------------------------------------
def _codes64(x):
    """e4m3 values: sign, four exponent bits of bias 7, three fraction bits."""
    v = []
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        y = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v.append(math.nan if e == 15 and f == 7 else (-y if code & 128 else y))
    return torch.tensor(v, dtype=torch.float64, device=x.device)[x.int()]


def _pool64(st):
    return {n: st[n] if n.endswith("exp") else _codes64(st[n]) for n in ("k", "v", "k_exp", "v_exp")}


def _angles64(c):
    """Pair by pair, from the rules' own statements."""
    rot, theta, r, out, factor = c["rot"], c["theta"], _RULES[c["rule"]], [], 1.0
    for i in range(rot // 2):
        f = math.exp(-2 * i / rot * math.log(theta))
        if r is not None and r["kind"] == "linear":
            f = f / r["factor"]
        elif r is not None and r["kind"] == "ntk":
            f = f * r["factor"] ** (-2 * i / (rot - 2))
        elif r is not None and r["kind"] == "llama3":
            wave = 2 * math.pi / f
            if wave > r["original"] / r["low_freq_factor"]:
                f = f / r["factor"]
            elif wave >= r["original"] / r["high_freq_factor"]:
                s = (r["original"] / wave - r["low_freq_factor"]) / (r["high_freq_factor"] - r["low_freq_factor"])
                f = (1 - s) * f / r["factor"] + s * f
        elif r is not None:
            full = lambda beta: rot * math.log(r["original"] / (2 * math.pi * beta)) / (2 * math.log(theta))  # noqa: E731
            lo, hi = max(0, math.floor(full(r["beta_fast"]))), min(rot - 1, math.ceil(full(r["beta_slow"])))
            s = 0.0 if i <= lo else (1.0 if i >= hi else (i - lo) / (hi - lo))
            f, factor = f * (1 - s) + f / r["factor"] * s, 0.1 * math.log(r["factor"]) + 1
        out.append(f)
    return out, factor


def exact(case, seed):
    c, st = case, prepare(case, seed)
    dev = torch.device("cuda")
    if c["op"] == "rope":
        f, factor = _angles64(c)
        out = {}
        for name in ("q", "k"):
            y = st[name].double()
            x = y.clone()
            for i, w in enumerate(f):
                a, b = (i, i + c["rot"] // 2) if c["pairs"] == "halves" else (2 * i, 2 * i + 1)
                angle = st["pos"].double()[:, None] * (-w if c["back"] else w)
                y[..., a] = factor * (x[..., a] * torch.cos(angle) - x[..., b] * torch.sin(angle))
                y[..., b] = factor * (x[..., a] * torch.sin(angle) + x[..., b] * torch.cos(angle))
            out[name] = y
        return out
    if c["op"] == "prompt":
        if work(c)["flops"] > 4e12:      # over about 20 seconds at this card's 64-bit rate
            return None
        G = c["nq"] // c["nkv"]
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
        lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=dev)
        for b in range(c["B"]):
            rows, keys = slice(st["ends"][b], st["ends"][b + 1]), slice(st["kends"][b], st["kends"][b + 1])
            n = rows.stop - rows.start
            if n == 0:
                continue
            before = keys.stop - keys.start - n
            see = torch.arange(n + before, device=dev)[None, :] <= torch.arange(before, before + n, device=dev)[:, None]
            for h in range(c["nq"]):
                s = st["q"][rows, h].double() @ st["k"][keys, h // G].double().T / math.sqrt(c["d"])
                s = torch.where(see, s, -math.inf)
                out[rows, h] = torch.softmax(s, -1) @ st["v"][keys, h // G].double()
                lse[rows, h] = torch.logsumexp(s, -1)
        return {"out": out, "lse": lse}
    if c["op"] == "compact":
        n_old, took, path = st["n_old"].tolist(), st["acc_len"].tolist(), st["path"].tolist()
        for b in range(c["B"]):
            def at(slot, b=b):
                return (b, slot) if st["table"] is None else (int(table[b][slot // c["block"]]), slot % c["block"])
            table = None if st["table"] is None else st["table"].cpu()
            for name in ("k", "v", "k_exp", "v_exp"):
                x = st[name]
                read = [x[:, at(n_old[b] + p)[0], :, at(n_old[b] + p)[1]].clone() for p in path[b][:took[b]]]
                for i, r in enumerate(read):
                    d0, d1 = at(n_old[b] + 1 + i)
                    x[:, d0, :, d1] = r
        return _pool64(st)
    # the bookkeeping, one sequence and one block at a time
    b = c["block"]
    table, ref = st["table"].tolist(), st["ref"].tolist()
    calls = [(st["length"].tolist(), st["parent"].tolist())] if c["op"] == "fork" else \
        [(st["grown"].tolist(), None), (st["kept"].tolist(), None)]
    for length, parent in calls:
        forks = [s for s in range(len(table)) if parent is not None and parent[s] >= 0 and length[s] >= 0]
        for s, n in enumerate(length):
            for j in range(len(table[s])):
                if n >= 0 and table[s][j] >= 0 and (s in forks or j * b >= n):
                    ref[table[s][j]] -= 1
                    table[s][j] = -1
        for s in forks:
            for j in range(-(-length[s] // b)):
                table[s][j] = table[parent[s]][j]
                ref[table[s][j]] += 1
        shared = [n > 1 for n in ref]
        free = [i for i, n in enumerate(ref) if n == 0]
        for s, n in enumerate(length):
            for j in range(-(-n // b) if n > 0 else 0):
                if table[s][j] < 0:
                    table[s][j] = free.pop(0)
                    ref[table[s][j]] = 1
                elif n < (j + 1) * b and shared[table[s][j]]:
                    old, new = table[s][j], free.pop(0)
                    table[s][j], ref[new], ref[old] = new, 1, ref[old] - 1
                    for name in ("k", "v", "k_exp", "v_exp"):
                        st[name][:, new, :, :n - j * b] = st[name][:, old, :, :n - j * b]
    out = {"table": torch.tensor(table, dtype=torch.int32), "ref": torch.tensor(ref, dtype=torch.int32)}
    return {**out, **_pool64(st)} if c["op"] == "fork" else out
