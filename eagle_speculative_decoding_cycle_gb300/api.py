"""Python binding of the EAGLE cycle library: argument marshalling only.

Every step of prefill, the draft-and-verify cycle and plain decoding runs in the CUDA
library (libeagle.so). PyTorch supplies device memory (weights, the workspace, inputs
and outputs) and the CUDA stream.
"""
from __future__ import annotations

import ctypes as C
import dataclasses
from contextlib import nullcontext
from typing import Dict, List, Optional, Sequence

import torch

from . import _lib as L
from .synth import Workload


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def configs(w: Workload, max_batch: Optional[int] = None, max_ctx: Optional[int] = None,
            prefill_chunk: int = 512, kv_block: Optional[int] = None):
    m = w.model
    mc = L.ModelCfg(m.n_layers, m.hidden, m.n_heads, m.n_kv_heads, m.head_dim, m.ffn, m.vocab,
                    m.rope_theta, m.rms_eps, L.DTYPE_F32 if m.dtype == "f32" else L.DTYPE_BF16)
    dc = L.DrafterCfg(w.drafter.kind, (C.c_int * 3)(*w.drafter.fuse_layers))
    t = w.tree
    tc = L.TreeCfg(t.topk, t.depth, t.m, t.temperature, w.seed, t.planted_p, t.planted_conf)
    if max_ctx is None:
        max_ctx = w.prompt_len[1] + w.new_tokens + 4 * (t.depth + 1) + 16
    lim = L.Limits(max_batch or w.batch, max_ctx, w.kv_block if kv_block is None else kv_block, prefill_chunk)
    return mc, dc, tc, lim


def read_stats(stats: torch.Tensor) -> dict:
    """The fields of an eagle_cycle_stats buffer (copied to the host): counters, and each
    phase's device time in microseconds."""
    raw = stats.detach().to("cpu").contiguous().view(torch.uint8)[:L.STATS_BYTES]
    cnt = raw[:24].view(torch.int32).tolist()
    t = raw[24:].view(torch.int64).tolist()
    out = dict(zip(("batch", "active", "accepted", "committed", "max_accepted", "verify_rows"), cnt))
    out["phase_us"] = {p: (t[i + 1] - t[i]) / 1e3 for i, p in enumerate(L.PHASES)}
    out["cycle_us"] = (t[-1] - t[0]) / 1e3
    return out


class Engine:
    """One context of the cycle library over caller-owned torch CUDA tensors."""

    def __init__(self, w: Workload, weights: Dict[str, torch.Tensor], max_batch: Optional[int] = None,
                 max_ctx: Optional[int] = None, prefill_chunk: int = 512,
                 stream: Optional[torch.cuda.Stream] = None, kv_block: Optional[int] = None):
        self.lib = L.lib()
        self.w = w
        self.k_created = w.tree.topk
        self.weights = weights
        self.stream = stream
        self.mc, self.dc, self.tc, self.lim = configs(w, max_batch, max_ctx, prefill_chunk, kv_block)
        nb = self.lib.eagle_workspace_bytes(C.byref(self.mc), C.byref(self.dc), C.byref(self.tc), C.byref(self.lim))
        if nb == 0:
            raise L.EagleError(L.EAGLE_EINVAL, "invalid configuration")
        dev = next(iter(weights.values())).device
        self.workspace = torch.empty(nb, dtype=torch.uint8, device=dev)
        g = lambda n: _ptr(weights.get(n))
        layers = (L.LayerWeights * w.model.n_layers)()
        for i in range(w.model.n_layers):
            p = f"layers.{i}."
            layers[i] = L.LayerWeights(g(p + "attn_norm"), g(p + "wqkv"), g(p + "wo"), g(p + "mlp_norm"),
                                       g(p + "wgu"), g(p + "wd"))
        self._layers = layers
        draft = L.LayerWeights(g("draft.attn_norm"), g("draft.wqkv"), g("draft.wo"), g("draft.mlp_norm"),
                               g("draft.wgu"), g("draft.wd"))
        self.cw = L.Weights(g("embed"), g("lm_head"), g("final_norm"), layers, g("draft.fc"),
                            g("draft.norm_g"), g("draft.norm_e"), draft)
        h = C.c_void_p()
        rc = self.lib.eagle_create(C.byref(self.mc), C.byref(self.dc), C.byref(self.tc), C.byref(self.cw),
                                   C.byref(self.lim), self.workspace.data_ptr(), nb, _stream(stream), C.byref(h))
        L.check(rc, "eagle_create")
        self.h = h
        self.batch = self.lim.max_batch
        if w.tree.static_parent:
            self.set_static_tree(w.tree.static_parent, w.tree.static_rank)
        self._ref = None
        self._tokens = None

    # -- calls ---------------------------------------------------------------------
    def _check(self, rc: int, what: str) -> None:
        if rc != L.EAGLE_OK:
            raise L.EagleError(rc, f"{what}: {self.lib.eagle_last_error(self.h).decode()}")

    def prefill(self, prompts: Sequence[torch.Tensor], ref: Optional[torch.Tensor] = None) -> None:
        """prompts: int32 CUDA tensors, one per sequence. ref: int32 CUDA [B][ref_len] plain
        continuation (first entry = the prefill token) enabling planted mode, or None."""
        self.batch = len(prompts)
        self._tokens = torch.cat([p.to(torch.int32) for p in prompts]).contiguous()
        lens = (C.c_int32 * self.batch)(*[int(p.numel()) for p in prompts])
        self._ref = None if ref is None else ref.to(torch.int32).contiguous()
        rc = self.lib.eagle_prefill(self.h, self.batch, self._tokens.data_ptr(), lens, _ptr(self._ref),
                                    0 if ref is None else int(self._ref.shape[1]))
        self._check(rc, "eagle_prefill")

    def cycle(self, out_tokens: Optional[torch.Tensor] = None, out_count: Optional[torch.Tensor] = None,
              stats: Optional[torch.Tensor] = None) -> None:
        """One cycle. stats (optional): a device tensor from new_stats(), filled by the device
        with the cycle's statistics (parse with read_stats)."""
        if stats is not None and (stats.numel() * stats.element_size() < L.STATS_BYTES or stats.data_ptr() % 8):
            raise ValueError("stats must be an 8-byte aligned device buffer of at least %d bytes" % L.STATS_BYTES)
        self._check(self.lib.eagle_cycle(self.h, _ptr(out_tokens), _ptr(out_count), _ptr(stats)), "eagle_cycle")

    def new_stats(self) -> torch.Tensor:
        """A device buffer for one cycle's statistics."""
        return torch.zeros(L.STATS_BYTES // 8, dtype=torch.int64, device=self.workspace.device)

    def decode_plain(self, n: int, out: torch.Tensor, margin: Optional[torch.Tensor] = None) -> None:
        self._check(self.lib.eagle_decode_plain(self.h, n, _ptr(out), _ptr(margin)), "eagle_decode_plain")

    def set_stop(self, limits: Sequence[int]) -> None:
        """Per-sequence limits on committed tokens (the prefill token included); an empty list
        removes them. A finished sequence is masked out of later cycles."""
        n = len(limits)
        arr = (C.c_int32 * max(n, 1))(*limits)
        self._check(self.lib.eagle_set_stop(self.h, n, arr), "eagle_set_stop")

    def set_tree_budget(self, topk: int, m: int) -> None:
        """Lower the tree's k and m for the next cycles (at most the created values)."""
        self._check(self.lib.eagle_set_tree_budget(self.h, topk, m), "eagle_set_tree_budget")
        self.w = self.w.replace(tree=dataclasses.replace(self.w.tree, topk=topk, m=m))

    def set_graph(self, on: bool) -> None:
        self._check(self.lib.eagle_set_graph(self.h, int(on)), "eagle_set_graph")

    def set_debug(self, flags: int) -> None:
        self._check(self.lib.eagle_set_debug(self.h, flags), "eagle_set_debug")

    def sync(self) -> None:
        """Wait for the stream and raise on latched device errors."""
        self._check(self.lib.eagle_status_sync(self.h), "eagle_status_sync")

    def profile_begin(self, max_launches: int) -> None:
        self._check(self.lib.eagle_profile_begin(self.h, max_launches), "eagle_profile_begin")

    def profile_end(self):
        """(launches, total device ms, total algorithmic bytes) of the profiled GEMM launches."""
        n, ms, by = C.c_int(), C.c_double(), C.c_double()
        self._check(self.lib.eagle_profile_end(self.h, C.byref(n), C.byref(ms), C.byref(by)), "eagle_profile_end")
        return n.value, ms.value, by.value

    def profile_phases(self):
        """(cycles timed, {phase: total device ms}) of the last profiled window."""
        n, ms = C.c_int(), (C.c_double * len(L.PHASES))()
        self._check(self.lib.eagle_profile_phases(self.h, C.byref(n), ms), "eagle_profile_phases")
        return n.value, dict(zip(L.PHASES, list(ms)))

    def profile_verify(self):
        """(verify passes timed, their total device ms) of the last profiled cycles."""
        n, ms = C.c_int(), C.c_double()
        self._check(self.lib.eagle_profile_verify(self.h, C.byref(n), C.byref(ms)), "eagle_profile_verify")
        return n.value, ms.value

    def ttt_forward(self, tokens: torch.Tensor, steps: int) -> torch.Tensor:
        """EAGLE-3 training-time-test forward over one sequence (int32 CUDA tensor): the mean
        token cross-entropy of each of `steps` self-fed drafter steps (float32 CUDA [steps]).
        Reuses sequence 0's caches; prefill again before cycling."""
        x = tokens.to(torch.int32).contiguous()
        loss = torch.zeros(steps, dtype=torch.float32, device=x.device)
        self._check(self.lib.eagle_ttt_forward(self.h, x.data_ptr(), int(x.numel()), steps, loss.data_ptr()),
                    "eagle_ttt_forward")
        return loss

    def set_static_tree(self, parent: Sequence[int], rank: Sequence[int]) -> None:
        """Static (EAGLE-1) tree of len(parent) == m nodes; an empty topology restores the
        dynamic tree."""
        n = len(parent)
        pa = (C.c_int32 * max(n, 1))(*parent)
        ra = (C.c_int32 * max(n, 1))(*rank)
        self._check(self.lib.eagle_set_static_tree(self.h, n, pa, ra), "eagle_set_static_tree")

    def kv_view(self):
        k, v, cap = C.c_void_p(), C.c_void_p(), C.c_int()
        self._check(self.lib.eagle_kv_view(self.h, C.byref(k), C.byref(v), C.byref(cap)), "eagle_kv_view")
        return k.value, v.value, cap.value

    def kv_table(self):
        """Paged target KV: (device pointer of the int32 block table [max_batch][tab_w], tab_w,
        pool blocks per layer, block size)."""
        t, tw, nb, bs = C.c_void_p(), C.c_int(), C.c_int(), C.c_int()
        self._check(self.lib.eagle_kv_table(self.h, C.byref(t), C.byref(tw), C.byref(nb), C.byref(bs)), "eagle_kv_table")
        return t.value, tw.value, nb.value, bs.value

    def dump_raw(self, what: int) -> torch.Tensor:
        n = self.lib.eagle_dump_bytes(self.h, what)
        buf = torch.empty(n, dtype=torch.uint8, device=self.workspace.device)
        self._check(self.lib.eagle_debug_dump(self.h, what, buf.data_ptr(), n), "eagle_debug_dump")
        return buf

    def dump(self, what: int):
        """Parsed debug view (host tensors)."""
        B = self.batch
        t = self.w.tree
        k, D, T1 = t.topk, t.depth, t.m + 1
        NG = t.n_gen
        raw = self.dump_raw(what).cpu()
        i32 = lambda a, b: raw[a:b].view(torch.int32)
        f32 = lambda a, b: raw[a:b].view(torch.float32)
        if what == L.DUMP_STATE:
            s = i32(0, 7 * B * 4).view(7, B)
            return dict(zip(["ctx_len", "root_tok", "committed", "on_track", "cycle", "acc_len", "bonus"], s))
        if what == L.DUMP_CAND:
            kc = self.k_created
            return i32(0, B * kc * 4).view(B, kc), f32(B * kc * 4, 2 * B * kc * 4).view(B, kc)
        if what == L.DUMP_NODES:
            n = B * NG * 4
            return (i32(0, n).view(B, NG), i32(n, 2 * n).view(B, NG), i32(2 * n, 3 * n).view(B, NG),
                    f32(3 * n, 4 * n).view(B, NG))
        if what == L.DUMP_TREE:
            n = B * T1 * 4
            W = (T1 + 63) // 64
            mask = raw[4 * n:4 * n + B * T1 * W * 8].view(torch.int64).view(B, T1, W)
            return (i32(0, n).view(B, T1), i32(n, 2 * n).view(B, T1), i32(2 * n, 3 * n).view(B, T1),
                    i32(3 * n, 4 * n).view(B, T1), mask)
        if what == L.DUMP_ACCEPT:
            return i32(0, B * 4), i32(B * 4, 2 * B * 4), i32(2 * B * 4, (2 * B + B * D) * 4).view(B, D)
        if what == L.DUMP_VERIFY_HEAD:
            K = 1 if t.temperature > 0 else 2
            R = B * T1
            a = R * K * 4
            return (i32(0, a).view(R, K), f32(a, 2 * a).view(R, K), f32(2 * a, 2 * a + R * 4),
                    f32(2 * a + R * 4, 2 * a + R * 4 + R * k * 4).view(R, k))
        if what == L.DUMP_VERIFY_LOGITS:
            return f32(0, raw.numel()).view(B * T1, self.w.model.vocab)
        if what == L.DUMP_FEATURES:
            dt = torch.float32 if self.w.model.dtype == "f32" else torch.bfloat16
            return raw.view(dt).view(B * T1, self.w.model.hidden)
        if what == L.DUMP_TTT:
            H = self.w.model.hidden
            es = 4 if self.w.model.dtype == "f32" else 2
            R = raw.numel() // (H * es + 4)
            dt = torch.float32 if es == 4 else torch.bfloat16
            return raw[:R * H * es].view(dt).view(R, H), f32(R * H * es, raw.numel())
        raise ValueError(what)

    def close(self) -> None:
        if getattr(self, "h", None):
            self.lib.eagle_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- kernel-level entry points ----------------------------------------------------------------
def _dtype_code(t: torch.Tensor) -> int:
    return L.DTYPE_F32 if t.dtype == torch.float32 else L.DTYPE_BF16


def gemm(W: torch.Tensor, X: torch.Tensor, epi: int = 0, out: Optional[torch.Tensor] = None,
         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Y = X W^T through the library's GEMM (tcgen05 for bf16, FFMA for fp32)."""
    lib = L.lib()
    N, K = W.shape
    M = X.shape[0]
    if epi == 4:            # SwiGLU: W holds [gate; up], the output has half as many features
        N //= 2
    if out is None:
        out = torch.zeros(M, N, dtype=torch.bfloat16 if epi in (1, 4) else torch.float32, device=X.device)
    nb = lib.eagle_op_gemm_scratch_bytes(M, 2 * N if epi == 4 else N)
    scratch = torch.zeros(max(nb, 1), dtype=torch.uint8, device=X.device)
    rc = lib.eagle_op_gemm(_dtype_code(W), _stream(stream), W.data_ptr(), N, K, X.data_ptr(), M, epi,
                           out.data_ptr(), out.stride(0), scratch.data_ptr(), nb)
    L.check(rc, "eagle_op_gemm")
    return out


def lm_head(W: torch.Tensor, X: torch.Tensor, K: int, inv_t: float = 1.0, gumbel: bool = False,
            lse_excl: bool = False, specials: Optional[torch.Tensor] = None,
            row_seq: Optional[torch.Tensor] = None, row_key: Optional[torch.Tensor] = None,
            cycle: int = 0, seed: int = 0, stream_id: int = 4,
            stream: Optional[torch.cuda.Stream] = None):
    """Fused LM head: returns (top_id [M][K], top_val [M][K], lse [M], spec_logit [M][S] or None)."""
    lib = L.lib()
    V, H = W.shape
    M = X.shape[0]
    dev = X.device
    dt = _dtype_code(W)
    nb = lib.eagle_op_lm_head_scratch_bytes(dt, V, M, K)
    scratch = torch.zeros(nb, dtype=torch.uint8, device=dev)
    top_id = torch.empty(M, K, dtype=torch.int32, device=dev)
    top_val = torch.empty(M, K, dtype=torch.float32, device=dev)
    lse = torch.empty(M, dtype=torch.float32, device=dev)
    S = 0 if specials is None else specials.shape[1]
    spec_logit = None if specials is None else torch.full((M, S), float("nan"), device=dev)
    rc = lib.eagle_op_lm_head(dt, _stream(stream), W.data_ptr(), V, H, X.data_ptr(), M, K, inv_t, int(gumbel),
                              int(lse_excl), _ptr(specials), S, _ptr(spec_logit), _ptr(row_seq), _ptr(row_key),
                              cycle, seed, stream_id, top_id.data_ptr(), top_val.data_ptr(), lse.data_ptr(),
                              scratch.data_ptr(), nb)
    L.check(rc, "eagle_op_lm_head")
    return top_id, top_val, lse, spec_logit


def attention(q, kcache, vcache, row_seq, row_slot, ctx_len, rows_per_seq, mode, tree_T=0, mask=None,
              scale=0.0, split_kv: bool = True, stream: Optional[torch.cuda.Stream] = None,
              max_batch: Optional[int] = None) -> torch.Tensor:
    """q [R][nq][d]; caches [B][nkv][cap][d]; returns out [R][nq][d]. max_batch: the caches'
    sequences B (default), which also sets the key-split length of an engine of that batch."""
    lib = L.lib()
    R, nq, d = q.shape
    _, nkv, cap, _ = kcache.shape
    out = torch.empty_like(q)
    mw = 0 if mask is None else mask.shape[1]
    nb = lib.eagle_op_attention_scratch_bytes(R, nq, d) if split_kv else 0
    scratch = torch.empty(max(nb, 1), dtype=torch.uint8, device=q.device)
    rc = lib.eagle_op_attention(_dtype_code(q), _stream(stream), q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(),
                                out.data_ptr(), R, nq, nkv, d, cap, rows_per_seq, row_seq.data_ptr(),
                                row_slot.data_ptr(), ctx_len.data_ptr(), mode, tree_T, _ptr(mask), mw, scale,
                                int(kcache.shape[0]) if max_batch is None else max_batch,
                                scratch.data_ptr() if nb else None, nb)
    L.check(rc, "eagle_op_attention")
    return out


def tree_build(k: int, depth: int, m: int, cand_tok, cand_logc, child_tok, child_logc, ctx_len, root_tok,
               stream: Optional[torch.cuda.Stream] = None):
    """Injected-confidence tree growth + rerank. Returns dict of node and tree tensors."""
    lib = L.lib()
    B = cand_tok.shape[0]
    dev = cand_tok.device
    NG = k + (depth - 1) * k * k
    T1 = m + 1
    W = (T1 + 63) // 64
    o = {n: torch.empty(B, NG, dtype=torch.int32, device=dev) for n in ("node_tok", "node_parent", "node_depth")}
    o["node_logv"] = torch.empty(B, NG, dtype=torch.float32, device=dev)
    for n in ("tree_tok", "tree_pos", "tree_parent", "tree_node"):
        o[n] = torch.empty(B, T1, dtype=torch.int32, device=dev)
    o["tree_mask"] = torch.empty(B, T1, W, dtype=torch.int64, device=dev)
    nb = lib.eagle_op_tree_scratch_bytes(B, k, depth, m)
    scratch = torch.zeros(nb, dtype=torch.uint8, device=dev)
    rc = lib.eagle_op_tree_build(_stream(stream), B, k, depth, m, cand_tok.data_ptr(), cand_logc.data_ptr(),
                                 _ptr(child_tok), _ptr(child_logc), ctx_len.data_ptr(), root_tok.data_ptr(),
                                 o["node_tok"].data_ptr(), o["node_parent"].data_ptr(), o["node_depth"].data_ptr(),
                                 o["node_logv"].data_ptr(), o["tree_tok"].data_ptr(), o["tree_pos"].data_ptr(),
                                 o["tree_parent"].data_ptr(), o["tree_node"].data_ptr(), o["tree_mask"].data_ptr(),
                                 scratch.data_ptr(), nb)
    L.check(rc, "eagle_op_tree_build")
    return o


def compact(kcache, vcache, n_old, acc_len, acc_path, stream: Optional[torch.cuda.Stream] = None) -> None:
    """In-place KV compaction; caches [layers][B][nkv][cap][d]."""
    lib = L.lib()
    layers, B, nkv, cap, d = kcache.shape
    rc = lib.eagle_op_compact(_dtype_code(kcache), _stream(stream), kcache.data_ptr(), vcache.data_ptr(), layers, B,
                              nkv, cap, d, n_old.data_ptr(), acc_len.data_ptr(), acc_path.data_ptr(),
                              acc_path.shape[1])
    L.check(rc, "eagle_op_compact")


def plan_budget(candidates, rows_pts: Sequence[int], verify_us: Sequence[float], batch: int):
    """Batch-aware draft budget (eagle_plan_budget). candidates: list of (k, draft_us,
    exp_tokens) with exp_tokens[m-1] the expected committed tokens of an m-node tree.
    Returns (k, m, tokens per microsecond)."""
    lib = L.lib()
    n_k = len(candidates)
    ks = (C.c_int32 * n_k)(*[c[0] for c in candidates])
    dr = (C.c_float * n_k)(*[c[1] for c in candidates])
    mm = (C.c_int32 * n_k)(*[len(c[2]) for c in candidates])
    flat = [float(v) for c in candidates for v in c[2]]
    ex = (C.c_float * max(1, len(flat)))(*flat)
    rp = (C.c_int32 * len(rows_pts))(*rows_pts)
    vu = (C.c_float * len(verify_us))(*verify_us)
    bk, bm, rate = C.c_int32(), C.c_int32(), C.c_float()
    L.check(lib.eagle_plan_budget(n_k, ks, dr, mm, ex, len(rows_pts), rp, vu, batch, C.byref(bk), C.byref(bm),
                                  C.byref(rate)), "eagle_plan_budget")
    return bk.value, bm.value, rate.value


# ---- 8-bit KV cache -----------------------------------------------------------------------------
def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _elsewhere(index: int) -> bool:
    """Whether another device than the cache's is current: a launch then goes under torch.cuda.device. A cache
    of the CPU (index -1, as of all the CPU's tensors) is refused here."""
    _need(index >= 0, "the cache and its call's tensors must be on a GPU")
    return torch._C._cuda_getDevice() != index


_HERE = nullcontext()


def _owned_by(stream: Optional[torch.cuda.Stream]):
    """New tensors belong to the stream that their kernel runs on: freed early, their memory is not handed to others."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _stream_of(index: int, stream: Optional[torch.cuda.Stream]) -> int:
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


class KV8Cache:
    """One layer's 8-bit KV cache (eagle_kv8) over caller-owned tensors: k, v uint8 e4m3 codes and
    k_exp, v_exp uint8 exponent bytes. Contiguous: [max_batch][nkv][cap][d] and [max_batch][nkv][cap];
    with an int32 block table [max_batch][cap / block]: pools [n_blocks][nkv][block][d] and
    [n_blocks][nkv][block]. The value of a code is code * 2^(byte - 127)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_exp: torch.Tensor, v_exp: torch.Tensor,
                 table: Optional[torch.Tensor] = None):
        for t in (k, v, k_exp, v_exp):
            _need(t.dtype == torch.uint8 and t.is_contiguous() and t.device == k.device,
                  "cache tensors must be contiguous uint8 tensors of one device")
        _need(k.dim() == 4 and k.shape == v.shape and k_exp.shape == k.shape[:3] and v_exp.shape == k.shape[:3],
              "codes must be [B][nkv][cap][d] (or [n_blocks][nkv][block][d]) and exponents the same without d")
        self.k, self.v, self.k_exp, self.v_exp, self.table = k, v, k_exp, v_exp, table
        self.device, self.index = k.device, k.get_device()
        n, self.nkv, slots, self.d = k.shape
        if table is None:
            self.max_batch, self.cap, self.block, self.n_blocks = n, slots, 0, 0
        else:
            _need(table.dtype == torch.int32 and table.dim() == 2 and table.is_contiguous() and
                  table.device == k.device, "table must be a contiguous int32 [max_batch][blocks] tensor")
            self.max_batch, self.cap, self.block, self.n_blocks = table.shape[0], table.shape[1] * slots, slots, n
        self.c = L.KV8(k.data_ptr(), v.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr(), _ptr(table), self.nkv, self.d,
                       self.max_batch, self.cap, self.block, self.n_blocks)
        self.ref = C.byref(self.c)

    @classmethod
    def empty(cls, max_batch: int, nkv: int, cap: int, d: int, device="cuda", block: int = 0,
              n_blocks: Optional[int] = None) -> "KV8Cache":
        """A new cache for max_batch sequences of up to cap slots (rounded up to 16, or to whole
        blocks). block > 0: paged, the table unassigned (-1) and n_blocks pool blocks (default: every
        sequence's worst case)."""
        unit = block or 16
        cap = -(-cap // unit) * unit
        if block:
            n_blocks = max_batch * (cap // block) if n_blocks is None else n_blocks
            table = torch.full((max_batch, cap // block), -1, dtype=torch.int32, device=device)
            shape = (n_blocks, nkv, block, d)
        else:
            table, shape = None, (max_batch, nkv, cap, d)
        new = lambda s: torch.zeros(s, dtype=torch.uint8, device=device)
        return cls(new(shape), new(shape), new(shape[:3]), new(shape[:3]), table)


def _row_list(cache: KV8Cache, t: torch.Tensor, n: int, name: str) -> int:
    if t.dtype is not torch.int32 or t.numel() < n or not t.is_contiguous() or t.get_device() != cache.index:
        raise ValueError(f"{name} must be a contiguous int32 tensor of >= {n} entries on the cache's device")
    return t.data_ptr()


def _err_word(cache: KV8Cache, err: Optional[torch.Tensor]) -> Optional[int]:
    if err is None:
        return None
    _need(err.dtype is torch.int32 and err.numel() >= 1 and err.get_device() == cache.index,
          "err must be an int32 tensor on the cache's device")
    return err.data_ptr()


_KV_TYPES = {torch.float32: L.DTYPE_F32, torch.bfloat16: L.DTYPE_BF16}


def _kv_rows(cache: KV8Cache, k: torch.Tensor, v: torch.Tensor):
    """(rows, type code, row strides) of k and v; a single row's stride is of no account."""
    shape = k.shape
    code = _KV_TYPES.get(k.dtype)
    if code is None or v.dtype is not k.dtype or k.get_device() != cache.index or v.get_device() != cache.index:
        raise ValueError("k and v must be float32 or bfloat16 tensors of one type on the cache's device")
    if len(shape) != 3 or v.shape != shape or shape[1] != cache.nkv or shape[2] != cache.d:
        raise ValueError("k and v must be [R][nkv][d]")
    R, width, ld = shape[0], cache.nkv * cache.d, []
    for t in (k, v):
        s0, s1, s2 = t.stride()
        if R and (s2 != 1 or (s1 != cache.d and cache.nkv != 1)):
            raise ValueError("k and v rows must be contiguous (the row stride is free)")
        ld.append(s0 if R > 1 else width)
    return R, code, ld[0], ld[1]


def kv8_write(cache: KV8Cache, k: torch.Tensor, v: torch.Tensor, row_seq: torch.Tensor, row_slot: torch.Tensor,
              err: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantise rows k, v [R][nkv][d] (fp32 or bf16, any row stride of whole 16 bytes) into slot row_slot[r] of
    sequence row_seq[r] (negative: padding, skipped). err: int32 word that out-of-range rows are latched into."""
    R, code, ldk, ldv = _kv_rows(cache, k, v)
    seq, slot = _row_list(cache, row_seq, R, "row_seq"), _row_list(cache, row_slot, R, "row_slot")
    e = _err_word(cache, err)
    if _elsewhere(cache.index):
        with torch.cuda.device(cache.index):
            return kv8_write(cache, k, v, row_seq, row_slot, err, stream)
    rc = L.lib().eagle_op_kv8_write(_stream_of(cache.index, stream), cache.ref, code, k.data_ptr(), ldk, v.data_ptr(),
                                    ldv, R, seq, slot, e)
    L.check(rc, "eagle_op_kv8_write")


def kv8_read(cache: KV8Cache, row_seq: torch.Tensor, row_slot: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
             out: Optional[Sequence[torch.Tensor]] = None, err: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """Entries (row_seq[r], row_slot[r]) as rows k, v [R][nkv][d] of `dtype` (exact), zeros for padding. out:
    (k, v) to fill, with any row stride of whole 16 bytes."""
    n = row_seq.numel()
    if out is None:
        _need(dtype in _KV_TYPES, "entries are read as float32 or bfloat16")
        with _owned_by(stream):
            k = torch.empty((n, cache.nkv, cache.d), dtype=dtype, device=cache.device)
            v = torch.empty_like(k)
    else:
        k, v = out
    R, code, ldk, ldv = _kv_rows(cache, k, v)
    _need(R == n, "out must have a row for each entry of row_seq")
    seq, slot = _row_list(cache, row_seq, R, "row_seq"), _row_list(cache, row_slot, R, "row_slot")
    e = _err_word(cache, err)
    if _elsewhere(cache.index):
        with torch.cuda.device(cache.index):
            return kv8_read(cache, row_seq, row_slot, dtype, (k, v), err, stream)
    rc = L.lib().eagle_op_kv8_read(_stream_of(cache.index, stream), cache.ref, code, k.data_ptr(), ldk, v.data_ptr(),
                                   ldv, R, seq, slot, e)
    L.check(rc, "eagle_op_kv8_read")
    return k, v


def attention_kv8_scratch(cache: KV8Cache, R: int, nq: int, rows_per_seq: int, prefix_len: int = 0) -> torch.Tensor:
    """Scratch for attention_kv8 / attention_shared_kv8 calls of these sizes (calls that may overlap on the GPU
    need their own)."""
    nb = L.lib().eagle_op_attention_kv8_scratch_bytes(cache.ref, R, nq, rows_per_seq, prefix_len)
    _need(nb > 0, "sizes that the 8-bit attention does not take")
    return torch.empty(nb, dtype=torch.uint8, device=cache.device)


def attention_shared_kv8(q: torch.Tensor, prefix_k: Optional[torch.Tensor], prefix_v: Optional[torch.Tensor],
                         cache: KV8Cache, row_seq: torch.Tensor, row_slot: Optional[torch.Tensor],
                         ctx_len: Optional[torch.Tensor], rows_per_seq: int, mode: int, tree_T: int = 0,
                         mask: Optional[torch.Tensor] = None, scale: float = 0.0, out: Optional[torch.Tensor] = None,
                         scratch: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """attention_kv8 for sequences behind one shared prefix: prefix_k, prefix_v bf16 [nkv][P][d], which every row
    sees before its own slots."""
    shape, index = q.shape, cache.index
    if len(shape) != 3 or shape[2] != cache.d or q.dtype is not torch.bfloat16 or not q.is_contiguous() or \
            q.get_device() != index:
        raise ValueError("q must be a contiguous bfloat16 [R][nq][d] tensor on the cache's device")
    R, nq, d = shape
    P, pk, pv = 0, None, None
    if prefix_k is not None:
        _need(prefix_v is not None and prefix_k.shape == prefix_v.shape, "prefix_k and prefix_v must have one shape")
        for t in (prefix_k, prefix_v):
            _need(t.dtype is torch.bfloat16 and t.is_contiguous() and t.get_device() == index and t.dim() == 3 and
                  t.shape[0] == cache.nkv and t.shape[2] == d,
                  "prefix_k and prefix_v must be contiguous bfloat16 [nkv][P][d] tensors on the cache's device")
        P = prefix_k.shape[1]
        if P:
            pk, pv = prefix_k.data_ptr(), prefix_v.data_ptr()
    seq = _row_list(cache, row_seq, R, "row_seq")
    slot = None if row_slot is None else _row_list(cache, row_slot, R, "row_slot")
    ctx = None if ctx_len is None else _row_list(cache, ctx_len, cache.max_batch, "ctx_len")
    e = _err_word(cache, err)
    mp, mw = None, 0
    if mask is not None:
        _need(mask.dim() == 2 and mask.shape[0] >= R and mask.dtype in (torch.int64, torch.uint64) and
              mask.is_contiguous() and mask.get_device() == index, "mask must be a contiguous 64-bit [R][words] tensor")
        mp, mw = mask.data_ptr(), mask.shape[1]
    if out is None:
        with _owned_by(stream):
            out = torch.empty_like(q)
    else:
        _need(out.shape == shape and out.dtype is torch.bfloat16 and out.is_contiguous() and out.get_device() == index,
              "out must be like q")
    if R == 0:
        return out
    if scratch is None:
        with _owned_by(stream):
            scratch = attention_kv8_scratch(cache, R, nq, rows_per_seq, P)
    if scratch.dtype is not torch.uint8 or not scratch.is_contiguous() or scratch.get_device() != index:
        raise ValueError("scratch must be a contiguous uint8 tensor on the cache's device")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return attention_shared_kv8(q, prefix_k, prefix_v, cache, row_seq, row_slot, ctx_len, rows_per_seq, mode,
                                        tree_T, mask, scale, out, scratch, err, stream)
    rc = L.lib().eagle_op_attention_shared_kv8(
        _stream_of(index, stream), cache.ref, pk, pv, P, q.data_ptr(), out.data_ptr(), R, nq, rows_per_seq, seq, slot,
        ctx, mode, tree_T, mp, mw, scale, scratch.data_ptr(), scratch.numel(), e)
    L.check(rc, "eagle_op_attention_shared_kv8")
    return out


def attention_kv8(q: torch.Tensor, cache: KV8Cache, row_seq: torch.Tensor, row_slot: Optional[torch.Tensor],
                  ctx_len: Optional[torch.Tensor], rows_per_seq: int, mode: int, tree_T: int = 0,
                  mask: Optional[torch.Tensor] = None, scale: float = 0.0, out: Optional[torch.Tensor] = None,
                  scratch: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Tree (mode 1) or causal (mode 0) attention of q [R][nq][d] (bf16) over an 8-bit cache; rows as in
    attention(), padding rows (row_seq < 0) and rows that see nothing give zeros."""
    return attention_shared_kv8(q, None, None, cache, row_seq, row_slot, ctx_len, rows_per_seq, mode, tree_T, mask,
                                scale, out, scratch, err, stream)
