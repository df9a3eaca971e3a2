"""Python-side handle on the native decode step (argument marshalling only).

``Decoder`` owns one ``mk_ctx``: it hands the library raw device pointers of
caller-owned torch tensors (weights, KV pools, step inputs, logits) and the
torch stream to launch on.  All computation happens in ``libmk.so``.
"""

from __future__ import annotations

import ctypes
from ctypes import byref, c_int32, c_void_p
from typing import Dict, Optional, Sequence

import numpy as np
import torch

from . import mk, ops


def _ptr(t: torch.Tensor) -> int:
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


class Decoder:
    """One decode-step engine bound to a model and its paged KV pools."""

    def __init__(self, shape: Dict, weights: Dict, k_pool: torch.Tensor, v_pool: torch.Tensor,
                 max_batch: int, device: int = 0):
        self.shape = dict(shape)
        self.L = shape["n_layers"]
        self.max_batch = max_batch
        self.device = int(device)
        self.n_pages = int(k_pool.shape[1])
        cfg = mk.make_config(shape, max_batch, self.n_pages)
        L = self.L
        keep = []

        def arr(ts):
            a = mk.ptr_array([None if t is None else _ptr(t) for t in ts])
            keep.append(a)
            return a

        t = mk.mk_tensors()
        t.embed = _ptr(weights["embed"])
        t.lm_head = _ptr(weights["lm_head"])
        t.final_norm = _ptr(weights["final_norm"])
        t.attn_norm = arr(weights["attn_norm"])
        t.w_qkv = arr(weights["w_qkv"])
        t.w_o = arr(weights["w_o"])
        t.w_router = arr(weights["w_router"])
        rb = weights.get("router_bias")
        t.router_bias = arr(rb) if rb is not None else None
        t.w_gate = arr(weights["w_gate"])
        t.w_up = arr(weights["w_up"])
        t.w_down = arr(weights["w_down"])
        t.k_pool = arr([k_pool[l] for l in range(L)])
        t.v_pool = arr([v_pool[l] for l in range(L)])
        # of append_kv, made here so that its first call may be captured
        self._inv_freq, _ = ops.rope_frequencies(shape["head_dim"], shape.get("rope_theta", 1.0e4),
                                                 device=k_pool.device)
        self._append_status = ops.Status(k_pool.device)
        self._appended = False                      # some call names that word
        self._tensors = (weights, k_pool, v_pool)   # keep caller tensors alive
        ctx = c_void_p()
        mk.check_status(mk.lib.mk_create(byref(cfg), byref(t), int(device), byref(ctx)),
                        "mk_create")
        self._ctx = ctx
        self.batch = 0
        self.max_pages = 0
        self.planned = []       # cached tokens that the fused steps of the schedule reach, per entry

    # ------------------------------------------------------------------
    def build_schedule(self, seq_lens: Sequence[int], max_pages_per_seq: int,
                       plan_len: Optional[Sequence[int]] = None) -> None:
        B = len(seq_lens)
        sl = mk.int32_array(seq_lens)
        pl = mk.int32_array(plan_len) if plan_len is not None else None
        mk.check_status(mk.lib.mk_build_schedule(self._ctx, B, sl, pl, int(max_pages_per_seq)),
                        "mk_build_schedule")
        self.batch = B
        self.max_pages = int(max_pages_per_seq)
        self.planned = [int(n) for n in plan_len] if plan_len is not None else [int(n) + 64 for n in seq_lens]

    def step(self, tokens: torch.Tensor, positions: torch.Tensor, page_table: torch.Tensor,
             seq_lens: torch.Tensor, logits: torch.Tensor, stream=None,
             unfused: bool = False) -> None:
        for t in (tokens, positions, page_table, seq_lens):
            if t.dtype != torch.int32 or not t.is_cuda:
                raise TypeError("step inputs must be int32 CUDA tensors")
        if logits.dtype != torch.float32 or not logits.is_cuda:
            raise TypeError("logits must be a float32 CUDA tensor")
        if page_table.shape[-1] != self.max_pages:
            raise ValueError("page_table row length differs from the schedule's")
        s = stream if stream is not None else torch.cuda.current_stream()
        fn = mk.lib.mk_decode_step_unfused if unfused else mk.lib.mk_decode_step
        st = fn(self._ctx, _ptr(tokens), _ptr(positions), _ptr(page_table), _ptr(seq_lens),
                _ptr(logits), c_void_p(s.cuda_stream))
        mk.check_status(st, "mk_decode_step")

    def greedy(self, n_steps: int, tokens: torch.Tensor, positions: torch.Tensor,
               page_table: torch.Tensor, seq_lens: torch.Tensor, logits: torch.Tensor,
               out_tokens: torch.Tensor, stream=None) -> None:
        """n_steps greedy steps on the device (mk_decode_greedy): tokens,
        positions and seq_lens are updated in place, out_tokens[i] receives
        step i's tokens.  Asynchronous."""
        for t in (tokens, positions, page_table, seq_lens, out_tokens):
            if t.dtype != torch.int32 or not t.is_cuda:
                raise TypeError("greedy inputs and outputs must be int32 CUDA tensors")
        if logits.dtype != torch.float32 or not logits.is_cuda:
            raise TypeError("logits must be a float32 CUDA tensor")
        if page_table.shape[-1] != self.max_pages:
            raise ValueError("page_table row length differs from the schedule's")
        if out_tokens.numel() < n_steps * self.batch:
            raise ValueError("out_tokens holds fewer than n_steps x batch tokens")
        s = stream if stream is not None else torch.cuda.current_stream()
        st = mk.lib.mk_decode_greedy(self._ctx, int(n_steps), _ptr(tokens), _ptr(positions),
                                     _ptr(page_table), _ptr(seq_lens), _ptr(logits),
                                     _ptr(out_tokens), c_void_p(s.cuda_stream))
        mk.check_status(st, "mk_decode_greedy")

    def _holds(self, name: str, t: torch.Tensor, dtype, size: int) -> None:
        """A tensor that the device reads or writes `size` values of."""
        if t.dtype != dtype or t.get_device() != self.device:
            raise TypeError(f"{name} must be a {str(dtype)[6:]} tensor on cuda:{self.device}")
        if t.numel() < size:
            raise ValueError(f"{name} holds fewer than {size} values")

    def _step_inputs(self, tokens, positions, page_table, seq_lens, logits) -> None:
        for name, t in (("tokens", tokens), ("positions", positions), ("seq_lens", seq_lens)):
            self._holds(name, t, torch.int32, self.batch)
        if page_table.shape[-1] != self.max_pages:
            raise ValueError("page_table row length differs from the schedule's")
        self._holds("page_table", page_table, torch.int32, self.batch * self.max_pages)
        self._holds("logits", logits, torch.float32, self.batch * self.shape["vocab"])

    def _stream(self, stream):
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        if s.device_index != self.device:
            raise ValueError(f"stream must be of cuda:{self.device}")
        return s

    def _groups(self, group_start: torch.Tensor, prefix_lens: torch.Tensor) -> int:
        self._holds("group_start", group_start, torch.int32, 0)
        self._holds("prefix_lens", prefix_lens, torch.int32, 0)
        n = prefix_lens.numel()
        if not 1 <= n <= self.batch or group_start.numel() != n + 1:
            raise ValueError("need 1 .. batch prefix lengths and one more group start")
        return n

    def step_shared(self, tokens: torch.Tensor, positions: torch.Tensor, page_table: torch.Tensor,
                    seq_lens: torch.Tensor, group_start: torch.Tensor, prefix_lens: torch.Tensor,
                    logits: torch.Tensor, stream=None) -> None:
        """One step of a batch whose entries share prefixes (mk_decode_step_shared):
        group g is entries group_start[g] .. group_start[g + 1] - 1, whose first
        prefix_lens[g] tokens are read through the first entry's page-table row."""
        self._step_inputs(tokens, positions, page_table, seq_lens, logits)
        n = self._groups(group_start, prefix_lens)
        s = self._stream(stream)
        st = mk.lib.mk_decode_step_shared(
            self._ctx, _ptr(tokens), _ptr(positions), _ptr(page_table), _ptr(seq_lens), n,
            _ptr(group_start), _ptr(prefix_lens), _ptr(logits), c_void_p(s.cuda_stream))
        mk.check_status(st, "mk_decode_step_shared")

    def sample(self, n_steps: int, tokens: torch.Tensor, positions: torch.Tensor,
               page_table: torch.Tensor, seq_lens: torch.Tensor, logits: torch.Tensor,
               out_tokens: torch.Tensor, u: torch.Tensor, *,
               temperature: Optional[torch.Tensor] = None, top_k: Optional[torch.Tensor] = None,
               top_p: Optional[torch.Tensor] = None, min_p: Optional[torch.Tensor] = None,
               logprobs: Optional[torch.Tensor] = None,
               group_start: Optional[torch.Tensor] = None,
               prefix_lens: Optional[torch.Tensor] = None, stream=None) -> None:
        """n_steps sampled steps on the device (mk_decode_sample): as ``greedy``,
        with step i's tokens drawn by the uniform numbers u[i] under the rules of
        ``ops.sample``; with group_start and prefix_lens the steps are those of
        ``step_shared``.  logprobs, if given, receives n_steps x batch
        log-probabilities.  Asynchronous."""
        self._step_inputs(tokens, positions, page_table, seq_lens, logits)
        self._holds("out_tokens", out_tokens, torch.int32, n_steps * self.batch)
        how = mk.mk_sampling()
        for name, t, dtype, size in (
                ("u", u, torch.float32, n_steps * self.batch),
                ("temperature", temperature, torch.float32, self.batch),
                ("top_k", top_k, torch.int32, self.batch),
                ("top_p", top_p, torch.float32, self.batch),
                ("min_p", min_p, torch.float32, self.batch),
                ("logprobs", logprobs, torch.float32, n_steps * self.batch)):
            if t is None:
                continue
            self._holds(name, t, dtype, size)
            setattr(how, name, _ptr(t))
        if (group_start is None) != (prefix_lens is None):
            raise ValueError("group_start and prefix_lens go together")
        if group_start is not None:
            how.n_groups = self._groups(group_start, prefix_lens)
            how.group_start, how.prefix_lens = _ptr(group_start), _ptr(prefix_lens)
        s = self._stream(stream)
        st = mk.lib.mk_decode_sample(self._ctx, int(n_steps), _ptr(tokens), _ptr(positions),
                                     _ptr(page_table), _ptr(seq_lens), _ptr(logits),
                                     _ptr(out_tokens), byref(how), c_void_p(s.cuda_stream))
        mk.check_status(st, "mk_decode_sample")

    def append_kv(self, layer: int, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                  page_table: torch.Tensor, seq: Optional[torch.Tensor] = None,
                  status: Optional["ops.Status"] = None, stream=None) -> None:
        """Rotate a layer's keys and append them with their values to the cache
        that the steps read (``ops.rope_append``): a prompt that was computed
        outside the step, handed over in one piece.  k and v are [tokens][kv
        heads][head size] before the rotation; the other arguments are
        ``ops.rope_append``'s.  Without a ``status`` of its own, a call's fault is
        the decoder's: the next ``check`` reports it."""
        _, k_pool, v_pool = self._tensors
        if status is None:
            status, self._appended = self._append_status, True
        ops.rope_append(None, k, v, positions, page_table, k_pool[layer], v_pool[layer],
                        self._inv_freq, seq=seq, status=status, stream=stream)

    def check(self):
        """Synchronize and return (status, detail list): of the steps, and where
        they are clean of the ``append_kv`` calls since the last check."""
        st = c_int32(0)
        detail = (c_int32 * 8)()
        rc = mk.lib.mk_check(self._ctx, byref(st), detail)
        if rc == mk.MK_OK and self._appended:
            rc, where = self._append_status.check()
            if rc != mk.MK_OK:
                return rc, [rc] + where + [0] * 3
        return int(rc), [int(v) for v in detail]

    def check_ok(self) -> None:
        rc, detail = self.check()
        if rc != mk.MK_OK:
            raise mk.MKError(rc, "device status", detail)

    def selftest_timeout(self, timeout_ms: int = 10):
        """Run the failure-detection self-test; returns (status, detail list)."""
        st = c_int32(0)
        detail = (c_int32 * 8)()
        rc = mk.lib.mk_selftest_timeout(self._ctx, int(timeout_ms), byref(st), detail)
        return int(rc), [int(v) for v in detail]

    def set_trace(self, enable: bool) -> None:
        mk.check_status(mk.lib.mk_set_trace(self._ctx, int(bool(enable))), "mk_set_trace")

    def trace(self):
        """(desc [n_tasks][32], trace [n_tasks][18]) of the last traced step."""
        desc = self.debug(mk.MK_BUF_PLAN).reshape(-1, 32)
        stamps = self.debug(mk.MK_BUF_TRACE).reshape(-1, mk.TRACE_WORDS)
        return desc, stamps

    def set_timeout_ms(self, ms: int) -> None:
        mk.check_status(mk.lib.mk_set_timeout_ms(self._ctx, int(ms)), "mk_set_timeout_ms")

    def debug(self, which: int) -> np.ndarray:
        n = mk.lib.mk_debug_size(self._ctx, which)
        if n == 0:
            raise mk.MKError(mk.MK_ERR_STATE, "mk_debug_size")
        ints = (mk.MK_BUF_TOPK, mk.MK_BUF_NSLOTS, mk.MK_BUF_PLAN)
        dtype = np.int32 if which in ints else (np.uint32 if which == mk.MK_BUF_TRACE
                                                else np.float32)
        out = np.empty(n // 4, dtype=dtype)
        mk.check_status(mk.lib.mk_debug_read(self._ctx, which, out.ctypes.data_as(c_void_p), n),
                        "mk_debug_read")
        return out

    def close(self) -> None:
        if getattr(self, "_ctx", None):
            mk.lib.mk_destroy(self._ctx)
            self._ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def plan_schedule(shape: Dict, n_ctas: int, seq_lens: Sequence[int],
                  plan_len: Optional[Sequence[int]] = None, max_batch: int = 8,
                  n_pages: int = 1 << 20):
    """Host-only planner (no GPU): returns (meta, desc [n_tasks][32], targets)."""
    cfg = mk.make_config(shape, max_batch, n_pages)
    B = len(seq_lens)
    sl = mk.int32_array(seq_lens)
    pl = mk.int32_array(plan_len) if plan_len is not None else None
    meta = (c_int32 * 16)()
    mk.check_status(mk.lib.mk_plan_schedule(byref(cfg), n_ctas, B, sl, pl, meta, None, None),
                    "mk_plan_schedule")
    m = [int(v) for v in meta]
    n_tasks, n_counters = m[0], m[1]
    desc = np.zeros((n_tasks, 32), dtype=np.int32)
    targets = np.zeros(n_counters, dtype=np.int32)
    P = ctypes.POINTER(c_int32)
    mk.check_status(mk.lib.mk_plan_schedule(byref(cfg), n_ctas, B, sl, pl, meta,
                                            desc.ctypes.data_as(P), targets.ctypes.data_as(P)),
                    "mk_plan_schedule")
    return m, desc, targets
