"""Serving operators beside the decode step: appending rotated keys and values
to the paged cache, attention over prefixes that batch entries share, and
sampling.

Each function checks its arguments, hands raw device pointers to ``libmk.so``
and returns after the launch; all computation happens in the library's
kernels.  Tensors live on one CUDA device, which need not be the current one;
``stream`` is a torch stream of that device (its current stream by default).
Outputs that a function allocates are made and cleared on that stream; tensors
that the caller passes have to be ready there, and to live until it has used them.
A call keeps nothing: it may be captured into a graph, and calls on other
streams may overlap it as long as they write other tensors.
"""

from __future__ import annotations

import functools
import math
import struct
from typing import Optional

import torch

from . import mk

PAGE = 64

_TYPE = {torch.float32: mk.MK_FP32, torch.bfloat16: mk.MK_BF16, torch.float16: mk.MK_FP16}
_POOL = (torch.bfloat16, torch.float16)
_I32, _F32, _F64 = torch.int32, torch.float32, torch.float64
_OPS = {mk.MK_OP_ROPE_APPEND: "rope_append", mk.MK_OP_PREFIX_ATTENTION: "prefix_attention",
        mk.MK_OP_SAMPLE: "sample"}


class Status:
    """Device word that latches the first device-side fault of the calls that
    name it (``status=``): a page id, position or parameter out of range.  Calls
    on any stream may name it, captured ones too; it is made outside a capture."""

    def __init__(self, device):
        self.word = torch.zeros(8, dtype=_I32, device=device)
        # cleared before any stream's call can name it
        torch.cuda.current_stream(self.word.device).synchronize()

    def check(self, stream=None):
        """Wait for the device's work (with ``stream``: for that stream's alone),
        read and clear: (status, [operator, entry, value, limit])."""
        if stream is None:
            torch.cuda.synchronize(self.word.device)
            stream = torch.cuda.current_stream(self.word.device)
        with torch.cuda.stream(stream):
            w = self.word.tolist()
            if w[0] != mk.MK_OK:
                self.word.zero_()
                stream.synchronize()
        return w[0], w[1:5]

    def check_ok(self, stream=None) -> None:
        rc, detail = self.check(stream)
        if rc != mk.MK_OK:
            raise mk.MKError(rc, _OPS.get(detail[0], "device status"), detail)


# The calls below are as short as a decode step's, and so are their checks:
# devices are compared by number, and the arguments are packed in one go in the
# layout of the C structs (fields as in mk.mk_*_args).
_PACK_APPEND = struct.Struct("@12if3P6q8P").pack
_PACK_ATTENTION = struct.Struct("@9ifPq9PNP").pack
_PACK_SAMPLE = struct.Struct("@4iPq8P").pack
_raw_stream = torch._C._cuda_getCurrentRawStream


def _array(t: torch.Tensor, dtype, name: str, dev: int, shape) -> int:
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be a {str(dtype)[6:]} tensor on cuda:{dev}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}")
    return t.data_ptr()


def _cuda(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return dev


@functools.lru_cache(maxsize=None)
def _workspace_size(batch: int, hq: int, hkv: int, hd: int) -> int:
    """mk_prefix_attention_workspace, which goes by these sizes alone."""
    return mk.lib.mk_prefix_attention_workspace(_PACK_ATTENTION(
        0, batch, 1, 1, 1, hq, hkv, hd, mk.MK_BF16, 1.0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0))


def _stream(stream, dev: int) -> int:
    """The stream's handle.  Without one, the current stream of the device."""
    if stream is None:
        return _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream must be of cuda:{dev}")
    return stream.cuda_stream


def _output(make, shape, dtype, device, stream) -> torch.Tensor:
    """An output of the caller's, made (and filled) on the call's stream: its
    memory is that stream's, and so is the order of filling and kernel.  The
    caller's current stream is noted, which may use it when the call's is past it."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _status(status: Optional[Status], dev: int) -> int:
    if status is None:
        return 0
    if status.word.get_device() != dev:
        raise ValueError(f"status must be on cuda:{dev}")
    return status.word.data_ptr()


def _pools(k_pool: torch.Tensor, v_pool: torch.Tensor, dev: int):
    """Checks one layer's pools; returns their type and shape (pages, heads, head size)."""
    dtype, shape = k_pool.dtype, k_pool.shape
    if dtype not in _POOL or v_pool.dtype is not dtype:
        raise TypeError("k_pool and v_pool must both be bfloat16 or both float16")
    if k_pool.get_device() != dev or v_pool.get_device() != dev:
        raise TypeError(f"k_pool and v_pool must be on cuda:{dev}")
    if len(shape) != 4 or v_pool.shape != shape or shape[2] != PAGE or shape[3] not in (64, 128):
        raise ValueError("k_pool and v_pool must be [pages][kv heads][64][64 or 128]")
    if not k_pool.is_contiguous() or not v_pool.is_contiguous():
        raise ValueError("k_pool and v_pool must be contiguous")
    return dtype, shape[0], shape[1], shape[3]


def rope_frequencies(rotary_dim: int, theta: float = 1.0e4, *, scaling: Optional[str] = None,
                     factor: float = 1.0, trained_len: int = 4096, slow_turns: float = 1.0,
                     fast_turns: float = 32.0, device="cuda"):
    """The angle per position of each rotated pair, float64[rotary_dim / 2],
    and the factor of cosine and sine: the ``inv_freq`` and ``magnitude`` of
    ``rope_append``.  Pair i turns by theta^(-2 i / rotary_dim) per position.

    scaling stretches a model trained on ``trained_len`` positions by ``factor``:
    None: not at all; "even": every angle divided by factor; "base": theta
    raised so that the slowest pair is divided by factor and the fastest kept;
    "parts": pairs that turn at least ``fast_turns`` times over trained_len
    are kept, those that turn at most ``slow_turns`` times divided by factor,
    those between blended linearly in their number of turns, with magnitude
    0.1 ln(factor) + 1.  (A model trained with a blend that is linear in the pair's
    index, as some are, needs its own table: any float64 tensor will do.)"""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    if not (theta > 0 and factor >= 1.0):
        raise ValueError("theta must be positive and factor at least 1")
    n = rotary_dim // 2
    magnitude = 1.0
    if scaling == "base" and n > 1:
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2))
    f = [theta ** (-2.0 * i / rotary_dim) for i in range(n)]
    if scaling == "even":
        f = [x / factor for x in f]
    elif scaling == "parts":
        if not fast_turns > slow_turns:
            raise ValueError("fast_turns must exceed slow_turns")
        keep = [min(1.0, max(0.0, (trained_len * x / (2.0 * math.pi) - slow_turns)
                             / (fast_turns - slow_turns))) for x in f]
        f = [x * k + x / factor * (1.0 - k) for x, k in zip(f, keep)]
        magnitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'even', 'base' or 'parts'")
    return torch.tensor(f, dtype=torch.float64, device=device), magnitude


def rope_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                positions: torch.Tensor, page_table: torch.Tensor, k_pool: torch.Tensor,
                v_pool: torch.Tensor, inv_freq: torch.Tensor, *,
                seq: Optional[torch.Tensor] = None, interleaved: bool = False,
                magnitude: float = 1.0, q_out: Optional[torch.Tensor] = None,
                status: Optional[Status] = None, stream=None) -> Optional[torch.Tensor]:
    """Rotate keys and append them with their values to one layer's paged
    cache; rotate queries on the way (mk_rope_append).

    q [tokens][query heads][hd] or None, k and v [tokens][kv heads][hd] (any
    strides, columns adjacent) of float32, bfloat16 or float16; k_pool and
    v_pool [pages][kv heads][64][hd] of bfloat16 or float16, written in place;
    positions int32[tokens]; page_table int32[rows][pages per row]; seq
    int32[tokens], each token's row (-1: padding, left out), or None: token t
    is row t.  inv_freq float64[rotary_dim / 2] and magnitude as from
    ``rope_frequencies``.  Returns q_out ([tokens][query heads][hd] of the
    pools' type; allocated if None, may be q itself), None without queries.  Rows
    of padding, and of tokens whose place is at fault, are left as they were:
    zero in a q_out that is allocated here (one that is passed saves the clearing)."""
    dev = _cuda(k, "k")
    handle = _stream(stream, dev)
    pool, n_pages, hkv, hd = _pools(k_pool, v_pool, dev)
    dtype, shape = k.dtype, k.shape
    t = shape[0]
    if dtype not in _TYPE or v.dtype is not dtype or v.get_device() != dev:
        raise TypeError("k and v must have the same type (float32, bfloat16 or float16) and device")
    if shape != (t, hkv, hd) or v.shape != shape:
        raise ValueError(f"k and v must be [tokens][{hkv}][{hd}]")
    ks, vs = k.stride(), v.stride()
    if t and (ks[2] != 1 or vs[2] != 1):
        raise ValueError("the columns of k and v must be adjacent")
    hq, qs, q_at, out_at = 0, (0, 0, 1), 0, 0
    if q is not None:
        shape = q.shape
        hq = shape[1] if len(shape) == 3 else 0
        if shape != (t, hq, hd) or hq < 1:
            raise ValueError(f"q must be [tokens][query heads][{hd}]")
        if q.dtype is not dtype or q.get_device() != dev:
            raise TypeError("q must have the type and device of k")
        qs = q.stride()
        if t and qs[2] != 1:
            raise ValueError("the columns of q must be adjacent")
        if q_out is None:
            q_out = _output(torch.zeros, (t, hq, hd), pool, q.device, stream)
        elif (q_out.shape != shape or not q_out.is_contiguous() or q_out.dtype is not pool
              or q_out.get_device() != dev):
            raise ValueError("q_out must be contiguous, shaped like q and of the pools' type and device")
        q_at, out_at = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if inv_freq.dtype is not _F64 or inv_freq.get_device() != dev or not inv_freq.is_contiguous():
        raise TypeError(f"inv_freq must be a contiguous float64 tensor on cuda:{dev}")
    freqs = inv_freq.numel()
    if inv_freq.dim() != 1 or 2 * freqs > hd:
        raise ValueError(f"inv_freq must hold at most {hd // 2} frequencies")
    table = page_table.shape
    if len(table) != 2:
        raise ValueError("page_table must be [rows][pages per row]")
    if seq is None and t > table[0]:
        raise ValueError("more tokens than page-table rows, and no seq")
    a = _PACK_APPEND(
        dev, t, table[0], table[1], n_pages, hq, hkv, hd, 2 * freqs, 1 if interleaved else 0, _TYPE[dtype],
        _TYPE[pool], magnitude, q_at, k.data_ptr(), v.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
        out_at, k_pool.data_ptr(), v_pool.data_ptr(), inv_freq.data_ptr(),
        _array(positions, _I32, "positions", dev, (t,)), 0 if seq is None else _array(seq, _I32, "seq", dev, (t,)),
        _array(page_table, _I32, "page_table", dev, table), _status(status, dev))
    if t:
        rc = mk.lib.mk_rope_append(a, handle)
        if rc:
            raise mk.MKError(rc, "mk_rope_append")
    return q_out


def prefix_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                     page_table: torch.Tensor, positions: torch.Tensor,
                     group_start: torch.Tensor, prefix_lens: torch.Tensor, *,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, status: Optional[Status] = None,
                     stream=None) -> torch.Tensor:
    """Attention of one query token per batch entry over the paged cache, shared
    prefixes read once for many entries of a group (mk_prefix_attention).

    q [batch][query heads][hd] of the pools' type; positions int32[batch]: entry
    b attends to tokens 0 .. positions[b] of its sequence (-1: to none, output
    zero); group g is entries group_start[g] .. group_start[g + 1] - 1, whose
    first prefix_lens[g] tokens are read through the first entry's page-table
    row; entries of no group keep their rows of out and lse.  A batch of one
    sequence's tokens at increasing positions under a prefix that covers them
    all is a causal piece of a prompt.  scale: factor of the scores, 1 /
    sqrt(hd) by default.  Returns out (allocated if None: entries of no group
    are then zero); lse, if given, float32[batch][query heads], receives the log
    of each row's sum of exponentials."""
    dev = _cuda(q, "q")
    handle = _stream(stream, dev)
    dtype, n_pages, hkv, hd = _pools(k_pool, v_pool, dev)
    shape = q.shape
    if len(shape) != 3 or shape[2] != hd:
        raise ValueError(f"q must be [batch][query heads][{hd}]")
    b, hq, _ = shape
    if q.dtype is not dtype:
        raise TypeError("q must have the pools' type")
    qs = q.stride()
    rows = qs[0] if b > 1 else hq * hd               # a stride that no element uses may be anything
    if b and (qs[2] != 1 or (qs[1] != hd and hq > 1) or rows % 8):
        raise ValueError("q's heads must be adjacent and its token stride a multiple of 8")
    if hq < 1 or hq % hkv:
        raise ValueError("query heads must be a multiple of the kv heads")
    if page_table.dim() != 2 or prefix_lens.dim() != 1:
        raise ValueError("page_table must be [batch][pages per row], group_start and prefix_lens flat")
    n, pages = prefix_lens.shape[0], page_table.shape[1]
    if out is None:
        out = _output(torch.zeros, shape, dtype, q.device, stream)
    elif (out.shape != shape or not out.is_contiguous() or out.dtype is not dtype
          or out.get_device() != dev):
        raise ValueError("out must be contiguous with q's shape, type and device")
    if b == 0 or n == 0:
        return out
    # the workspace is this call's own; torch hands its memory on in stream order
    size = _workspace_size(b, hq, hkv, hd)
    if stream is None:
        work = q.new_empty(size, dtype=torch.uint8)
    else:
        with torch.cuda.stream(stream):
            work = q.new_empty(size, dtype=torch.uint8)
    a = _PACK_ATTENTION(
            dev, b, n, pages, n_pages, hq, hkv, hd, _TYPE[dtype],
            1.0 / math.sqrt(hd) if scale is None else scale, q.data_ptr(), rows, k_pool.data_ptr(),
            v_pool.data_ptr(), _array(page_table, _I32, "page_table", dev, (b, pages)),
            _array(positions, _I32, "positions", dev, (b,)),
            _array(group_start, _I32, "group_start", dev, (n + 1,)),
            _array(prefix_lens, _I32, "prefix_lens", dev, (n,)), out.data_ptr(),
            0 if lse is None else _array(lse, _F32, "lse", dev, (b, hq)), work.data_ptr(), size,
            _status(status, dev))
    rc = mk.lib.mk_prefix_attention(a, handle)
    if rc:
        raise mk.MKError(rc, "mk_prefix_attention")
    return out


def sample(logits: torch.Tensor, u: torch.Tensor, *, temperature: Optional[torch.Tensor] = None,
           top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
           min_p: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
           logprobs: Optional[torch.Tensor] = None, status: Optional[Status] = None,
           stream=None) -> torch.Tensor:
    """Draw one token per row of logits from given uniform numbers (mk_sample).

    logits [batch][vocab] of float32, bfloat16 or float16 (columns adjacent);
    u float32[batch] in [0, 1).  temperature, top_p, min_p float32[batch] and
    top_k int32[batch] are each optional.  The kept tokens are those of the
    top_k largest logits whose preceding probability, among these, is below
    top_p, and whose probability is at least min_p of the largest; the drawn
    one is the first, by ascending id, at which their running probability
    passes u.  temperature 0 picks the largest logit.  Returns tokens
    int32[batch] (allocated if None; -1 where a row has nothing to draw);
    logprobs, if given, float32[batch], receives each drawn token's log-probability
    among the kept ones."""
    dev = _cuda(logits, "logits")
    handle = _stream(stream, dev)
    kind = _TYPE.get(logits.dtype)
    if kind is None:
        raise TypeError("logits must be float32, bfloat16 or float16")
    shape = logits.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError("logits must be [batch][vocab]")
    b, v = shape
    ls = logits.stride()
    if b and ls[1] != 1 and v > 1:
        raise ValueError("the columns of logits must be adjacent")
    rows = (b,)
    if tokens is None:
        tokens = _output(torch.empty, rows, _I32, logits.device, stream)
    a = _PACK_SAMPLE(
        dev, b, v, kind, logits.data_ptr(), ls[0], _array(u, _F32, "u", dev, rows),
        0 if temperature is None else _array(temperature, _F32, "temperature", dev, rows),
        0 if top_k is None else _array(top_k, _I32, "top_k", dev, rows),
        0 if top_p is None else _array(top_p, _F32, "top_p", dev, rows),
        0 if min_p is None else _array(min_p, _F32, "min_p", dev, rows),
        _array(tokens, _I32, "tokens", dev, rows),
        0 if logprobs is None else _array(logprobs, _F32, "logprobs", dev, rows), _status(status, dev))
    if b:
        rc = mk.lib.mk_sample(a, handle)
        if rc:
            raise mk.MKError(rc, "mk_sample")
    return tokens
