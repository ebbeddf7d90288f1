"""B200-native TriAttention KV-cache key scoring, top-B selection and compaction.

A thin binding over ``libtri.so`` (C ABI in ``include/tri.h``): the functions
below only marshal torch tensors into pointers and sizes; every step of the
computation runs in the library's sm_100a CUDA kernels.  Importing the package
fails if the library has not been built (``build.py``) - there is no other
implementation to fall back to.

Method: "TriAttention：基于三角函数 KV 压缩的高效长推理" (whatsmy.fun paper
digest), section 流程详解 steps 1-4 - calibrate pre-RoPE query centres, score
each cached key by a trigonometric series in its RoPE distance plus a norm
term, keep the top keys per KV head, compact the cache.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._abi import (TRI_ELEM_BF16, TRI_ELEM_FP8_E4M3, TRI_FLAG_BLOCK_TABLE,  # noqa: F401
                   TRI_FLAG_NONFINITE, TRI_FLAG_ROW_OFFSETS, TRI_FLAG_STAGE_TIMEOUT,
                   TRI_KEYS_POST_ROPE, TRI_KEYS_PRE_ROPE, TRI_KV_CONTIG, TRI_KV_PAGED,
                   TRI_MAX_OFFSETS, TRI_ROPE_HALF, TRI_ROPE_INTERLEAVED, TriKvDesc, TriModel, TriOutDesc, TriTokenDesc)

_L = _abi.load()


class TriError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {_L.tri_status_str(status).decode()}"
        if status == _abi.TRI_ERR_CUDA:
            msg += f" [{_L.tri_last_error().decode()}]"
        super().__init__(msg)


def _check(st: int, what: str) -> None:
    if st != _abi.TRI_OK:
        raise TriError(st, what)


def _p(t):
    """Device pointer of a tensor argument (None -> NULL).  Every tensor the library
    reads or writes must be a contiguous CUDA tensor: a host pointer handed to a
    kernel would fault, a strided view would be read as if it were dense."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor (call .contiguous())")
    return ctypes.c_void_p(t.data_ptr())


def _pd(t):
    """Pointer of a tensor the gather reads or writes record by record (V and the
    compacted outputs): a contiguous CUDA tensor, or a contiguous page-locked host
    tensor, which the device addresses at the same pointer under unified
    addressing - the kept records then cross the host link directly.  Pageable
    host memory is refused: the device cannot address it."""
    if t is not None and not t.is_cuda:
        if not t.is_pinned():
            raise ValueError("expected a CUDA tensor or a pinned (page-locked) host tensor")
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor (call .contiguous())")
        return ctypes.c_void_p(t.data_ptr())
    return _p(t)


def _s(stream):
    if stream is None:
        if torch.cuda.is_initialized():  # the handle itself: a Stream object costs more than some kernels
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def version() -> int:
    return int(_L.tri_version())


def library_path() -> str:
    return _abi.LIB_PATH


# ------------------------------------------------------------- descriptors

def model(n_layers: int, n_q_heads: int, n_kv_heads: int, rope_theta: float,
          head_dim: int = 128, rope_style: int = TRI_ROPE_HALF) -> TriModel:
    """Model shape; ``rope_style`` TRI_ROPE_HALF pairs dims (f, f+d/2), TRI_ROPE_INTERLEAVED (2f, 2f+1)."""
    return TriModel(head_dim, n_layers, n_q_heads, n_kv_heads, float(rope_theta), int(rope_style), 0)


# A descriptor holds raw device pointers; it also keeps a reference to the tensors
# they point into, so the memory cannot be freed (and reused) while it is alive.

def elem_type_of(t: torch.Tensor) -> int:
    """TRI_ELEM_* of a K/V tensor (bf16 or float8_e4m3fn)."""
    if t.dtype == torch.bfloat16:
        return TRI_ELEM_BF16
    if t.dtype == torch.float8_e4m3fn:
        return TRI_ELEM_FP8_E4M3
    raise TypeError(f"unsupported K/V dtype {t.dtype}")


def kv_contig(n_seqs: int, row_off: torch.Tensor, total_keys: int,
              elem_type: int = TRI_ELEM_BF16) -> TriKvDesc:
    """Rows laid end to end; ``row_off`` int64 [R+1] on the device."""
    d = TriKvDesc(TRI_KV_CONTIG, n_seqs, int(total_keys), _p(row_off).value, None, 0, 0, 0,
                  int(elem_type), 0)
    d._keep, d._held = (row_off,), (row_off.numel(), n_seqs, row_off.get_device())
    return d


def kv_paged(n_seqs: int, row_off: torch.Tensor, total_keys: int, block_table: torch.Tensor,
             block_size: int, n_blocks: int, elem_type: int = TRI_ELEM_BF16) -> TriKvDesc:
    """vLLM block layout; ``block_table`` int32 [S][max_blocks] on the device."""
    d = TriKvDesc(TRI_KV_PAGED, n_seqs, int(total_keys), _p(row_off).value,
                  _p(block_table).value, block_table.shape[1], block_size, int(n_blocks),
                  int(elem_type), 0)
    if row_off.device != block_table.device:
        raise ValueError("kv_paged: row_off and block_table on different devices")
    d._keep, d._held = (row_off, block_table), (row_off.numel(), block_table.shape[0], row_off.get_device())
    return d


def out_contig() -> TriOutDesc:
    return TriOutDesc(TRI_KV_CONTIG, 0, None, 0, 0, 0)


def out_paged(block_table: torch.Tensor, block_size: int, n_blocks: int) -> TriOutDesc:
    d = TriOutDesc(TRI_KV_PAGED, block_table.shape[1], _p(block_table).value, block_size, 0,
                   int(n_blocks))
    d._keep = (block_table,)
    return d


def _token_rows(t: torch.Tensor, what: str):
    """A [T][heads][d] (one layer) or [L][T][heads][d] bf16 tensor whose heads are dense: (pointer, elements
    from one token's row to the next)."""
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor, got one on {t.device}")
    if t.dtype != torch.bfloat16 or t.dim() not in (3, 4):
        raise ValueError(f"{what}: expected a bf16 tensor [T][heads][d] or [L][T][heads][d]")
    st, sh = t.stride(), t.shape
    if t.numel() == 0:
        return t.data_ptr(), sh[-2] * sh[-1]
    row = st[-3] if sh[-3] > 1 else (st[0] if t.dim() == 4 and sh[0] > 1 else sh[-2] * sh[-1])
    if st[-1] != 1 or (sh[-2] > 1 and st[-2] != sh[-1]) or (t.dim() == 4 and sh[0] > 1 and st[0] != sh[1] * row):
        raise ValueError(f"{what}: heads must be dense and tokens evenly spaced (call .contiguous())")
    return t.data_ptr(), row


def tokens(k: torch.Tensor, v: torch.Tensor, tok_off: torch.Tensor, positions: torch.Tensor, q=None) -> TriTokenDesc:
    """New tokens for ``tri_append``: pre-RoPE ``q``/``k``/``v`` bf16 [L][T][heads][d] (or [T][heads][d] for one
    layer; they may be column slices of one fused projection), ``tok_off`` int64 [S+1], ``positions`` int32 [T]."""
    T = k.shape[-3]
    if k.shape != v.shape or positions.shape != (T,) or (q is not None and q.shape[:-2] != k.shape[:-2]):
        raise ValueError("tokens: q, k, v and positions disagree on the number of tokens, layers or heads")
    if tok_off.dtype != torch.int64 or positions.dtype != torch.int32:
        raise ValueError("tokens: tok_off must be int64 and positions int32")
    if len({t.device for t in (k, v, tok_off, positions, k if q is None else q)}) != 1:
        raise ValueError("tokens: tensors on different devices")
    (kp, ks), (vp, vs) = _token_rows(k, "k"), _token_rows(v, "v")
    qp, qs = _token_rows(q, "q") if q is not None else (None, 0)
    d = TriTokenDesc(T, _p(tok_off).value, _p(positions).value, qp, kp, vp, qs, ks, vs)
    d._keep = (q, k, v, tok_off, positions)
    return d


# ------------------------------------------------------------------- calls

def tri_workspace_size(m: TriModel, n_seqs: int, B: int) -> int:
    return int(_L.tri_workspace_size(ctypes.byref(m), n_seqs, B))


def tri_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check(_L.tri_workspace_init(_p(ws), ws.numel() * ws.element_size(), _s(stream)),
           "tri_workspace_init")


def alloc_workspace(m: TriModel, n_seqs: int, B: int, device=None, stream=None) -> torch.Tensor:
    """Allocate (through torch) and initialise a workspace for ``tri_score``/``tri_compact``."""
    n = tri_workspace_size(m, n_seqs, B)
    if n == 0:
        raise TriError(_abi.TRI_ERR_INVALID_ARG, "tri_workspace_size")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    tri_workspace_init(ws, stream)
    return ws


def tri_calib(m: TriModel, qpre: torch.Tensor, nq: int, centres: torch.Tensor,
              mean_norm: torch.Tensor, stream=None) -> None:
    _check(_L.tri_calib(ctypes.byref(m), _p(qpre), int(nq), _p(centres), _p(mean_norm), _s(stream)),
           "tri_calib")


def tri_score(m: TriModel, kv: TriKvDesc, K: torch.Tensor, pos, centres: torch.Tensor,
              mean_norm: torch.Tensor, p_now: torch.Tensor, offsets, key_mode: int,
              scores: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    offs = (ctypes.c_int32 * max(len(offsets), 1))(*[int(o) for o in offsets])
    _check(_L.tri_score(ctypes.byref(m), ctypes.byref(kv), _p(K), _p(pos), _p(centres),
                        _p(mean_norm), _p(p_now), offs, len(offsets), int(key_mode), _p(scores),
                        _p(ws), ws.numel() * ws.element_size(), _s(stream)), "tri_score")


def tri_compact(m: TriModel, kv: TriKvDesc, scores: torch.Tensor, B: int, W: int,
                K: torch.Tensor, V: torch.Tensor, pos, out: TriOutDesc, K_out: torch.Tensor,
                V_out: torch.Tensor, pos_out, kept_idx, kept_count, ws: torch.Tensor,
                stream=None) -> None:
    _check(_L.tri_compact(ctypes.byref(m), ctypes.byref(kv), _p(scores), int(B), int(W), _p(K),
                          _pd(V), _p(pos), ctypes.byref(out), _pd(K_out), _pd(V_out), _pd(pos_out),
                          _p(kept_idx), _p(kept_count), _p(ws), ws.numel() * ws.element_size(),
                          _s(stream)), "tri_compact")


def tri_calib_update(m: TriModel, qpre: torch.Tensor, nq: int, decay: float, sums: torch.Tensor,
                     weight: torch.Tensor, centres: torch.Tensor, mean_norm: torch.Tensor, stream=None) -> None:
    """Fold a batch of pre-RoPE queries into the decayed running statistics (fp64
    ``sums`` [L][Hq][d/2][3], ``weight`` [L][Hq]) and write the updated centres."""
    _check(_L.tri_calib_update(ctypes.byref(m), _p(qpre), int(nq), float(decay), _p(sums), _p(weight), _p(centres),
                               _p(mean_norm), _s(stream)), "tri_calib_update")


def tri_calib_stats(m: TriModel, n_heads: int, centres: torch.Tensor, mean_norm: torch.Tensor,
                    ref_centres=None, ref_mean_norm=None, concentration=None, head_stats=None,
                    stream=None) -> None:
    """Per-pair concentration and per-head (concentration, drift vs the reference)."""
    _check(_L.tri_calib_stats(ctypes.byref(m), int(n_heads), _p(centres), _p(mean_norm), _p(ref_centres),
                              _p(ref_mean_norm), _p(concentration), _p(head_stats), _s(stream)),
           "tri_calib_stats")


def tri_key_centres_ws_size(m: TriModel, n_seqs: int) -> int:
    return int(_L.tri_key_centres_ws_size(ctypes.byref(m), int(n_seqs)))


def tri_key_centres(m: TriModel, kv: TriKvDesc, K: torch.Tensor, pos, key_mode: int, centres: torch.Tensor,
                    mean_norm: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """Pre-RoPE key centre [R][d/2][2] and mean magnitude [R][d/2] of every cache row."""
    _check(_L.tri_key_centres(ctypes.byref(m), ctypes.byref(kv), _p(K), _p(pos), int(key_mode), _p(centres),
                              _p(mean_norm), _p(ws), ws.numel() * ws.element_size(), _s(stream)),
           "tri_key_centres")


def alloc_key_centres_workspace(m: TriModel, n_seqs: int, device=None, stream=None) -> torch.Tensor:
    n = tri_key_centres_ws_size(m, n_seqs)
    if n == 0:
        raise TriError(_abi.TRI_ERR_INVALID_ARG, "tri_key_centres_ws_size")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    tri_workspace_init(ws, stream)
    return ws


def tri_attention_ws_size(m: TriModel, n_seqs: int) -> int:
    return int(_L.tri_attention_ws_size(ctypes.byref(m), int(n_seqs)))


def alloc_attention_workspace(m: TriModel, n_seqs: int, device=None, stream=None) -> torch.Tensor:
    n = tri_attention_ws_size(m, n_seqs)
    if n == 0:
        raise TriError(_abi.TRI_ERR_INVALID_ARG, "tri_attention_ws_size")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    tri_workspace_init(ws, stream)
    return ws


def tri_decode_attention(m: TriModel, kv: TriKvDesc, K: torch.Tensor, V: torch.Tensor, q: torch.Tensor,
                         softmax_scale: float, out: torch.Tensor, lse, ws: torch.Tensor, stream=None) -> None:
    """Softmax attention of one decode query per (layer, sequence, query head) over the cache rows."""
    _check(_L.tri_decode_attention(ctypes.byref(m), ctypes.byref(kv), _p(K), _p(V), _p(q), float(softmax_scale),
                                   _p(out), _p(lse), _p(ws), ws.numel() * ws.element_size(), _s(stream)),
           "tri_decode_attention")


def tri_decode_attention_tc(m: TriModel, kv: TriKvDesc, K: torch.Tensor, V: torch.Tensor, q: torch.Tensor,
                            softmax_scale: float, out: torch.Tensor, lse, ws: torch.Tensor, stream=None) -> None:
    """tri_decode_attention on the tensor-memory (tcgen05) kernel: bf16 contiguous caches, head dim 128, G <= 16."""
    _check(_L.tri_decode_attention_tc(ctypes.byref(m), ctypes.byref(kv), _p(K), _p(V), _p(q), float(softmax_scale),
                                      _p(out), _p(lse), _p(ws), ws.numel() * ws.element_size(), _s(stream)),
           "tri_decode_attention_tc")


def _arg(t, dev: int, dtype=None, n: int = -1, what: str = ""):
    """Address of a contiguous tensor on the current device ``dev``, where kernels are launched (None -> NULL), with
    its type and number of elements checked where given."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{what or 'a tensor'} on {t.device} in a call on cuda:{dev} (use torch.cuda.device)")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor (call .contiguous())")
    if (dtype is not None and t.dtype != dtype) or (n >= 0 and t.numel() != n):
        raise ValueError(f"{what}: expected {n} elements of {dtype}, got {t.numel()} of {t.dtype}")
    return t.data_ptr()


def _slots(kv: TriKvDesc, m: TriModel, dev: int) -> int:
    """Records (a head's key or value of one slot) of the cache ``kv`` describes, whose row offsets and block table
    are on ``dev`` and reach as far as the kernels read."""
    held = getattr(kv, "_held", None)  # (a descriptor made by hand has none)
    if held is not None:
        offsets, tables, on = held
        if offsets <= m.n_layers * kv.n_seqs * m.n_kv_heads or tables < kv.n_seqs:
            raise ValueError(f"kv: {offsets} row offsets and {tables} block tables for {m.n_layers} layers, {kv.n_seqs} "
                             f"sequences and {m.n_kv_heads} KV heads")
        if on != dev:
            raise ValueError(f"kv: descriptor on cuda:{on} in a call on cuda:{dev} (use torch.cuda.device)")
    if kv.layout == TRI_KV_PAGED:
        return m.n_layers * kv.n_blocks * kv.block_size * m.n_kv_heads
    return kv.total_keys


def _cache(t: torch.Tensor, slots: int, kv: TriKvDesc, m: TriModel, dev: int, what: str):
    """Address of a cache tensor that holds the ``slots`` records ``kv`` describes."""
    if elem_type_of(t) != kv.elem_type or t.numel() < slots * m.head_dim:
        raise ValueError(f"{what}: {t.numel()} elements of {t.dtype} do not hold the {slots} records of head dim "
                         f"{m.head_dim} that the descriptor says")
    return _arg(t, dev, what=what)


def alloc_append_workspace(device=None, stream=None) -> torch.Tensor:
    """The flag word ``tri_append`` reports anomalies in (read with ``tri_status_check``)."""
    ws = torch.empty(256, dtype=torch.uint8, device=device or "cuda")
    tri_workspace_init(ws, stream)
    return ws


def tri_append(m: TriModel, kv: TriKvDesc, tokens: TriTokenDesc, key_mode: int, q_out, K: torch.Tensor,
               V: torch.Tensor, pos, ws: torch.Tensor, stream=None) -> None:
    """Rotate new tokens' queries and keys by their positions; write keys, values and positions to the last slots
    of the rows ``kv`` describes.  ``q_out`` bf16 [L][T][Hq][d] (None when the tokens have no q), ``pos`` int32, a
    position per record of K (or None)."""
    keep = getattr(tokens, "_keep", None)
    if keep is None:  # a descriptor filled in by hand holds addresses only: nothing here could check them
        raise ValueError("tokens: expected what tokens() returns")
    q, k, _, tok_off, _ = keep
    dev = torch.cuda.current_device()
    per = m.n_layers * tokens.total_tokens * m.head_dim
    if k.numel() != per * m.n_kv_heads or (q is not None and q.numel() != per * m.n_q_heads):
        raise ValueError("tokens do not match the model's layers, heads and head dim")
    if tok_off.numel() != kv.n_seqs + 1:
        raise ValueError(f"tok_off: {tok_off.numel()} offsets for {kv.n_seqs} sequences (expected one more)")
    slots = _slots(kv, m, dev)
    if pos is not None and pos.numel() < slots:
        raise ValueError(f"pos: {pos.numel()} positions for the {slots} records that the descriptor says")
    if k.get_device() != dev:
        raise ValueError(f"tokens on {k.device} in a call on cuda:{dev} (use torch.cuda.device)")
    _check(_L.tri_append(ctypes.byref(m), ctypes.byref(kv), ctypes.byref(tokens), int(key_mode),
                         _arg(q_out, dev, torch.bfloat16, per * m.n_q_heads, "q_out"), _cache(K, slots, kv, m, dev, "K"),
                         _cache(V, slots, kv, m, dev, "V"), _arg(pos, dev, torch.int32, what="pos"), _arg(ws, dev, what="ws"),
                         ws.numel() * ws.element_size(), _s(stream)), "tri_append")


def tri_prefill_attention_ws_size(m: TriModel, n_seqs: int, total_tokens: int) -> int:
    return int(_L.tri_prefill_attention_ws_size(ctypes.byref(m), int(n_seqs), int(total_tokens)))


def alloc_prefill_attention_workspace(m: TriModel, n_seqs: int, total_tokens: int, device=None,
                                      stream=None) -> torch.Tensor:
    n = tri_prefill_attention_ws_size(m, n_seqs, total_tokens)
    if n == 0:
        raise TriError(_abi.TRI_ERR_INVALID_ARG, "tri_prefill_attention_ws_size")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    tri_workspace_init(ws, stream)
    return ws


def _prefill_args(m, kv, K, V, q, tok_off, softmax_scale, out, lse, ws):
    dev = torch.cuda.current_device()
    heads, d = m.n_layers * m.n_q_heads, m.head_dim
    T = q.numel() // (heads * d)
    slots = _slots(kv, m, dev)
    return (ctypes.byref(m), ctypes.byref(kv), _cache(K, slots, kv, m, dev, "K"), _cache(V, slots, kv, m, dev, "V"),
            _arg(q, dev, torch.bfloat16, T * heads * d, "q"), _arg(tok_off, dev, torch.int64, kv.n_seqs + 1, "tok_off"), T,
            float(softmax_scale), _arg(out, dev, torch.bfloat16, T * heads * d, "out"),
            _arg(lse, dev, torch.float32, T * heads, "lse"), _arg(ws, dev, what="ws"), ws.numel() * ws.element_size())


def tri_prefill_attention(m: TriModel, kv: TriKvDesc, K: torch.Tensor, V: torch.Tensor, q: torch.Tensor,
                          tok_off: torch.Tensor, softmax_scale: float, out: torch.Tensor, lse, ws: torch.Tensor,
                          stream=None) -> None:
    """Causal softmax attention of the appended tokens' queries ``q`` bf16 [L][T][Hq][d] over the cache rows that
    end with them -> ``out`` bf16 [L][T][Hq][d], ``lse`` float [L][T][Hq] or None."""
    _check(_L.tri_prefill_attention(*_prefill_args(m, kv, K, V, q, tok_off, softmax_scale, out, lse, ws), _s(stream)),
           "tri_prefill_attention")


def tri_selftest_prefill_timeout(m: TriModel, kv: TriKvDesc, K: torch.Tensor, V: torch.Tensor, q: torch.Tensor,
                                 tok_off: torch.Tensor, softmax_scale: float, out: torch.Tensor, lse, ws: torch.Tensor,
                                 wait_tries: int, stream=None) -> None:
    """``tri_prefill_attention`` (head dims 64 and 256) whose waits give up after ``wait_tries`` tries: with few, its
    blocks end early and set TRI_FLAG_STAGE_TIMEOUT (read it with ``tri_status_check``)."""
    _check(_L.tri_selftest_prefill_timeout(*_prefill_args(m, kv, K, V, q, tok_off, softmax_scale, out, lse, ws),
                                           int(wait_tries), _s(stream)), "tri_selftest_prefill_timeout")


def tri_score_compact(m: TriModel, kv: TriKvDesc, K: torch.Tensor, V: torch.Tensor, pos, centres: torch.Tensor,
                      mean_norm: torch.Tensor, p_now: torch.Tensor, offsets, key_mode: int, B: int, W: int,
                      max_row_len: int, out: TriOutDesc, K_out: torch.Tensor, V_out: torch.Tensor, pos_out,
                      kept_idx, kept_count, scores, ws: torch.Tensor, stream=None) -> None:
    """tri_score + tri_compact in one call, fused on chip when max_row_len <= TRI_FUSED_MAX_ROW."""
    offs = (ctypes.c_int32 * max(len(offsets), 1))(*[int(o) for o in offsets])
    _check(_L.tri_score_compact(ctypes.byref(m), ctypes.byref(kv), _p(K), _pd(V), _p(pos), _p(centres),
                                _p(mean_norm), _p(p_now), offs, len(offsets), int(key_mode), int(B), int(W),
                                int(max_row_len), ctypes.byref(out), _pd(K_out), _pd(V_out), _pd(pos_out),
                                _p(kept_idx), _p(kept_count), _p(scores), _p(ws), ws.numel() * ws.element_size(),
                                _s(stream)), "tri_score_compact")


def tri_status_check(ws: torch.Tensor, stream=None):
    """Synchronise, read and clear the device flag word.  Returns (status, flags)."""
    flags = ctypes.c_uint32(0)
    st = _L.tri_status_check(_p(ws), ctypes.byref(flags), _s(stream))
    return st, int(flags.value)


def tri_calib_save(path: str, m: TriModel, nq: int, centres: torch.Tensor, mean_norm: torch.Tensor) -> None:
    """Write a calibration file (model shape, nq and the centres bit for bit).  The
    centres may be on any device; they are copied to contiguous host float32
    tensors for the call (the library reads host memory here)."""
    c = centres.detach().to("cpu", torch.float32).contiguous()
    n = mean_norm.detach().to("cpu", torch.float32).contiguous()
    F = m.head_dim // 2
    if c.numel() != m.n_layers * m.n_q_heads * F * 2 or n.numel() != m.n_layers * m.n_q_heads * F:
        raise ValueError("centres / mean_norm do not match the model shape")
    _check(_L.tri_calib_save(str(path).encode(), ctypes.byref(m), int(nq), ctypes.c_void_p(c.data_ptr()),
                             ctypes.c_void_p(n.data_ptr())), "tri_calib_save")


def tri_calib_load(path: str, device=None):
    """Read a calibration file -> (model, nq, centres [L][Hq][d/2][2], mean_norm
    [L][Hq][d/2]) as float32 tensors on `device` (host when None)."""
    m = TriModel()
    nq = ctypes.c_int64(0)
    _check(_L.tri_calib_load(str(path).encode(), ctypes.byref(m), ctypes.byref(nq), None, None, 0),
           "tri_calib_load (header)")
    F = m.head_dim // 2
    c = torch.empty(m.n_layers, m.n_q_heads, F, 2, dtype=torch.float32)
    n = torch.empty(m.n_layers, m.n_q_heads, F, dtype=torch.float32)
    m2 = TriModel()
    _check(_L.tri_calib_load(str(path).encode(), ctypes.byref(m2), ctypes.byref(nq), ctypes.c_void_p(c.data_ptr()),
                             ctypes.c_void_p(n.data_ptr()), n.numel()), "tri_calib_load")
    if device is not None:
        c, n = c.to(device), n.to(device)
    return m2, int(nq.value), c, n


def tri_selftest_wait_timeout(ws: torch.Tensor, limit_ns: int, stream=None) -> None:
    """Enqueue the self-test of the staged kernels' bounded wait: one warp waits
    `limit_ns` on a barrier nothing completes and sets TRI_FLAG_STAGE_TIMEOUT
    (read it with ``tri_status_check``)."""
    _check(_L.tri_selftest_wait_timeout(_p(ws), ws.numel() * ws.element_size(), int(limit_ns), _s(stream)),
           "tri_selftest_wait_timeout")


def tri_score_noalloc(m: TriModel, kv: TriKvDesc, K: torch.Tensor, pos, centres: torch.Tensor,
                      mean_norm: torch.Tensor, p_now: torch.Tensor, offsets, key_mode: int,
                      scores: torch.Tensor, stream=None) -> None:
    """``tri_score`` for callers that cannot allocate device memory: the scratch is a
    fixed array inside the library (at most TRI_NOALLOC_MAX_ROWS rows; calls on a
    device share it, so calls that overlap on the GPU race)."""
    offs = (ctypes.c_int32 * max(len(offsets), 1))(*[int(o) for o in offsets])
    _check(_L.tri_score_noalloc(ctypes.byref(m), ctypes.byref(kv), _p(K), _p(pos), _p(centres),
                                _p(mean_norm), _p(p_now), offs, len(offsets), int(key_mode),
                                _p(scores), _s(stream)), "tri_score_noalloc")
