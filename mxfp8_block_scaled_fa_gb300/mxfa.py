"""Thin ctypes binding over libmxfa.so (include/mxfa.h).

The functions named ``mxfa_*`` mirror the C entry points one to one and only
marshal arguments (torch CUDA tensors -> device pointers, the current torch
stream -> ``cudaStream_t``).  The helpers below them (``quantize``,
``attention_fwd`` ...) allocate outputs with torch and call those entry points;
every arithmetic step runs in the library's CUDA kernels.  Nothing here falls
back to the CPU: a missing library or a CUDA-less process raises.

A training step on bf16 q, k, v, do of shape [B * S, H, 128] (dense, causal):

    seqs = Seqs.dense(B, S)
    scale = 1 / math.sqrt(128)
    o, lse = attention_fwd(quantize(q, ROW, seqs), quantize(k, ROW, seqs),
                           quantize(v, COL, seqs), seqs, seqs, scale, causal=True)
    dq, dk, dv = attention_bwd(quantize(q, SQ, seqs), quantize(k, SQ, seqs),
                               quantize(v, ROW, seqs), quantize(do, SQ, seqs),
                               o, do, lse, seqs, seqs, scale, causal=True)

Jagged batches use ``Seqs.varlen(lengths, device)`` for queries and keys;
``o_mx=True`` / ``grads_mx=True`` also return O / the gradients as MXFP8.

A serving step over a 4-bit cache (MXFP4 or NVFP4) of R requests, with the new
tokens' q [T, Hq, 128] and k, v [T, H, 128] in request order:

    cache = KvCache.empty(num_blocks, H, page=64)
    free, state = kv_ring(num_blocks)
    step = kv_plan(ctx_lens, new_lens, block_table, free, state, 64, T)
    kv_append(cache, k, v, step.slots)
    o, lse = kv_attention(q, cache, step.cu_q, step.kv_lens, block_table, max_q, scale)
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import math
import os
from dataclasses import FrozenInstanceError, dataclass
from typing import Optional, Sequence

import numpy as np
import torch

from . import build as _build

ROW, COL, SQ = 0, 1, 2
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration",
           3: "pointer not 16-byte aligned", 4: "workspace too small", 5: "CUDA error",
           6: "device wait timed out", 7: "device index check failed"}


class MxfaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_STATUS.get(status, status)} (status {status})")
        self.status = status


class MxOut(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sf_compact", ctypes.c_void_p),
                ("sf_packed", ctypes.c_void_p)]


class MxIn(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sf", ctypes.c_void_p)]


P_SCALE_BLOCK, P_SCALE_CONST = 0, 1
RESCALE_THRESHOLD = 8.0


class AttnOpts(ctypes.Structure):
    """mxfa_attn_opts: forward rescale threshold (log2 units) and the P scale mode."""
    _fields_ = [("rescale_threshold", ctypes.c_float), ("p_scale", ctypes.c_int)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmxfa.so from the package's build folder (raises if absent)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB):
            raise RuntimeError(
                "libmxfa.so is not built: run mxfp8_block_scaled_fa_gb300.build.build()")
        L = ctypes.CDLL(_build.LIB)
        P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        S = ctypes.c_size_t
        sig = {
            "mxfa_status_string": (ctypes.c_char_p, [I]),
            "mxfa_version": (I, []),
            "mxfa_packed_tiles": (I64, [P, I, I]),
            "mxfa_sf_packed_bytes": (S, [I, I64, I]),
            "mxfa_quantize": (I, [P, I64, I, I, I, P, I, I, I64, P, P]),
            "mxfa_sf_pack": (I, [P, I64, I, I, I, P, I, I, I64, P, P]),
            "mxfa_quantize_dual": (I, [P, I64, I, I, I, P, I, I, I64, P, P, P]),
            "mxfa_sf_unpack": (I, [P, I64, I, I, I, P, I, I, I64, P, P]),
            "mxfa_fwd": (I, [P, P, P, I, I, I, I, F, I, P, P, P]),
            "mxfa_varlen_fwd": (I, [P, P, P, P, P, I, I, I, I64, I64, I64, I64, I, I, F, I, P, P,
                                    P]),
            "mxfa_fwd_mxo": (I, [P, P, P, I, I, I, I, F, I, P, P, P, P]),
            "mxfa_varlen_fwd_mxo": (I, [P, P, P, P, P, I, I, I, I64, I64, I64, I64, I, I, F, I, P,
                                        P, P, P]),
            "mxfa_fwd_opts": (I, [P, P, P, I, I, I, I, F, I, P, P, P, P]),
            "mxfa_varlen_fwd_opts": (I, [P, P, P, P, P, I, I, I, I64, I64, I64, I64, I, I, F, I,
                                         P, P, P, P]),
            "mxfa_bwd_opts": (I, [P, P, P, P, P, P, P, I, I, I, I, F, I, P, I, F, P, P, P, P, S,
                                  P]),
            "mxfa_varlen_bwd_opts": (I, [P, P, P, P, P, P, P, P, P, I, I, I, I64, I64, I64, I64,
                                         I, I, F, I, P, I, F, P, P, P, P, S, P]),
            "mxfa_bwd_workspace_size": (S, [I64, I, I, I, I]),
            "mxfa_bwd": (I, [P, P, P, P, P, P, P, I, I, I, I, F, I, I, F, P, P, P, P, S, P]),
            "mxfa_varlen_bwd": (I, [P, P, P, P, P, P, P, P, P, I, I, I, I64, I64, I64, I64, I, I,
                                    F, I, I, F, P, P, P, P, S, P]),
            "mxfa_bwd_mxg": (I, [P, P, P, P, P, P, P, I, I, I, I, F, I, I, F, P, P, P, P, S, P, P,
                                 P, P]),
            "mxfa_varlen_bwd_mxg": (I, [P, P, P, P, P, P, P, P, P, I, I, I, I64, I64, I64, I64, I,
                                        I, F, I, I, F, P, P, P, P, S, P, P, P, P]),
            "mxfa_rmsnorm_quant": (I, [P, P, I64, I64, F, I, I, P, P, P, P]),
            "mxfa_get_device_status": (I, [P, ctypes.POINTER(ctypes.c_uint)]),
            "mxfa_gemm_quant": (I, [P, P, I64, I64, I64, P, P, P, P]),
            "mxfa_gemm_quant_fmt": (I, [P, I, P, I, I64, I64, I64, P, P, P, P]),
            "mxfa_quantize_lowp": (I, [P, I64, I, I, I, P, P, P, P, P]),
            "mxfa_tensor_peak_probe": (I, [I, I, P, P]),
            "mxfa_bwd_noalloc": (I, [P, P, P, P, P, P, P, I, I, I, I, F, I, I, F, P, P, P, P]),
            "mxfa_bwd_noalloc_scratch_bytes": (S, []),
            "mxfa_kv_codes_bytes": (S, [I64, I, I]),
            "mxfa_kv_sf_bytes": (S, [I64, I, I, I]),
            "mxfa_kv_plan": (I, [P, P, I, P, I, P, I64, P, P, I, I64, P, P, P, P, P]),
            "mxfa_kv_append": (I, [P, P, P, I64, I64, I64, P, P]),
            "mxfa_kv_load": (I, [P, P, I64, P, P, P]),
            "mxfa_kv_attn_workspace_size": (S, [I, I, I64, I, I]),
            "mxfa_kv_attn": (I, [P, P, I64, I64, P, P, I, P, I, I, I, F, I, P, P, P, S, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _p(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(st: int, where: str):
    if st != 0:
        raise MxfaError(st, where)


# ------------------------------------------------------------ C-named calls
def mxfa_packed_tiles(cu_host: Optional[np.ndarray], nseq: int, seqlen: int) -> int:
    if cu_host is None:
        return int(lib().mxfa_packed_tiles(None, nseq, seqlen))
    cu = np.ascontiguousarray(cu_host, dtype=np.int32)
    return int(lib().mxfa_packed_tiles(cu.ctypes.data_as(ctypes.c_void_p), nseq, seqlen))


def mxfa_quantize(x, tokens, H, D, blk, cu_seqlens, nseq, max_seqlen, packed_tiles, out: MxOut,
                  stream=None):
    _check(lib().mxfa_quantize(_p(x), tokens, H, D, blk, _p(cu_seqlens), nseq, max_seqlen,
                               packed_tiles, ctypes.byref(out), _stream(stream)), "mxfa_quantize")


def mxfa_sf_pack(sf_compact, tokens, H, D, blk, cu_seqlens, nseq, max_seqlen, packed_tiles,
                 sf_packed, stream=None):
    _check(lib().mxfa_sf_pack(_p(sf_compact), tokens, H, D, blk, _p(cu_seqlens), nseq, max_seqlen,
                              packed_tiles, _p(sf_packed), _stream(stream)), "mxfa_sf_pack")


def mxfa_sf_unpack(sf_packed, tokens, H, D, blk, cu_seqlens, nseq, max_seqlen, packed_tiles,
                   sf_compact, stream=None):
    _check(lib().mxfa_sf_unpack(_p(sf_packed), tokens, H, D, blk, _p(cu_seqlens), nseq,
                                max_seqlen, packed_tiles, _p(sf_compact), _stream(stream)),
           "mxfa_sf_unpack")


def mxfa_fwd(q: MxIn, k: MxIn, v: MxIn, B, S, H, D, scale, causal, o, lse, stream=None):
    _check(lib().mxfa_fwd(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), B, S, H, D,
                          float(scale), int(causal), _p(o), _p(lse), _stream(stream)), "mxfa_fwd")


def mxfa_varlen_fwd(q, k, v, cu_q, cu_k, nseq, max_sq, max_sk, total_q, total_k, ptq, ptk, H, D,
                    scale, causal, o, lse, stream=None):
    _check(lib().mxfa_varlen_fwd(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), _p(cu_q),
                                 _p(cu_k), nseq, max_sq, max_sk, total_q, total_k, ptq, ptk, H, D,
                                 float(scale), int(causal), _p(o), _p(lse), _stream(stream)),
           "mxfa_varlen_fwd")


def mxfa_fwd_mxo(q: MxIn, k: MxIn, v: MxIn, B, S, H, D, scale, causal, o, lse, o_mx: MxOut,
                 stream=None):
    _check(lib().mxfa_fwd_mxo(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), B, S, H, D,
                              float(scale), int(causal), _p(o), _p(lse), ctypes.byref(o_mx),
                              _stream(stream)), "mxfa_fwd_mxo")


def mxfa_varlen_fwd_mxo(q, k, v, cu_q, cu_k, nseq, max_sq, max_sk, total_q, total_k, ptq, ptk, H,
                        D, scale, causal, o, lse, o_mx: MxOut, stream=None):
    _check(lib().mxfa_varlen_fwd_mxo(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), _p(cu_q),
                                     _p(cu_k), nseq, max_sq, max_sk, total_q, total_k, ptq, ptk, H,
                                     D, float(scale), int(causal), _p(o), _p(lse),
                                     ctypes.byref(o_mx), _stream(stream)), "mxfa_varlen_fwd_mxo")


def mxfa_bwd_workspace_size(total_q, nseq, H, D, dq_mode) -> int:
    return int(lib().mxfa_bwd_workspace_size(total_q, nseq, H, D, dq_mode))


def mxfa_bwd(q, k, v, do_mx, o, do, lse, B, S, H, D, scale, causal, dq_mode, dq_static, dq, dk,
             dv, ws, ws_bytes, stream=None):
    _check(lib().mxfa_bwd(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), ctypes.byref(do_mx),
                          _p(o), _p(do), _p(lse), B, S, H, D, float(scale), int(causal), dq_mode,
                          float(dq_static), _p(dq), _p(dk), _p(dv), _p(ws), ws_bytes,
                          _stream(stream)), "mxfa_bwd")


def mxfa_bwd_noalloc(q, k, v, do_mx, o, do, lse, B, S, H, D, scale, causal, dq_mode, dq_static,
                     dq, dk, dv, stream=None):
    """mxfa_bwd without a caller workspace (the library's built-in scratch array)."""
    _check(lib().mxfa_bwd_noalloc(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v),
                                  ctypes.byref(do_mx), _p(o), _p(do), _p(lse), B, S, H, D,
                                  float(scale), int(causal), dq_mode, float(dq_static), _p(dq),
                                  _p(dk), _p(dv), _stream(stream)), "mxfa_bwd_noalloc")


def mxfa_varlen_bwd(q, k, v, do_mx, o, do, lse, cu_q, cu_k, nseq, max_sq, max_sk, total_q,
                    total_k, ptq, ptk, H, D, scale, causal, dq_mode, dq_static, dq, dk, dv, ws,
                    ws_bytes, stream=None):
    _check(lib().mxfa_varlen_bwd(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v),
                                 ctypes.byref(do_mx), _p(o), _p(do), _p(lse), _p(cu_q), _p(cu_k),
                                 nseq, max_sq, max_sk, total_q, total_k, ptq, ptk, H, D,
                                 float(scale), int(causal), dq_mode, float(dq_static), _p(dq),
                                 _p(dk), _p(dv), _p(ws), ws_bytes, _stream(stream)),
           "mxfa_varlen_bwd")


def mxfa_rmsnorm_quant(x, gamma, T, C, eps, seg_len, H, row: Optional[MxOut],
                       col: Optional[MxOut], sq: Optional[MxOut], stream=None):
    ref = lambda m: ctypes.byref(m) if m is not None else None
    _check(lib().mxfa_rmsnorm_quant(_p(x), _p(gamma), T, C, float(eps), seg_len, H, ref(row),
                                    ref(col), ref(sq), _stream(stream)), "mxfa_rmsnorm_quant")


def mxfa_get_device_status(stream=None) -> int:
    flags = ctypes.c_uint(0)
    st = lib().mxfa_get_device_status(_stream(stream), ctypes.byref(flags))
    return st


# ----------------------------------------------------------- convenience layer
@dataclass
class Seqs:
    """Host-side description of packed sequences (dense = uniform lengths)."""
    nseq: int
    max_len: int
    total: int
    cu_host: Optional[np.ndarray]      # int32 [nseq+1] or None (uniform)
    cu_dev: Optional[torch.Tensor]     # int32 device copy or None
    ptiles: int                        # sum ceil(len/128)
    blocks32: int                      # sum ceil(len/32)

    @staticmethod
    def dense(B: int, S: int) -> "Seqs":
        return Seqs(B, S, B * S, None, None, B * math.ceil(S / 128), B * math.ceil(S / 32))

    @staticmethod
    def varlen(lengths: Sequence[int], device) -> "Seqs":
        lens = np.asarray(lengths, dtype=np.int64)
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        cu_dev = torch.from_numpy(cu).to(device)
        return Seqs(len(lens), int(lens.max()) if len(lens) else 0, int(cu[-1]), cu, cu_dev,
                    int(np.sum((lens + 127) // 128)), int(np.sum((lens + 31) // 32)))


@dataclass
class Mx:
    """An MXFP8 tensor produced by the library (payload + scales)."""
    data: torch.Tensor                 # uint8 [tokens, H, D]
    sf_compact: Optional[torch.Tensor]
    sf_packed: Optional[torch.Tensor]
    blk: int

    def mx_in(self) -> MxIn:
        return MxIn(self.data.data_ptr(), self.sf_packed.data_ptr())


def _sf_shapes(blk, seqs: Seqs, H, D):
    cols = H * D
    if blk == ROW:
        comp = (seqs.total, cols // 32)
    elif blk == COL:
        comp = (seqs.blocks32, cols)
    else:
        comp = (seqs.blocks32, cols // 32)
    packed = seqs.ptiles * H * (16 if blk == SQ else 512)
    return comp, packed


def quantize(x: torch.Tensor, blk: int, seqs: Seqs, compact=True, packed=True,
             stream=None) -> Mx:
    """bf16 [tokens, H, D] (or [B, S, H, D]) -> Mx via mxfa_quantize."""
    H, D = x.shape[-2], x.shape[-1]
    x3 = x.reshape(-1, H, D)
    dev = x.device
    data = torch.empty(x3.shape, dtype=torch.uint8, device=dev)
    comp_shape, pbytes = _sf_shapes(blk, seqs, H, D)
    sfc = torch.empty(comp_shape, dtype=torch.uint8, device=dev) if compact else None
    sfp = torch.empty(max(pbytes, 16), dtype=torch.uint8, device=dev) if packed else None
    out = MxOut(data.data_ptr(), _p(sfc), _p(sfp))
    mxfa_quantize(x3, seqs.total, H, D, blk, seqs.cu_dev, seqs.nseq, seqs.max_len, seqs.ptiles,
                  out, stream)
    return Mx(data, sfc, sfp, blk)


def mxfa_quantize_dual(x, tokens, H, D, blk, cu_seqlens, nseq, max_seqlen, packed_tiles,
                       out: MxOut, out_row: MxOut, stream=None):
    _check(lib().mxfa_quantize_dual(_p(x), tokens, H, D, blk, _p(cu_seqlens), nseq, max_seqlen,
                                    packed_tiles, ctypes.byref(out), ctypes.byref(out_row),
                                    _stream(stream)), "mxfa_quantize_dual")


def quantize_dual(x: torch.Tensor, blk: int, seqs: Seqs, stream=None):
    """bf16 [tokens, H, D] -> (Mx in layout blk (COL or SQ), Mx in ROW) from one read."""
    H, D = x.shape[-2], x.shape[-1]
    x3 = x.reshape(-1, H, D)
    dev = x.device
    outs, structs = [], []
    for b in (blk, ROW):
        data = torch.empty(x3.shape, dtype=torch.uint8, device=dev)
        comp_shape, pbytes = _sf_shapes(b, seqs, H, D)
        sfc = torch.empty(comp_shape, dtype=torch.uint8, device=dev)
        sfp = torch.empty(max(pbytes, 16), dtype=torch.uint8, device=dev)
        outs.append(Mx(data, sfc, sfp, b))
        structs.append(MxOut(data.data_ptr(), sfc.data_ptr(), sfp.data_ptr()))
    mxfa_quantize_dual(x3, seqs.total, H, D, blk, seqs.cu_dev, seqs.nseq, seqs.max_len, seqs.ptiles,
                       structs[0], structs[1], stream)
    return outs[0], outs[1]


def sf_pack(sf_compact: torch.Tensor, blk: int, seqs: Seqs, H: int, D: int = 128,
            stream=None) -> torch.Tensor:
    _, pbytes = _sf_shapes(blk, seqs, H, D)
    sfp = torch.empty(max(pbytes, 16), dtype=torch.uint8, device=sf_compact.device)
    mxfa_sf_pack(sf_compact, seqs.total, H, D, blk, seqs.cu_dev, seqs.nseq, seqs.max_len,
                 seqs.ptiles, sfp, stream)
    return sfp


def sf_unpack(sf_packed: torch.Tensor, blk: int, seqs: Seqs, H: int, D: int = 128,
              stream=None) -> torch.Tensor:
    """Packed scales -> compact scales (the inverse of sf_pack)."""
    comp_shape, _ = _sf_shapes(blk, seqs, H, D)
    sfc = torch.empty(comp_shape, dtype=torch.uint8, device=sf_packed.device)
    mxfa_sf_unpack(sf_packed, seqs.total, H, D, blk, seqs.cu_dev, seqs.nseq, seqs.max_len,
                   seqs.ptiles, sfc, stream)
    return sfc


def _opts_ref(opts):
    return None if opts is None else ctypes.byref(opts)


def mxfa_fwd_opts(q, k, v, B, S, H, D, scale, causal, opts, o, lse, stream=None):
    _check(lib().mxfa_fwd_opts(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), B, S, H, D,
                               float(scale), int(causal), _opts_ref(opts), _p(o), _p(lse),
                               _stream(stream)), "mxfa_fwd_opts")


def mxfa_varlen_fwd_opts(q, k, v, cu_q, cu_k, nseq, max_sq, max_sk, total_q, total_k, ptq, ptk, H,
                         D, scale, causal, opts, o, lse, stream=None):
    _check(lib().mxfa_varlen_fwd_opts(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), _p(cu_q),
                                      _p(cu_k), nseq, max_sq, max_sk, total_q, total_k, ptq, ptk,
                                      H, D, float(scale), int(causal), _opts_ref(opts), _p(o),
                                      _p(lse), _stream(stream)), "mxfa_varlen_fwd_opts")


def mxfa_bwd_opts(q, k, v, do_mx, o, do, lse, B, S, H, D, scale, causal, opts, dq_mode, dq_static,
                  dq, dk, dv, ws, ws_bytes, stream=None):
    _check(lib().mxfa_bwd_opts(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v),
                               ctypes.byref(do_mx), _p(o), _p(do), _p(lse), B, S, H, D,
                               float(scale), int(causal), _opts_ref(opts), dq_mode,
                               float(dq_static), _p(dq), _p(dk), _p(dv), _p(ws), ws_bytes,
                               _stream(stream)), "mxfa_bwd_opts")


def mxfa_varlen_bwd_opts(q, k, v, do_mx, o, do, lse, cu_q, cu_k, nseq, max_sq, max_sk, total_q,
                         total_k, ptq, ptk, H, D, scale, causal, opts, dq_mode, dq_static, dq, dk,
                         dv, ws, ws_bytes, stream=None):
    _check(lib().mxfa_varlen_bwd_opts(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v),
                                      ctypes.byref(do_mx), _p(o), _p(do), _p(lse), _p(cu_q),
                                      _p(cu_k), nseq, max_sq, max_sk, total_q, total_k, ptq, ptk,
                                      H, D, float(scale), int(causal), _opts_ref(opts), dq_mode,
                                      float(dq_static), _p(dq), _p(dk), _p(dv), _p(ws), ws_bytes,
                                      _stream(stream)), "mxfa_varlen_bwd_opts")


def attention_fwd(q: Mx, k: Mx, v: Mx, seqs_q: Seqs, seqs_k: Seqs, scale: float,
                  causal: bool = False, stream=None, out=None, o_mx: bool = False,
                  opts: Optional[AttnOpts] = None):
    """Forward on quantized operands -> (O bf16 [tokens, H, D], lse fp32), and with
    o_mx=True also O as MXFP8 (Mx with ROW compact and packed scales) as a third item.
    opts (AttnOpts) selects the rescale threshold and the P scale mode (no MXFP8 O then)."""
    if opts is not None and o_mx:
        raise ValueError("opts and o_mx cannot be combined")
    H, D = q.data.shape[-2], q.data.shape[-1]
    dev = q.data.device
    o = out[0] if out is not None else torch.empty(q.data.shape, dtype=torch.bfloat16, device=dev)
    omx = omx_s = None
    if o_mx:
        u8 = dict(dtype=torch.uint8, device=dev)
        omx = Mx(torch.empty(q.data.shape, **u8), torch.empty((seqs_q.total, H * D // 32), **u8),
                 torch.empty(seqs_q.ptiles * H * 512, **u8), ROW)
        omx_s = MxOut(omx.data.data_ptr(), omx.sf_compact.data_ptr(), omx.sf_packed.data_ptr())
    if seqs_q.cu_host is None and seqs_k.cu_host is None:
        lse = out[1] if out is not None else torch.empty((seqs_q.nseq, H, seqs_q.max_len),
                                                         dtype=torch.float32, device=dev)
        args = (q.mx_in(), k.mx_in(), v.mx_in(), seqs_q.nseq, seqs_q.max_len, H, D, scale,
                causal, o, lse)
        if o_mx:
            mxfa_fwd_mxo(*args, omx_s, stream)
        elif opts is not None:
            mxfa_fwd_opts(*args[:9], opts, o, lse, stream)
        else:
            mxfa_fwd(*args, stream)
    else:
        lse = out[1] if out is not None else torch.empty((H, seqs_q.total), dtype=torch.float32,
                                                         device=dev)
        args = (q.mx_in(), k.mx_in(), v.mx_in(), seqs_q.cu_dev, seqs_k.cu_dev, seqs_q.nseq,
                seqs_q.max_len, seqs_k.max_len, seqs_q.total, seqs_k.total, seqs_q.ptiles,
                seqs_k.ptiles, H, D, scale, causal, o, lse)
        if o_mx:
            mxfa_varlen_fwd_mxo(*args, omx_s, stream)
        elif opts is not None:
            mxfa_varlen_fwd_opts(*args[:16], opts, o, lse, stream)
        else:
            mxfa_varlen_fwd(*args, stream)
    return (o, lse, omx) if o_mx else (o, lse)


def mxfa_bwd_mxg(q, k, v, do_mx, o, do, lse, B, S, H, D, scale, causal, dq_mode, dq_static, dq,
                 dk, dv, ws, ws_bytes, dq_mx, dk_mx, dv_mx, stream=None):
    ref = lambda m: ctypes.byref(m) if m is not None else None
    _check(lib().mxfa_bwd_mxg(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v),
                              ctypes.byref(do_mx), _p(o), _p(do), _p(lse), B, S, H, D,
                              float(scale), int(causal), dq_mode, float(dq_static), _p(dq), _p(dk),
                              _p(dv), _p(ws), ws_bytes, ref(dq_mx), ref(dk_mx), ref(dv_mx),
                              _stream(stream)), "mxfa_bwd_mxg")


def mxfa_varlen_bwd_mxg(q, k, v, do_mx, o, do, lse, cu_q, cu_k, nseq, max_sq, max_sk, total_q,
                        total_k, ptq, ptk, H, D, scale, causal, dq_mode, dq_static, dq, dk, dv, ws,
                        ws_bytes, dq_mx, dk_mx, dv_mx, stream=None):
    ref = lambda m: ctypes.byref(m) if m is not None else None
    _check(lib().mxfa_varlen_bwd_mxg(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v),
                                     ctypes.byref(do_mx), _p(o), _p(do), _p(lse), _p(cu_q),
                                     _p(cu_k), nseq, max_sq, max_sk, total_q, total_k, ptq, ptk, H,
                                     D, float(scale), int(causal), dq_mode, float(dq_static),
                                     _p(dq), _p(dk), _p(dv), _p(ws), ws_bytes, ref(dq_mx),
                                     ref(dk_mx), ref(dv_mx), _stream(stream)),
           "mxfa_varlen_bwd_mxg")


def attention_bwd(q: Mx, k: Mx, v: Mx, do_mx: Mx, o: torch.Tensor, do: torch.Tensor,
                  lse: torch.Tensor, seqs_q: Seqs, seqs_k: Seqs, scale: float,
                  causal: bool = False, dq_mode: int = 0, dq_static: float = 1.0, stream=None,
                  ws=None, out=None, grads_mx: bool = False, opts: Optional[AttnOpts] = None):
    """Backward on quantized operands -> (dQ, dK, dV) bf16; with grads_mx=True also the
    three gradients as MXFP8 (Mx with ROW compact and packed scales), six items in all.
    opts (AttnOpts) selects the P scale mode (no MXFP8 gradients then)."""
    if opts is not None and grads_mx:
        raise ValueError("opts and grads_mx cannot be combined")
    H, D = q.data.shape[-2], q.data.shape[-1]
    dev = q.data.device
    wsb = mxfa_bwd_workspace_size(seqs_q.total, seqs_q.nseq, H, D, dq_mode)
    if ws is None:
        ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    if out is None:
        dq = torch.empty(q.data.shape, dtype=torch.bfloat16, device=dev)
        dk = torch.empty(k.data.shape, dtype=torch.bfloat16, device=dev)
        dv = torch.empty(v.data.shape, dtype=torch.bfloat16, device=dev)
    else:
        dq, dk, dv = out
    gmx = gs = None
    if grads_mx:
        u8 = dict(dtype=torch.uint8, device=dev)
        gmx = [Mx(torch.empty(t.shape, **u8), torch.empty((sq.total, H * D // 32), **u8),
                  torch.empty(sq.ptiles * H * 512, **u8), ROW)
               for t, sq in ((dq, seqs_q), (dk, seqs_k), (dv, seqs_k))]
        gs = [MxOut(m.data.data_ptr(), m.sf_compact.data_ptr(), m.sf_packed.data_ptr())
              for m in gmx]
    if seqs_q.cu_host is None and seqs_k.cu_host is None:
        args = (q.mx_in(), k.mx_in(), v.mx_in(), do_mx.mx_in(), o, do, lse, seqs_q.nseq,
                seqs_q.max_len, H, D, scale, causal, dq_mode, dq_static, dq, dk, dv, ws,
                ws.numel())
        if grads_mx:
            mxfa_bwd_mxg(*args, *gs, stream)
        elif opts is not None:
            mxfa_bwd_opts(*args[:13], opts, *args[13:], stream)
        else:
            mxfa_bwd(*args, stream)
    else:
        args = (q.mx_in(), k.mx_in(), v.mx_in(), do_mx.mx_in(), o, do, lse, seqs_q.cu_dev,
                seqs_k.cu_dev, seqs_q.nseq, seqs_q.max_len, seqs_k.max_len, seqs_q.total,
                seqs_k.total, seqs_q.ptiles, seqs_k.ptiles, H, D, scale, causal, dq_mode,
                dq_static, dq, dk, dv, ws, ws.numel())
        if grads_mx:
            mxfa_varlen_bwd_mxg(*args, *gs, stream)
        elif opts is not None:
            mxfa_varlen_bwd_opts(*args[:20], opts, *args[20:], stream)
        else:
            mxfa_varlen_bwd(*args, stream)
    return (dq, dk, dv, *gmx) if grads_mx else (dq, dk, dv)


def rmsnorm_quant(x: torch.Tensor, gamma: torch.Tensor, eps: float, seg_len: int, H: int,
                  outputs=("row", "col", "sq"), packed=True, stream=None):
    """Fused RMSNorm + quantization -> dict name -> Mx (compact + packed scales)."""
    T, C = x.shape
    dev = x.device
    seqs = Seqs.dense(T // seg_len, seg_len) if T % seg_len == 0 else None
    res, structs = {}, {}
    for name, blk in (("row", ROW), ("col", COL), ("sq", SQ)):
        if name not in outputs:
            continue
        data = torch.empty((T, C), dtype=torch.uint8, device=dev)
        nb32 = (T + 31) // 32
        comp = {ROW: (T, C // 32), COL: (nb32, C), SQ: (nb32, C // 32)}[blk]
        sfc = torch.empty(comp, dtype=torch.uint8, device=dev)
        sfp = None
        if packed:
            if seqs is None:
                raise ValueError("packed scales need T to be a multiple of seg_len")
            sfp = torch.empty(seqs.ptiles * H * (16 if blk == SQ else 512), dtype=torch.uint8,
                              device=dev)
        res[name] = Mx(data, sfc, sfp, blk)
        structs[name] = MxOut(data.data_ptr(), sfc.data_ptr(), _p(sfp))
    mxfa_rmsnorm_quant(x, gamma, T, C, eps, seg_len, H, structs.get("row"), structs.get("col"),
                       structs.get("sq"), stream)
    return res


def mxfa_gemm_quant(a: MxIn, b: MxIn, M, N, K, y_bf16, y_row: Optional[MxOut],
                    y_col: Optional[MxOut], stream=None):
    ref = lambda m: ctypes.byref(m) if m is not None else None
    _check(lib().mxfa_gemm_quant(ctypes.byref(a), ctypes.byref(b), M, N, K, _p(y_bf16), ref(y_row),
                                 ref(y_col), _stream(stream)), "mxfa_gemm_quant")


LOWP_MXFP4, LOWP_MXFP6_E2M3, LOWP_MXFP6_E3M2, LOWP_NVFP4 = 0, 1, 2, 3
LOWP_CODES, LOWP_MMA = 0, 1
ELEM_E4M3, ELEM_E2M3, ELEM_E3M2, ELEM_E2M1 = 0, 1, 2, 3


def mxfa_quantize_lowp(x, rows, cols, fmt, q_layout, q, sf, sf_packed, tensor_scale, stream=None):
    _check(lib().mxfa_quantize_lowp(_p(x), rows, cols, fmt, q_layout, _p(q), _p(sf), _p(sf_packed),
                                    _p(tensor_scale), _stream(stream)), "mxfa_quantize_lowp")


def quantize_lowp(x: torch.Tensor, fmt: int, packed: bool = False, mma: bool = False, stream=None):
    """bf16 [rows, cols] -> dict: 'q' u8 [rows, cols] (codes one per byte, or with
    mma=True the MMA operand form of the MX formats), 'sf' scales, optional
    'sf_packed' (MX formats), and 'tensor_scale' (NVFP4, a 1-element fp32 tensor)."""
    rows, cols = x.shape[0], x.numel() // x.shape[0]
    dev = x.device
    u8 = dict(dtype=torch.uint8, device=dev)
    q = torch.empty((rows, cols), **u8)
    sf = torch.empty((rows, cols // (16 if fmt == LOWP_NVFP4 else 32)), **u8)
    sfp = torch.empty((rows // 128) * (cols // 128) * 512, **u8) if packed else None
    ts = torch.empty(1, dtype=torch.float32, device=dev) if fmt == LOWP_NVFP4 else None
    mxfa_quantize_lowp(x, rows, cols, fmt, LOWP_MMA if mma else LOWP_CODES, q, sf, sfp, ts, stream)
    return {"q": q, "sf": sf, "sf_packed": sfp, "tensor_scale": ts}


def mxfa_gemm_quant_fmt(a: MxIn, a_fmt, b: MxIn, b_fmt, M, N, K, y_bf16, y_row, y_col, stream=None):
    ref = lambda m: ctypes.byref(m) if m is not None else None
    _check(lib().mxfa_gemm_quant_fmt(ctypes.byref(a), a_fmt, ctypes.byref(b), b_fmt, M, N, K,
                                     _p(y_bf16), ref(y_row), ref(y_col), _stream(stream)),
           "mxfa_gemm_quant_fmt")


def mxfa_tensor_peak_probe(iters, ctas, cycles, stream=None):
    _check(lib().mxfa_tensor_peak_probe(int(iters), int(ctas), _p(cycles), _stream(stream)),
           "mxfa_tensor_peak_probe")


def gemm_quant(a: Mx, b: Mx, bf16: bool = True, row: bool = True, col: bool = True,
               stream=None):
    """Y = A B^T on ROW-quantized A [M, K] and B [N, K] (Mx with packed scales, as
    quantize(x.view(rows, K // 128, 128), ROW, Seqs.dense(1, rows)) makes them) ->
    dict with 'bf16' (tensor [M, N]) and 'row' / 'col' (Mx over [M, N])."""
    M, K = a.data.shape[0], a.data.numel() // a.data.shape[0]
    N = b.data.shape[0]
    dev = a.data.device
    u8 = dict(dtype=torch.uint8, device=dev)
    res, outs = {}, {}
    if bf16:
        res["bf16"] = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    for name, blk, comp in (("row", ROW, (M, N // 32)), ("col", COL, (M // 32, N))):
        if (name == "row" and row) or (name == "col" and col):
            m = Mx(torch.empty((M, N), **u8), torch.empty(comp, **u8),
                   torch.empty((M // 128) * (N // 128) * 512, **u8), blk)
            res[name] = m
            outs[name] = MxOut(m.data.data_ptr(), m.sf_compact.data_ptr(), m.sf_packed.data_ptr())
    mxfa_gemm_quant(a.mx_in(), b.mx_in(), M, N, K, res.get("bf16"), outs.get("row"),
                    outs.get("col"), stream)
    return res


# ------------------------------------------------------------------ 4-bit KV cache
KV_MXFP4, KV_NVFP4 = 0, 1


class KvPages(ctypes.Structure):
    """mxfa_kv_cache: the device pointers and sizes of one layer's cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_sf", ctypes.c_void_p),
                ("v_sf", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int64), ("page", ctypes.c_int), ("H", ctypes.c_int),
                ("D", ctypes.c_int), ("fmt", ctypes.c_int)]


def mxfa_kv_plan(ctx_lens, new_lens, R, block_table, max_blocks, free_ring, ring_size, ring_in,
                 ring_out, page, tokens, cu_q, kv_lens, slots, positions, stream=None):
    _check(lib().mxfa_kv_plan(_p(ctx_lens), _p(new_lens), R, _p(block_table), max_blocks,
                              _p(free_ring), ring_size, _p(ring_in), _p(ring_out), page, tokens,
                              _p(cu_q), _p(kv_lens), _p(slots), _p(positions), _stream(stream)),
           "mxfa_kv_plan")


def mxfa_kv_append(pages: KvPages, k, v, k_stride, v_stride, tokens, slots, stream=None):
    _check(lib().mxfa_kv_append(ctypes.byref(pages), _p(k), _p(v), k_stride, v_stride, tokens,
                                _p(slots), _stream(stream)), "mxfa_kv_append")


def mxfa_kv_load(pages: KvPages, slots, tokens, k, v, stream=None):
    _check(lib().mxfa_kv_load(ctypes.byref(pages), _p(slots), tokens, _p(k), _p(v),
                              _stream(stream)), "mxfa_kv_load")


def mxfa_kv_attn_workspace_size(R, max_q, max_k, Hq, H) -> int:
    return int(lib().mxfa_kv_attn_workspace_size(R, max_q, max_k, Hq, H))


def mxfa_kv_attn(pages: KvPages, q, q_stride, total_q, cu_q, kv_lens, R, block_table, max_blocks,
                 max_q, Hq, scale, causal, o, lse, ws, ws_bytes, stream=None):
    _check(lib().mxfa_kv_attn(ctypes.byref(pages), _p(q), q_stride, total_q, _p(cu_q), _p(kv_lens),
                              R, _p(block_table), max_blocks, max_q, Hq, float(scale), int(causal),
                              _p(o), _p(lse), _p(ws), ws_bytes, _stream(stream)), "mxfa_kv_attn")


_kv = None


def _fast():
    """kv_py: the calls below for ordinary arguments (new buffers, the current device and
    stream).  Its functions return None where they do not apply, and for arguments that do not
    fit; what follows each of them here checks the arguments one by one."""
    global _kv
    if _kv is None:
        lib()
        spec = importlib.util.spec_from_file_location("kv_py", _build.PY_MODULE)
        if spec is None or not os.path.exists(_build.PY_MODULE):
            raise RuntimeError(f"{_build.PY_MODULE} is missing; build it with mxfp8_block_scaled_fa_gb300.build")
        _kv = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_kv)
    return _kv


def _raw_stream(index: int) -> int:
    """The current stream of CUDA device `index`."""
    return torch._C._cuda_getCurrentRawStream(index)


def _flat(name: str, t: torch.Tensor, dtype, index: int):
    """t has this dtype, is contiguous and on CUDA device `index` (-1: the CPU)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected device {index}")


def _rows(name: str, x: torch.Tensor, heads: int, index: int):
    """bf16 [tokens, heads, 128] with the heads of a token one after another, on device `index` ->
    elements between tokens."""
    if x.dtype is not torch.bfloat16:
        raise TypeError(f"{name} is {x.dtype}, expected torch.bfloat16")
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != 128:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [tokens, {heads}, 128]")
    stride = x.stride()
    if shape[0] and (stride[2] != 1 or (heads > 1 and stride[1] != 128)):
        raise ValueError(f"{name}: the heads of a token must lie one after another")
    if x.get_device() != index:
        raise ValueError(f"{name} is on {x.device}, expected device {index}")
    return stride[0] if shape[0] > 1 else heads * 128


def _here(index: int, stream) -> bool:
    """Whether a call on device `index` can go ahead: it is the current device, and the stream the
    current one.  Otherwise the caller starts again within _place()."""
    if index < 0:
        raise ValueError("the 4-bit cache lives on a CUDA device")
    return stream is None and torch._C._cuda_getDevice() == index


def _place(index: int, stream):
    """The context in which a call on device `index` allocates and launches: its stream if one is
    given (memory taken from the allocator then belongs to that stream), else the device's current one."""
    if stream is None:
        return torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on device {index}")
    return torch.cuda.stream(stream)


_KV_FIXED = frozenset(("k", "v", "k_sf", "v_sf", "fmt", "k_scale", "v_scale", "H", "page", "index", "raw", "pages"))


@dataclass(init=False)
class KvCache:
    """One layer's keys and values in 4 bits, in pages (layout: mxfa_kv_cache in mxfa.h).  Calls
    go by the addresses of the tensors that it was made with: its fields cannot be assigned, and
    a tensor of it must keep its storage.  Other buffers take another KvCache."""
    k: torch.Tensor                    # uint8 [num_blocks, H, page, 64]
    v: torch.Tensor
    k_sf: torch.Tensor                 # uint8 [num_blocks, H, page, 4 (MXFP4) or 8 (NVFP4)]
    v_sf: torch.Tensor
    fmt: int
    k_scale: Optional[torch.Tensor] = None   # NVFP4: fp32, one element
    v_scale: Optional[torch.Tensor] = None

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_sf: torch.Tensor, v_sf: torch.Tensor, fmt: int,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None):
        d = self.__dict__
        d["k"], d["v"], d["k_sf"], d["v_sf"], d["fmt"] = k, v, k_sf, v_sf, fmt
        made = _fast().cache(k, v, k_sf, v_sf, fmt, k_scale, v_scale)
        if fmt == KV_MXFP4:
            k_scale = v_scale = None
        d["k_scale"], d["v_scale"] = k_scale, v_scale
        if made is not None:
            d["raw"], d["H"], d["page"], d["index"] = made
            return
        if fmt != KV_MXFP4 and fmt != KV_NVFP4:
            raise ValueError(f"unknown cache format {fmt}")
        shape = k.shape
        if len(shape) != 4 or shape[3] != 64 or v.shape != shape:
            raise ValueError("k and v must be [num_blocks, H, page, 64]")
        n, h, page, _ = shape
        if 0 in shape:
            raise ValueError("a cache has at least one block, one head and one row a page")
        sf = (n, h, page, 4 if fmt == KV_MXFP4 else 8)
        if k_sf.shape != sf or v_sf.shape != sf:
            raise ValueError(f"k_sf and v_sf must be {list(sf)}")
        index = k.get_device()
        _flat("k", k, torch.uint8, index)
        _flat("v", v, torch.uint8, index)
        _flat("k_sf", k_sf, torch.uint8, index)
        _flat("v_sf", v_sf, torch.uint8, index)
        ks = vs = None
        if fmt == KV_NVFP4:
            if k_scale is None or v_scale is None:
                raise ValueError("an NVFP4 cache needs k_scale and v_scale")
            _flat("k_scale", k_scale, torch.float32, index)
            _flat("v_scale", v_scale, torch.float32, index)
            if k_scale.numel() != 1 or v_scale.numel() != 1:
                raise ValueError("k_scale and v_scale have one element")
            ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
        d["raw"], d["H"], d["page"], d["index"] = None, h, page, index
        d["pages"] = KvPages(k.data_ptr(), v.data_ptr(), k_sf.data_ptr(), v_sf.data_ptr(), ks, vs, n, page, h, 128, fmt)

    def __setattr__(self, name, value):
        if name in _KV_FIXED:
            raise FrozenInstanceError(f"a KvCache keeps its {name}; other buffers take another KvCache")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        if name in _KV_FIXED:
            raise FrozenInstanceError(f"a KvCache keeps its {name}")
        object.__delattr__(self, name)

    def __reduce__(self):  # a copy is made of its own tensors, not of their addresses
        return KvCache, (self.k, self.v, self.k_sf, self.v_sf, self.fmt, self.k_scale, self.v_scale)

    @functools.cached_property
    def pages(self) -> KvPages:
        return KvPages.from_buffer_copy(self.raw)

    @staticmethod
    def empty(num_blocks: int, H: int, page: int = 64, fmt: int = KV_MXFP4, k_scale: float = 1.0,
              v_scale: float = 1.0, device="cuda") -> "KvCache":
        """A cache whose rows all read as zero.  k_scale and v_scale (NVFP4) are
        about the largest magnitude to hold, over 448 * 6."""
        codes, sf = (num_blocks, H, page, 64), (num_blocks, H, page, 4 if fmt == KV_MXFP4 else 8)
        z = lambda shape: torch.zeros(shape, dtype=torch.uint8, device=device)
        s = lambda x: torch.tensor([x], dtype=torch.float32, device=device) if fmt == KV_NVFP4 else None
        return KvCache(z(codes), z(codes), z(sf), z(sf), fmt, s(k_scale), s(v_scale))


@dataclass
class KvStep:
    """What kv_plan says about a step (mxfa_kv_plan in mxfa.h).  Where ring_state[2] > 0 some requests
    got no blocks: their tokens' slots are -1, and what the attention returns for them is to be left aside."""
    cu_q: torch.Tensor        # int32 [R + 1]
    kv_lens: torch.Tensor     # int32 [R]
    slots: torch.Tensor       # int64 [tokens]
    positions: torch.Tensor   # int32 [tokens]
    ring_state: torch.Tensor  # int64 [3]: taken, put, lacked


def kv_ring(num_blocks: int, device="cuda"):
    """The queue of free blocks of a new cache -> (free_ring, ring_state) for kv_plan."""
    return (torch.arange(num_blocks, dtype=torch.int32, device=device),
            torch.tensor([0, num_blocks, 0], dtype=torch.int64, device=device))


def kv_plan(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
            free_ring: torch.Tensor, ring_state: torch.Tensor, page: int, tokens: int,
            out: Optional[KvStep] = None, stream=None) -> KvStep:
    """The plan of a step from context lengths and counts of new tokens (int32 [R];
    a negative count ends a request): writes new blocks into block_table (int32
    [R, max_blocks]), gives the blocks of ended requests back to free_ring, and
    returns offsets, lengths, and slot and position of `tokens` tokens.  `out`
    gives the result's buffers; its kv_lens may be ctx_lens and its ring_state
    may be ring_state, for a step that is captured once and replayed."""
    if out is None and stream is None:
        made = _fast().plan(ctx_lens, new_lens, block_table, free_ring, ring_state, page, tokens)
        if type(made) is tuple:
            return KvStep(*made)
        if made is not None:
            _check(made, "mxfa_kv_plan")
    R, index = ctx_lens.numel(), ctx_lens.get_device()
    shape = block_table.shape
    if new_lens.numel() != R or len(shape) != 2 or shape[0] != R:
        raise ValueError("ctx_lens, new_lens and block_table describe different numbers of requests")
    i32, i64 = torch.int32, torch.int64
    _flat("ctx_lens", ctx_lens, i32, index)
    _flat("new_lens", new_lens, i32, index)
    _flat("block_table", block_table, i32, index)
    _flat("free_ring", free_ring, i32, index)
    _flat("ring_state", ring_state, i64, index)
    if not _here(index, stream):
        with _place(index, stream):
            return kv_plan(ctx_lens, new_lens, block_table, free_ring, ring_state, page, tokens, out)
    if out is None:
        dev = ctx_lens.device
        out = KvStep(torch.empty(R + 1, dtype=i32, device=dev), torch.empty(R, dtype=i32, device=dev),
                     torch.empty(tokens, dtype=i64, device=dev),
                     torch.empty(tokens, dtype=i32, device=dev), torch.empty(3, dtype=i64, device=dev))
    else:
        if (out.cu_q.numel(), out.kv_lens.numel(), out.slots.numel(), out.positions.numel()) != (
                R + 1, R, tokens, tokens):
            raise ValueError("out has buffers of other sizes")
        _flat("cu_q", out.cu_q, i32, index)
        _flat("kv_lens", out.kv_lens, i32, index)
        _flat("slots", out.slots, i64, index)
        _flat("positions", out.positions, i32, index)
        _flat("out.ring_state", out.ring_state, i64, index)
    if ring_state.numel() != 3 or out.ring_state.numel() != 3:
        raise ValueError("ring_state has three elements")
    _check(lib().mxfa_kv_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), R, block_table.data_ptr(),
                              shape[1], free_ring.data_ptr(), free_ring.numel(),
                              ring_state.data_ptr(), out.ring_state.data_ptr(), page, tokens,
                              out.cu_q.data_ptr(), out.kv_lens.data_ptr(), out.slots.data_ptr(),
                              out.positions.data_ptr(), _raw_stream(index)), "mxfa_kv_plan")
    return out


def kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None):
    """Quantizes bf16 k, v [tokens, H, 128] (tokens may be strided, as slices of a
    fused projection are) into the cache rows `slots` (int64 [tokens], distinct;
    negative: skipped)."""
    if stream is None:
        status = _fast().append(cache.raw, k, v, slots)
        if status is not None:
            return _check(status, "mxfa_kv_append")
    index, H = cache.index, cache.H
    ks, vs = _rows("k", k, H, index), _rows("v", v, H, index)
    T = k.shape[0]
    if v.shape[0] != T or slots.numel() != T:
        raise ValueError("k, v and slots have different numbers of tokens")
    _flat("slots", slots, torch.int64, index)
    if not _here(index, stream):
        with _place(index, stream):
            return kv_append(cache, k, v, slots)
    if T:
        _check(lib().mxfa_kv_append(ctypes.byref(cache.pages), k.data_ptr(), v.data_ptr(), ks, vs, T,
                                    slots.data_ptr(), _raw_stream(index)), "mxfa_kv_append")


def kv_load(cache: KvCache, slots: torch.Tensor, out=None, stream=None):
    """The cached values of `slots` (int64 [tokens]) -> bf16 (k, v) [tokens, H, 128];
    zeros for a negative slot."""
    if out is None and stream is None:
        made = _fast().load(cache.raw, slots)
        if type(made) is tuple:
            return made
        if made is not None:
            _check(made, "mxfa_kv_load")
    index, T = cache.index, slots.numel()
    shape = (T, cache.H, 128)
    _flat("slots", slots, torch.int64, index)
    if not _here(index, stream):
        with _place(index, stream):
            return kv_load(cache, slots, out)
    if out is None:
        dev = slots.device
        k = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        v = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        k, v = out
        if k.shape != shape or v.shape != shape:
            raise ValueError(f"out must be two tensors of shape {shape}")
        _flat("out k", k, torch.bfloat16, index)
        _flat("out v", v, torch.bfloat16, index)
    if T:
        _check(lib().mxfa_kv_load(ctypes.byref(cache.pages), slots.data_ptr(), T, k.data_ptr(),
                                  v.data_ptr(), _raw_stream(index)), "mxfa_kv_load")
    return k, v


def kv_attention(q: torch.Tensor, cache: KvCache, cu_q: torch.Tensor, kv_lens: torch.Tensor,
                 block_table: torch.Tensor, max_q: int, scale: float, causal: bool = True,
                 out=None, ws=None, stream=None):
    """Attention of new query tokens over the cache -> (O bf16 [tokens, Hq, 128], lse
    fp32 [Hq, tokens]).  q: bf16 [tokens, Hq, 128], tokens may be strided; cu_q
    (int32 [R + 1]), kv_lens (int32 [R], new tokens included) and block_table as
    kv_plan gives them; max_q: the most query tokens of a request.  causal aligns
    the last query to the last key.  Rows outside cu_q's are not written."""
    if out is None and ws is None and stream is None:
        made = _fast().attention(q, cache.raw, cu_q, kv_lens, block_table, max_q, scale, causal)
        if type(made) is tuple:
            return made
        if made is not None:
            _check(made, "mxfa_kv_attn")
    H, index = cache.H, cache.index
    shape = q.shape
    if len(shape) != 3 or shape[1] == 0 or shape[1] % H:
        raise ValueError(f"q has shape {tuple(shape)}, expected [tokens, a multiple of {H}, 128]")
    T, Hq, _ = shape
    qs = _rows("q", q, Hq, index)
    R = kv_lens.numel()
    tshape = block_table.shape
    if cu_q.numel() != R + 1 or len(tshape) != 2 or tshape[0] != R:
        raise ValueError("cu_q, kv_lens and block_table describe different numbers of requests")
    i32 = torch.int32
    _flat("cu_q", cu_q, i32, index)
    _flat("kv_lens", kv_lens, i32, index)
    _flat("block_table", block_table, i32, index)
    if not _here(index, stream):
        with _place(index, stream):
            return kv_attention(q, cache, cu_q, kv_lens, block_table, max_q, scale, causal, out, ws)
    dev = q.device
    if out is None:
        o = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    else:
        o, lse = out
        if o.shape != shape or lse.shape != (Hq, T):
            raise ValueError(f"out must have shapes {tuple(shape)} and {(Hq, T)}")
        _flat("out o", o, torch.bfloat16, index)
        _flat("out lse", lse, torch.float32, index)
    if T == 0 or R == 0:
        return o, lse
    L = lib()
    ws_at, ws_bytes = None, 0
    if ws is None:
        ws_bytes = L.mxfa_kv_attn_workspace_size(R, max_q, tshape[1] * cache.page, Hq, H)
        if ws_bytes:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
            ws_at = ws.data_ptr()
    elif ws.get_device() != index:
        raise ValueError(f"ws is on {ws.device}, expected device {index}")
    elif not ws.is_contiguous():
        raise ValueError("ws is not contiguous")
    else:
        ws_at, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _check(L.mxfa_kv_attn(ctypes.byref(cache.pages), q.data_ptr(), qs, T, cu_q.data_ptr(),
                          kv_lens.data_ptr(), R, block_table.data_ptr(), tshape[1], max_q, Hq, scale,
                          1 if causal else 0, o.data_ptr(), lse.data_ptr(), ws_at, ws_bytes,
                          _raw_stream(index)), "mxfa_kv_attn")
    return o, lse


def device_status(stream=None) -> int:
    """Synchronise and return (and clear) the kernels' device status (0 = ok)."""
    return mxfa_get_device_status(stream)
