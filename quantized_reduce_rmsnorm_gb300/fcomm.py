"""Thin Python binding of libfcomm (ctypes): argument marshalling only.

Every step of the path runs in libfcomm's CUDA kernels; this module only
turns torch tensors into device pointers and the current torch stream into a
cudaStream_t, calls the C entry point of the same name, and raises FcommError
on a non-OK status.  There is no CPU fallback: if the library cannot be
built or loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

from . import build as _build

FMT_BF16, FMT_INT8_SYM, FMT_INT4_ASYM, FMT_BF16_TAGGED, FMT_F32 = 0, 1, 2, 3, 4
FMT_INT8_TAGGED, FMT_INT4_TAGGED = 5, 6
FC_OK, FC_ERR_INVALID, FC_ERR_CUDA, FC_ERR_STALE_BLOCK, FC_ERR_UNSUPPORTED = 0, 1, 2, 3, 4
STATUS_NO_INDEX = 0x7F7F7F7F

# Names exported by the C ABI (include/fcomm.h)
EXPORTS = (
    "fc_codes_bytes", "fc_groups", "fc_tagged_bytes", "fc_shard_range", "fc_group_quantize",
    "fc_group_quantize_multi", "fc_reduce_dequant_sum", "fc_requant_gather", "fc_pack_tagged",
    "fc_pack_tagged_multi", "fc_group_quantize_tagged",
    "fc_allreduce_residual_rmsnorm", "fc_allreduce_residual_rmsnorm_ex", "fc_status_string",
    "fc_last_error", "fc_version", "fc_token_split", "fc_select_protocol", "fc_allgather_dequant",
    "fc_protocol_estimate", "fc_mx4_codes_bytes", "fc_mx4_scales_bytes", "fc_mx4_quantize",
    "fc_mx4_dequantize", "fc_mx4_matmul", "fc_block_norm", "fc_block_norm_backward_workspace",
    "fc_block_norm_backward", "fc_layer_norm", "fc_layer_norm_backward_workspace",
    "fc_layer_norm_backward", "fc_fp8_scales", "fc_fp8_quantize", "fc_fp8_dequantize",
    "fc_fp8_matmul", "fc_gated_ffn", "fc_gated_ffn_backward_workspace", "fc_gated_ffn_backward",
    "fc_gated_ffn_backward_ex_workspace", "fc_gated_ffn_backward_ex",
)


class FcommError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_STATUS_NAMES = {0: "FC_OK", 1: "FC_ERR_INVALID", 2: "FC_ERR_CUDA", 3: "FC_ERR_STALE_BLOCK",
                 4: "FC_ERR_UNSUPPORTED"}


class QSpec(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("group", ctypes.c_int32)]

    def __repr__(self):
        return f"QSpec(fmt={self.fmt}, group={self.group})"


class QTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p)]


class LinkModel(ctypes.Structure):
    _fields_ = [("link_gbps", ctypes.c_double), ("barrier_us", ctypes.c_double)]


class LaunchOpts(ctypes.Structure):
    _fields_ = [("max_ctas", ctypes.c_int32), ("kernel", ctypes.c_int32)]


class Mx4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class Fp8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class BlockNormSpec(ctypes.Structure):
    _fields_ = [("post_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("pre_weight", ctypes.c_void_p), ("gate_rows", ctypes.c_int64),
                ("residual_scale", ctypes.c_float), ("block_scale", ctypes.c_float),
                ("post_eps", ctypes.c_float), ("pre_eps", ctypes.c_float)]


class BlockNormGrads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("dresidual", ctypes.c_void_p),
                ("dpost_weight", ctypes.c_void_p), ("dgate", ctypes.c_void_p),
                ("dpre_weight", ctypes.c_void_p)]


KERNEL_AUTO, KERNEL_STREAM, KERNEL_TMA = 0, 1, 2
ACT_SILU, ACT_GELU_TANH = 0, 1


INT8_G128 = QSpec(FMT_INT8_SYM, 128)
INT4_G32 = QSpec(FMT_INT4_ASYM, 32)
BF16 = QSpec(FMT_BF16, 0)
BF16_TAGGED = QSpec(FMT_BF16_TAGGED, 0)
INT8_G128_TAGGED = QSpec(FMT_INT8_TAGGED, 128)
INT4_G32_TAGGED = QSpec(FMT_INT4_TAGGED, 32)

_lib = None


def lib_path() -> str:
    return _build.LIB


def load(path: Optional[str] = None):
    """Load libfcomm.so (building it with nvcc if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or _build.build()
    lib = ctypes.CDLL(p)
    P, i64, i32, u32, f32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32,
                             ctypes.c_float)
    QS, QT = QSpec, QTensor
    sigs = {
        "fc_codes_bytes": (ctypes.c_size_t, [QS, i64, i64]),
        "fc_groups": (ctypes.c_size_t, [QS, i64, i64]),
        "fc_tagged_bytes": (ctypes.c_size_t, [i64, i64]),
        "fc_shard_range": (i32, [QS, i64, i64, i32, i32, ctypes.POINTER(i64),
                                 ctypes.POINTER(i64)]),
        "fc_group_quantize": (i32, [P, i64, i64, QS, QT, P, P]),
        "fc_group_quantize_multi": (i32, [P, i32, i64, i64, QS, P, P, P]),
        "fc_reduce_dequant_sum": (i32, [P, i32, i64, i64, QS, i32, P, P]),
        "fc_requant_gather": (i32, [P, i64, i64, QS, QT, P, i32, P]),
        "fc_allgather_dequant": (i32, [ctypes.POINTER(QT), i32, i64, i64, QS, i32, P, u32, P, P]),
        "fc_pack_tagged": (i32, [P, i64, i64, u32, P, P]),
        "fc_pack_tagged_multi": (i32, [P, i32, i64, i64, u32, P, P]),
        "fc_group_quantize_tagged": (i32, [P, i32, i64, i64, QS, u32, P, P, P]),
        "fc_allreduce_residual_rmsnorm": (
            i32, [P, i32, i64, i64, QS, P, P, P, f32, QT, P, u32, P, P]),
        "fc_allreduce_residual_rmsnorm_ex": (
            i32, [P, i32, i64, i64, QS, P, P, P, f32, QT, P, u32, P, P, P]),
        "fc_status_string": (ctypes.c_char_p, [i32]),
        "fc_last_error": (ctypes.c_char_p, []),
        "fc_version": (ctypes.c_char_p, []),
        "fc_token_split": (i32, [i32, i64, i64, QS, ctypes.POINTER(i64), ctypes.POINTER(i64)]),
        "fc_select_protocol": (i32, [i64, i64, i32, i32, P, ctypes.POINTER(QSpec),
                                     ctypes.POINTER(ctypes.c_double)]),
        "fc_protocol_estimate": (i32, [i64, i64, i32, QS, P, ctypes.POINTER(ctypes.c_double)]),
        "fc_mx4_codes_bytes": (ctypes.c_size_t, [i64, i64]),
        "fc_mx4_scales_bytes": (ctypes.c_size_t, [i64, i64]),
        "fc_mx4_quantize": (i32, [P, i32, i64, i64, Mx4, P]),
        "fc_mx4_dequantize": (i32, [Mx4, i64, i64, P, i32, P]),
        "fc_mx4_matmul": (i32, [Mx4, Mx4, i64, i64, i64, P, i32, P, P]),
        "fc_block_norm": (i32, [P, P, i64, i64, i32, P, P, P, Mx4, P]),
        "fc_block_norm_backward_workspace": (ctypes.c_size_t, [i64, i64, i64]),
        "fc_block_norm_backward": (i32, [P, P, P, P, i64, i64, i32, P, P, P, P, P]),
        "fc_layer_norm": (i32, [P, P, i64, i64, i32, P, P, f32, P, P, P, P]),
        "fc_layer_norm_backward_workspace": (ctypes.c_size_t, [i64, i64]),
        "fc_layer_norm_backward": (i32, [P, P, P, P, i64, i64, i32, P, P, P, P, P, P, P]),
        "fc_fp8_scales": (ctypes.c_size_t, [i64, i64, i64]),
        "fc_fp8_quantize": (i32, [P, i32, i64, i64, i64, Fp8, P]),
        "fc_fp8_dequantize": (i32, [Fp8, i64, i64, i64, P, i32, P]),
        "fc_fp8_matmul": (i32, [Fp8, Fp8, i64, i64, i64, P, i32, P, P]),
        "fc_gated_ffn": (i32, [P, P, P, i64, i64, i64, i32, P, P, P, P, P]),
        "fc_gated_ffn_backward_workspace": (ctypes.c_size_t, [i64, i64]),
        "fc_gated_ffn_backward": (i32, [P, P, P, P, P, P, i64, i64, i64, i32, P, P, P, P, P, P]),
        "fc_gated_ffn_backward_ex_workspace": (ctypes.c_size_t, [i64, i64, i32]),
        "fc_gated_ffn_backward_ex": (i32, [P, P, P, P, P, P, i64, i64, i64, i32, i32, P, P, P, P, P, P]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int):
    if status != FC_OK:
        raise FcommError(status, _lib.fc_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libfcomm takes CUDA tensors (device memory)")
    if not t.is_contiguous():
        raise ValueError("libfcomm takes contiguous tensors")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:  # the handle alone: a torch Stream object costs more than a launch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _qt(q) -> QTensor:
    """(codes, scales, zeros) tuple of tensors (or None entries) -> QTensor."""
    if q is None:
        return QTensor(None, None, None)
    codes, scales, zeros = (tuple(q) + (None, None, None))[:3]
    return QTensor(_ptr(codes), _ptr(scales), _ptr(zeros))


class Bound:
    """One libfcomm call with its arguments marshalled once.

    Calling it launches the entry point again with the same device pointers
    on `stream` (default: the current torch stream), with no per-call
    argument conversion: the host cost of a call is the C entry point
    itself.  The object holds a reference to every tensor it was bound to,
    so their memory cannot be freed and handed to another tensor while the
    bound call exists.  For the calls that carry an epoch (tagged formats),
    `epoch` may be changed between calls.  Threads may share a bound call: a
    call changes nothing that another one reads (the epoch is the setter's)."""
    __slots__ = ("_fn", "_args", "_si", "_ei", "_keep")

    def __init__(self, fn, args, stream_index, epoch_index=None, keep=()):
        self._fn, self._args, self._si, self._ei, self._keep = fn, list(args), stream_index, \
            epoch_index, keep

    @property
    def epoch(self) -> int:
        return self._args[self._ei].value

    @epoch.setter
    def epoch(self, e: int):
        self._args[self._ei] = ctypes.c_uint32(e & 0xFFFFFFFF)

    def __call__(self, stream=None):
        a = self._args.copy()
        a[self._si] = _stream(stream)
        st = self._fn(*a)
        if st != FC_OK:
            _check(st)


class DeviceBound(Bound):
    """A Bound call that belongs to the device of its tensors: it runs there, on
    that device's current stream by default, whichever device is current.

    Its arguments are ctypes objects of the entry point's own types from the
    start and go through a function object without argtypes, so that a call
    converts none of them (2.6 us a launch on GB300's host, 3.1 with)."""
    __slots__ = ("_dev", "_last")

    def __init__(self, fn, args, stream_index, keep, device: int):
        def exact(a, t):
            return a if isinstance(a, t) or type(a).__name__ == "CArgObject" else t(a)
        super().__init__(_lib[fn.__name__], [exact(a, t) for a, t in zip(args, fn.argtypes)],
                         stream_index, keep=keep)
        self._dev = device
        self._last = (None, None)  # a stream and the arguments for it, replaced together

    def __call__(self, stream=None):
        if torch._C._cuda_getDevice() != self._dev:
            with torch.cuda.device(self._dev):
                return self(stream)
        s = torch._C._cuda_getCurrentRawStream(self._dev) if stream is None else _stream(stream)
        last = self._last
        if s != last[0]:
            a = self._args.copy()
            a[self._si] = ctypes.c_void_p(s)
            self._last = last = (s, a)
        st = self._fn(*last[1])
        if st != FC_OK:
            _check(st)


def _rows_hidden(x: torch.Tensor):
    if x.dim() != 2:
        raise ValueError("expected a [rows, hidden] tensor")
    return x.shape[0], x.shape[1]


# ----------------------------------------------------------------- sizes ---
def codes_bytes(spec: QSpec, rows: int, hidden: int) -> int:
    return load().fc_codes_bytes(spec, rows, hidden)


def groups(spec: QSpec, rows: int, hidden: int) -> int:
    return load().fc_groups(spec, rows, hidden)


def tagged_bytes(rows: int, hidden: int) -> int:
    return load().fc_tagged_bytes(rows, hidden)


def shard_range(spec: QSpec, rows: int, hidden: int, P: int, shard: int):
    g0, g1 = ctypes.c_int64(), ctypes.c_int64()
    _check(load().fc_shard_range(spec, rows, hidden, P, shard, ctypes.byref(g0), ctypes.byref(g1)))
    return g0.value, g1.value


def alloc_qtensor(spec: QSpec, rows: int, hidden: int, device="cuda"):
    """Caller-owned (codes, scales, zeros) torch tensors for a quantized tensor."""
    nb = codes_bytes(spec, rows, hidden)
    ng = groups(spec, rows, hidden)
    codes = torch.empty(nb, dtype=torch.uint8, device=device)
    scales = torch.empty(ng, dtype=torch.float32, device=device)
    zeros = torch.empty(ng, dtype=torch.float32, device=device) if spec.fmt == FMT_INT4_ASYM \
        else None
    return codes, scales, zeros


# --------------------------------------------------------------- compute ---
def group_quantize(x: torch.Tensor, spec: QSpec, out, stream=None,
                   d_status: Optional[torch.Tensor] = None):
    """Quantize one [rows, hidden] bf16 slab into out = (codes, scales[, zeros]);
    d_status: optional int32[2] device status words (see fcomm.h)."""
    rows, hidden = _rows_hidden(x)
    _check(load().fc_group_quantize(_ptr(x), rows, hidden, spec, _qt(out), _ptr(d_status),
                                    _stream(stream)))


def bind_group_quantize_multi(xs: Sequence[torch.Tensor], spec: QSpec, outs,
                              d_status: Optional[torch.Tensor] = None) -> Bound:
    rows, hidden = _rows_hidden(xs[0])
    xp = (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])
    qo = (QTensor * len(outs))(*[_qt(o) for o in outs])
    return Bound(load().fc_group_quantize_multi,
                 [xp, len(xs), rows, hidden, spec, qo, ctypes.c_void_p(_ptr(d_status)), None], 7,
                 keep=(tuple(xs), tuple(outs), d_status))


def group_quantize_multi(xs: Sequence[torch.Tensor], spec: QSpec, outs, stream=None,
                         d_status: Optional[torch.Tensor] = None):
    bind_group_quantize_multi(xs, spec, outs, d_status)(stream)


def reduce_dequant_sum(slabs, spec: QSpec, rows: int, hidden: int, out: torch.Tensor,
                       shard: int = -1, stream=None):
    """out[rows, hidden] fp32 = fixed-order sum of the dequantized slabs (or one shard)."""
    qs = (QTensor * len(slabs))(*[_qt(s) for s in slabs])
    _check(load().fc_reduce_dequant_sum(qs, len(slabs), rows, hidden, spec, shard, _ptr(out),
                                        _stream(stream)))


def requant_gather(reduced: torch.Tensor, spec: QSpec, requant_out=None,
                   out: Optional[torch.Tensor] = None, out_dtype: int = FMT_BF16, stream=None):
    rows, hidden = _rows_hidden(reduced)
    _check(load().fc_requant_gather(_ptr(reduced), rows, hidden, spec, _qt(requant_out),
                                    _ptr(out), out_dtype, _stream(stream)))


def allgather_dequant(shards, spec: QSpec, rows: int, hidden: int, out: torch.Tensor,
                      expected_epoch: int = 0, d_status: Optional[torch.Tensor] = None,
                      stream=None):
    """Standalone quantized all-gather: shards = P (codes, scales, zeros) tuples
    (or tagged-block tensors), shard p holding groups [p*per, min((p+1)*per,
    n_g)) from its own index 0; out = the whole dequantized [rows, hidden]
    tensor (bf16 or fp32, by its dtype)."""
    qs = (QTensor * len(shards))(*[_qt(s if isinstance(s, (tuple, list)) else (s,))
                                   for s in shards])
    od = FMT_F32 if out.dtype == torch.float32 else FMT_BF16
    _check(load().fc_allgather_dequant(qs, len(shards), rows, hidden, spec, od, _ptr(out),
                                       expected_epoch, _ptr(d_status), _stream(stream)))


def bind_allgather_dequant(shards, spec: QSpec, rows: int, hidden: int, out: torch.Tensor,
                           expected_epoch: int = 0, d_status: Optional[torch.Tensor] = None) -> Bound:
    """allgather_dequant with its arguments marshalled once (fcomm.Bound)."""
    qs = (QTensor * len(shards))(*[_qt(s if isinstance(s, (tuple, list)) else (s,))
                                   for s in shards])
    od = FMT_F32 if out.dtype == torch.float32 else FMT_BF16
    return Bound(load().fc_allgather_dequant,
                 [qs, len(shards), rows, hidden, spec, od, ctypes.c_void_p(_ptr(out)),
                  ctypes.c_uint32(expected_epoch & 0xFFFFFFFF), ctypes.c_void_p(_ptr(d_status)),
                  None], 9,
                 epoch_index=7, keep=(shards, out, d_status, qs))


def shard_views(q, spec: QSpec, rows: int, hidden: int, P: int):
    """The P shard payloads (views, no copy) of a whole payload q = (codes,
    scales, zeros) or tagged blocks, in the partition fc_allgather_dequant reads."""
    ng = groups(spec, rows, hidden)
    per = -(-ng // P)
    if spec.fmt in (FMT_INT8_TAGGED, FMT_INT4_TAGGED):
        nbg = 11 if spec.fmt == FMT_INT8_TAGGED else 2
        b = q if isinstance(q, torch.Tensor) else q[0]
        return [b[min(j * per, ng) * nbg * 16:min((j + 1) * per, ng) * nbg * 16] for j in range(P)]
    cb = spec.group if spec.fmt == FMT_INT8_SYM else spec.group // 2
    codes, scales, zeros = (tuple(q) + (None, None, None))[:3]
    out = []
    for j in range(P):
        g0, g1 = min(j * per, ng), min((j + 1) * per, ng)
        if g1 <= g0:
            out.append((None, None, None))
            continue
        out.append((codes[g0 * cb:g1 * cb], scales[g0:g1], None if zeros is None else zeros[g0:g1]))
    return out


def pack_tagged(x: torch.Tensor, epoch: int, blocks: torch.Tensor, stream=None):
    rows, hidden = _rows_hidden(x)
    _check(load().fc_pack_tagged(_ptr(x), rows, hidden, epoch, _ptr(blocks), _stream(stream)))


def bind_group_quantize_tagged(xs: Sequence[torch.Tensor], spec: QSpec, epoch: int,
                               blocks: Sequence[torch.Tensor],
                               d_status: Optional[torch.Tensor] = None) -> Bound:
    rows, hidden = _rows_hidden(xs[0])
    xp = (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])
    bp = (ctypes.c_void_p * len(blocks))(*[_ptr(b) for b in blocks])
    return Bound(load().fc_group_quantize_tagged,
                 [xp, len(xs), rows, hidden, spec, ctypes.c_uint32(epoch), bp,
                  ctypes.c_void_p(_ptr(d_status)), None], 8, 5,
                 keep=(tuple(xs), tuple(blocks), d_status))


def group_quantize_tagged(xs: Sequence[torch.Tensor], spec: QSpec, epoch: int,
                          blocks: Sequence[torch.Tensor], stream=None,
                          d_status: Optional[torch.Tensor] = None):
    """Quantize P bf16 slabs straight into self-synchronizing blocks."""
    bind_group_quantize_tagged(xs, spec, epoch, blocks, d_status)(stream)


def bind_pack_tagged_multi(xs: Sequence[torch.Tensor], epoch: int,
                           blocks: Sequence[torch.Tensor]) -> Bound:
    rows, hidden = _rows_hidden(xs[0])
    xp = (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])
    bp = (ctypes.c_void_p * len(blocks))(*[_ptr(b) for b in blocks])
    return Bound(load().fc_pack_tagged_multi,
                 [xp, len(xs), rows, hidden, ctypes.c_uint32(epoch), bp, None], 6, 4,
                 keep=(tuple(xs), tuple(blocks)))


def pack_tagged_multi(xs: Sequence[torch.Tensor], epoch: int, blocks: Sequence[torch.Tensor],
                      stream=None):
    bind_pack_tagged_multi(xs, epoch, blocks)(stream)


def allreduce_residual_rmsnorm(slabs, spec: QSpec, rows: int, hidden: int,
                               residual_in: torch.Tensor, residual_out: torch.Tensor,
                               gamma: torch.Tensor, eps: float, y: torch.Tensor,
                               requant_out=None, expected_epoch: int = 0,
                               d_status: Optional[torch.Tensor] = None, max_ctas: int = 0,
                               kernel: int = KERNEL_AUTO, stream=None):
    """The fused quantized All-Reduce + residual add + RMSNorm.

    slabs: list of P (codes, scales, zeros) tuples (INT8/INT4), or of bf16
    tensors / tagged-block tensors (BF16 / BF16_TAGGED)."""
    bind_allreduce_residual_rmsnorm(slabs, spec, rows, hidden, residual_in, residual_out, gamma,
                                    eps, y, requant_out, expected_epoch, d_status, max_ctas,
                                    kernel)(stream)


def bind_allreduce_residual_rmsnorm(slabs, spec: QSpec, rows: int, hidden: int,
                                    residual_in: torch.Tensor, residual_out: torch.Tensor,
                                    gamma: torch.Tensor, eps: float, y: torch.Tensor,
                                    requant_out=None, expected_epoch: int = 0,
                                    d_status: Optional[torch.Tensor] = None, max_ctas: int = 0,
                                    kernel: int = KERNEL_AUTO) -> Bound:
    """allreduce_residual_rmsnorm with its arguments marshalled once (Bound)."""
    qs = (QTensor * len(slabs))(*[_qt(s if isinstance(s, (tuple, list)) else (s,))
                                  for s in slabs])
    opts = LaunchOpts(max_ctas, kernel)
    P = ctypes.c_void_p
    args = [qs, len(slabs), rows, hidden, spec, P(_ptr(residual_in)), P(_ptr(residual_out)),
            P(_ptr(gamma)), ctypes.c_float(eps), _qt(requant_out), P(_ptr(y)),
            ctypes.c_uint32(expected_epoch), P(_ptr(d_status)), ctypes.byref(opts), None]
    return Bound(load().fc_allreduce_residual_rmsnorm_ex, args, 14, 11,
                 keep=(opts, tuple(slabs), residual_in, residual_out, gamma, y, requant_out,
                       d_status))


def token_split(spec: QSpec, P: int, rows: int, hidden: int):
    """(first subset's rows, wave rows) of the wave-aware token split."""
    sp, wv = ctypes.c_int64(), ctypes.c_int64()
    _check(load().fc_token_split(P, rows, hidden, spec, ctypes.byref(sp), ctypes.byref(wv)))
    return sp.value, wv.value


def select_protocol(rows: int, hidden: int, P: int, min_bits: int,
                    link_gbps: Optional[float] = None, barrier_us: float = 0.0):
    """(QSpec, estimated us) of the cost-guided format choice."""
    link = LinkModel(link_gbps, barrier_us) if link_gbps is not None else None
    choice, est = QSpec(), ctypes.c_double()
    _check(load().fc_select_protocol(rows, hidden, P, min_bits,
                                     ctypes.byref(link) if link is not None else None,
                                     ctypes.byref(choice), ctypes.byref(est)))
    return choice, est.value


def version() -> str:
    return load().fc_version().decode()


def protocol_estimate(rows: int, hidden: int, P: int, spec: QSpec,
                      link_gbps: Optional[float] = None, barrier_us: float = 0.0) -> float:
    """The selector's estimated us of one step in encoding `spec`."""
    link = LinkModel(link_gbps, barrier_us) if link_gbps is not None else None
    est = ctypes.c_double()
    _check(load().fc_protocol_estimate(rows, hidden, P, spec,
                                       ctypes.byref(link) if link is not None else None,
                                       ctypes.byref(est)))
    return est.value


# --------------------------------------------------- around the boundary ---
# stream: None (the current one of the tensors' device), a torch.cuda.Stream, or a
# raw handle, with which the caller keeps the tensors until the call has run.  A call by
# name checks and binds its arguments every time (10 to 15 us on GB300's host, 21 on a
# torch side stream); one kept from its bind_ function is a launch (2.9 us).
def _dtype(t: torch.Tensor, name: str) -> int:
    try:
        return {torch.bfloat16: FMT_BF16, torch.float32: FMT_F32}[t.dtype]
    except KeyError:
        raise ValueError(f"{name} must be bfloat16 or float32 (got {t.dtype})") from None


def _want(t: Optional[torch.Tensor], shape, dtype, name: str):
    """t's pointer, after checking its shape and type (None: NULL)."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype} (got {tuple(t.shape)} {t.dtype})")
    return _ptr(t)


def _mx4(q, rows: int, hidden: int, name: str) -> Mx4:
    if q is None:
        return Mx4(None, None)
    codes, scales = q
    n = mx4_scales_bytes(rows, hidden)
    if codes.dtype != torch.uint8 or tuple(codes.shape) != (rows, hidden // 2):
        raise ValueError(f"{name}'s codes must be [{rows}, {hidden // 2}] uint8 "
                         f"(got {tuple(codes.shape)} {codes.dtype})")
    if scales.dtype != torch.uint8 or scales.numel() != n:
        raise ValueError(f"{name}'s scales must be {n} uint8 (got {scales.numel()} {scales.dtype})")
    return Mx4(_ptr(codes), _ptr(scales))


def _one_device(*tensors) -> int:
    devices = {t.device for t in tensors if t is not None}
    if len(devices) != 1:
        raise ValueError(f"the tensors of a call are on one device (got {sorted(map(str, devices))})")
    return devices.pop().index


def _once(call: DeviceBound, stream):
    """Run a call bound for this one time.  On a torch stream other than the
    current one, its tensors' memory is kept from reuse until that stream is done.
    A stream given as a raw handle is the caller's, who may end it at any time: so
    are the tensors then, until the call has run."""
    call(stream)
    if isinstance(stream, torch.cuda.Stream):
        for t in call._keep:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)


def mx4_codes_bytes(rows: int, hidden: int) -> int:
    return load().fc_mx4_codes_bytes(rows, hidden)


def mx4_scales_bytes(rows: int, hidden: int) -> int:
    return load().fc_mx4_scales_bytes(rows, hidden)


def alloc_mx4(rows: int, hidden: int, device="cuda"):
    """Caller-owned (codes, scales) of a microscaled 4-bit [rows, hidden] tensor."""
    if hidden <= 0 or hidden % 32:
        raise ValueError(f"hidden must be a positive multiple of 32 (got {hidden})")
    return (torch.empty(rows, hidden // 2, dtype=torch.uint8, device=device),
            torch.empty(mx4_scales_bytes(rows, hidden), dtype=torch.uint8, device=device))


def bind_mx4_quantize(x: torch.Tensor, out) -> DeviceBound:
    rows, hidden = _rows_hidden(x)
    return DeviceBound(load().fc_mx4_quantize,
                 [ctypes.c_void_p(_ptr(x)), _dtype(x, "x"), rows, hidden,
                  _mx4(out, rows, hidden, "out"), None], 5,
                 keep=(x, *out), device=_one_device(x, *out))


def mx4_quantize(x: torch.Tensor, out, stream=None):
    """Quantize [rows, hidden] bf16 or fp32 to microscaled 4-bit out = (codes, scales)."""
    _once(bind_mx4_quantize(x, out), stream)


def bind_mx4_dequantize(q, out: torch.Tensor) -> DeviceBound:
    rows, hidden = _rows_hidden(out)
    return DeviceBound(load().fc_mx4_dequantize,
                 [_mx4(q, rows, hidden, "q"), rows, hidden, ctypes.c_void_p(_ptr(out)),
                  _dtype(out, "out"), None], 5,
                 keep=(*q, out), device=_one_device(*q, out))


def mx4_dequantize(q, out: torch.Tensor, stream=None):
    """out[rows, hidden] (bf16 or fp32) = the values q = (codes, scales) stands for."""
    _once(bind_mx4_dequantize(q, out), stream)


def bind_mx4_matmul(x, w, out: torch.Tensor, d_status: Optional[torch.Tensor] = None) -> DeviceBound:
    rows, features = _rows_hidden(out)
    if w[0].dim() != 2 or w[0].shape[0] != features:
        raise ValueError(f"w's codes must be [{features}, hidden / 2] (got {tuple(w[0].shape)})")
    hidden = 2 * w[0].shape[1]
    return DeviceBound(load().fc_mx4_matmul,
                 [_mx4(x, rows, hidden, "x"), _mx4(w, features, hidden, "w"), rows, features,
                  hidden, ctypes.c_void_p(_ptr(out)), _dtype(out, "out"),
                  ctypes.c_void_p(_want(d_status, (2,), torch.int32, "d_status")), None], 8,
                 keep=(*x, *w, out, d_status), device=_one_device(*x, *w, out, d_status))


def mx4_matmul(x, w, out: torch.Tensor, d_status: Optional[torch.Tensor] = None, stream=None):
    """out[rows, features] = x w^T of two microscaled tensors: x = (codes, scales) of
    [rows, hidden], w of [features, hidden], both as alloc_mx4 lays them out."""
    _once(bind_mx4_matmul(x, w, out, d_status), stream)


def _block_norm_spec(x, post_weight, gate, pre_weight, residual_scale, block_scale, post_eps,
                     pre_eps) -> BlockNormSpec:
    rows, hidden = _rows_hidden(x)
    gate_rows = 0
    if gate is not None:
        if gate.dim() != 2:
            raise ValueError("gate must be [gate_rows, hidden]")
        gate_rows = gate.shape[0]
    return BlockNormSpec(_want(post_weight, (hidden,), x.dtype, "post_weight"),
                         _want(gate, (gate_rows, hidden), x.dtype, "gate"),
                         _want(pre_weight, (hidden,), x.dtype, "pre_weight"),
                         gate_rows, residual_scale, block_scale, post_eps, pre_eps)


def bind_block_norm(x: torch.Tensor, residual_in: Optional[torch.Tensor],
                    residual_out: torch.Tensor, y: Optional[torch.Tensor] = None,
                    post_weight: Optional[torch.Tensor] = None,
                    gate: Optional[torch.Tensor] = None,
                    pre_weight: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                    block_scale: float = 1.0, post_eps: float = 1e-5, pre_eps: float = 1e-5,
                    y_mx4=None) -> DeviceBound:
    rows, hidden = _rows_hidden(x)
    spec = _block_norm_spec(x, post_weight, gate, pre_weight, residual_scale, block_scale, post_eps,
                            pre_eps)
    P = ctypes.c_void_p
    args = [P(_ptr(x)), P(_want(residual_in, x.shape, x.dtype, "residual_in")), rows, hidden,
            _dtype(x, "x"), ctypes.byref(spec),
            P(_want(residual_out, x.shape, x.dtype, "residual_out")),
            P(_want(y, x.shape, x.dtype, "y")), _mx4(y_mx4, rows, hidden, "y_mx4"), None]
    keep = (x, residual_in, residual_out, y, post_weight, gate, pre_weight, *(y_mx4 or ()))
    return DeviceBound(load().fc_block_norm, args, 9, keep=(*keep, spec), device=_one_device(*keep))


def block_norm(x: torch.Tensor, residual_in: Optional[torch.Tensor], residual_out: torch.Tensor,
               y: Optional[torch.Tensor] = None, stream=None, **spec):
    """The norms after a block and before the next, with the block's gate and the
    residual scale, in one pass over the rows:

    residual_out = residual_scale * residual_in + block_scale * gate * norm(x; post_weight)
    y            = norm(residual_out; pre_weight)

    x, residual_in, residual_out, y: [rows, hidden], bf16 or fp32.  Keywords:
    post_weight, pre_weight [hidden] and gate [gate_rows, hidden], each optional
    (rows / gate_rows neighbouring rows share a row of gate), residual_scale,
    block_scale, post_eps, pre_eps; y_mx4 = (codes, scales) receives y quantised."""
    _once(bind_block_norm(x, residual_in, residual_out, y, **spec), stream)


def alloc_block_norm_workspace(rows: int, hidden: int, gate_rows: int = 0, device="cuda"):
    """Workspace of one block_norm_backward call at a time (gate_rows: 0 without a gate)."""
    n = load().fc_block_norm_backward_workspace(rows, hidden, gate_rows)
    return torch.empty(max(n, 32), dtype=torch.uint8, device=device)


def bind_block_norm_backward(x: torch.Tensor, h: Optional[torch.Tensor],
                             dy: Optional[torch.Tensor], dh: Optional[torch.Tensor],
                             dx: torch.Tensor, workspace: torch.Tensor,
                             dresidual: Optional[torch.Tensor] = None,
                             dpost_weight: Optional[torch.Tensor] = None,
                             dgate: Optional[torch.Tensor] = None,
                             dpre_weight: Optional[torch.Tensor] = None,
                             post_weight: Optional[torch.Tensor] = None,
                             gate: Optional[torch.Tensor] = None,
                             pre_weight: Optional[torch.Tensor] = None,
                             residual_scale: float = 1.0, block_scale: float = 1.0,
                             post_eps: float = 1e-5, pre_eps: float = 1e-5,
                             d_status: Optional[torch.Tensor] = None) -> DeviceBound:
    rows, hidden = _rows_hidden(x)
    spec = _block_norm_spec(x, post_weight, gate, pre_weight, residual_scale, block_scale, post_eps,
                            pre_eps)
    need = load().fc_block_norm_backward_workspace(rows, hidden, spec.gate_rows)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    grads = BlockNormGrads(_want(dx, x.shape, x.dtype, "dx"),
                           _want(dresidual, x.shape, x.dtype, "dresidual"),
                           _want(dpost_weight, (hidden,), torch.float32, "dpost_weight"),
                           _want(dgate, (spec.gate_rows, hidden), x.dtype, "dgate"),
                           _want(dpre_weight, (hidden,), torch.float32, "dpre_weight"))
    P = ctypes.c_void_p
    args = [P(_ptr(x)), P(_want(h, x.shape, x.dtype, "h")), P(_want(dy, x.shape, x.dtype, "dy")),
            P(_want(dh, x.shape, x.dtype, "dh")), rows, hidden, _dtype(x, "x"),
            ctypes.byref(spec), ctypes.byref(grads), P(_ptr(workspace)),
            P(_want(d_status, (2,), torch.int32, "d_status")), None]
    keep = (x, h, dy, dh, dx, workspace, dresidual, dpost_weight, dgate, dpre_weight, post_weight,
            gate, pre_weight, d_status)
    return DeviceBound(load().fc_block_norm_backward, args, 11, keep=(*keep, spec, grads),
                 device=_one_device(*keep))


def block_norm_backward(x: torch.Tensor, h: Optional[torch.Tensor], dy: Optional[torch.Tensor],
                        dh: Optional[torch.Tensor], dx: torch.Tensor, workspace: torch.Tensor,
                        stream=None, **kw):
    """Gradient of block_norm.  x and h (= residual_out) are what the forward pass
    read and wrote, dy and dh the gradients of y and residual_out; writes dx and,
    where given, dresidual, dpost_weight, dpre_weight (fp32) and dgate.  Keywords
    as block_norm's; workspace from alloc_block_norm_workspace."""
    _once(bind_block_norm_backward(x, h, dy, dh, dx, workspace, **kw), stream)


# ------------------------------------------------------------- layer norm ---
def bind_layer_norm(x: torch.Tensor, y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                    bias: Optional[torch.Tensor] = None,
                    residual_in: Optional[torch.Tensor] = None,
                    residual_out: Optional[torch.Tensor] = None, eps: float = 1e-5,
                    stats: Optional[torch.Tensor] = None) -> DeviceBound:
    rows, hidden = _rows_hidden(x)
    P = ctypes.c_void_p
    args = [P(_ptr(x)), P(_want(residual_in, x.shape, x.dtype, "residual_in")), rows, hidden,
            _dtype(x, "x"), P(_want(weight, (hidden,), x.dtype, "weight")),
            P(_want(bias, (hidden,), x.dtype, "bias")), eps,
            P(_want(residual_out, x.shape, x.dtype, "residual_out")),
            P(_want(y, x.shape, x.dtype, "y")),
            P(_want(stats, (rows, 2), torch.float32, "stats")), None]
    keep = (x, residual_in, weight, bias, residual_out, y, stats)
    return DeviceBound(load().fc_layer_norm, args, 11, keep=keep, device=_one_device(*keep))


def layer_norm(x: torch.Tensor, y: torch.Tensor, stream=None, **kw):
    """Residual add and layer norm in one pass over the rows:

    residual_out = x + residual_in
    y            = (h - mean(h)) / sqrt(var(h) + eps) * weight + bias, h = residual_out

    x, y and, given together, residual_in and residual_out (without them h is x):
    [rows, hidden], bf16 or fp32.  Keywords: weight and bias [hidden], each optional,
    eps, and stats, fp32 [rows, 2], which receives each row's mean and inverse
    deviation for layer_norm_backward."""
    _once(bind_layer_norm(x, y, **kw), stream)


def alloc_layer_norm_workspace(rows: int, hidden: int, device="cuda"):
    """Workspace of one layer_norm_backward call at a time."""
    n = load().fc_layer_norm_backward_workspace(rows, hidden)
    return torch.empty(max(n, 32), dtype=torch.uint8, device=device)


def bind_layer_norm_backward(h: torch.Tensor, stats: torch.Tensor, dy: torch.Tensor,
                             dx: torch.Tensor, workspace: torch.Tensor,
                             dh: Optional[torch.Tensor] = None,
                             weight: Optional[torch.Tensor] = None,
                             dweight: Optional[torch.Tensor] = None,
                             dbias: Optional[torch.Tensor] = None,
                             d_status: Optional[torch.Tensor] = None) -> DeviceBound:
    rows, hidden = _rows_hidden(h)
    need = load().fc_layer_norm_backward_workspace(rows, hidden)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    P = ctypes.c_void_p
    args = [P(_ptr(h)), P(_want(stats, (rows, 2), torch.float32, "stats")),
            P(_want(dy, h.shape, h.dtype, "dy")), P(_want(dh, h.shape, h.dtype, "dh")), rows, hidden,
            _dtype(h, "h"), P(_want(weight, (hidden,), h.dtype, "weight")),
            P(_want(dx, h.shape, h.dtype, "dx")),
            P(_want(dweight, (hidden,), torch.float32, "dweight")),
            P(_want(dbias, (hidden,), torch.float32, "dbias")), P(_ptr(workspace)),
            P(_want(d_status, (2,), torch.int32, "d_status")), None]
    keep = (h, stats, dy, dh, weight, dx, dweight, dbias, workspace, d_status)
    return DeviceBound(load().fc_layer_norm_backward, args, 13, keep=keep, device=_one_device(*keep))


def layer_norm_backward(h: torch.Tensor, stats: torch.Tensor, dy: torch.Tensor, dx: torch.Tensor,
                        workspace: torch.Tensor, stream=None, **kw):
    """Gradient of layer_norm.  h is what was normed (residual_out, or x), stats what the
    forward pass wrote, dy the gradient of y; dx receives that of h, which is that of
    x and of residual_in.  Keywords: dh (the gradient of residual_out by itself),
    weight, dweight and dbias (fp32), d_status; workspace from
    alloc_layer_norm_workspace."""
    _once(bind_layer_norm_backward(h, stats, dy, dx, workspace, **kw), stream)


# ------------------------------------------------ 8-bit floating point -----
def fp8_scales(rows: int, hidden: int, block_rows: int = 1) -> int:
    return load().fc_fp8_scales(rows, hidden, block_rows)


def alloc_fp8(rows: int, hidden: int, block_rows: int = 1, device="cuda"):
    """Caller-owned (codes, scales) of an 8-bit [rows, hidden] tensor with a scale for each
    block of block_rows (1: an activation's, 128: a weight's) by 128."""
    if hidden <= 0 or hidden % 16:
        raise ValueError(f"hidden must be a positive multiple of 16 (got {hidden})")
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows must be 1 or 128 (got {block_rows})")
    return (torch.empty(rows, hidden, dtype=torch.uint8, device=device),
            torch.empty(-(-rows // block_rows), -(-hidden // 128), dtype=torch.float32, device=device))


def _fp8(q, rows: int, hidden: int, block_rows: int, name: str) -> Fp8:
    codes, scales = q
    if codes.dtype != torch.uint8 or tuple(codes.shape) != (rows, hidden):
        raise ValueError(f"{name}'s codes must be [{rows}, {hidden}] uint8 "
                         f"(got {tuple(codes.shape)} {codes.dtype})")
    want = (-(-rows // block_rows), -(-hidden // 128))
    if scales.dtype != torch.float32 or tuple(scales.shape) != want:
        raise ValueError(f"{name}'s scales must be {want} float32 (got {tuple(scales.shape)} {scales.dtype})")
    return Fp8(_ptr(codes), _ptr(scales))


def _block_rows(q, rows: int) -> int:
    """1 or 128, by the scales' rows (one row is the same block either way)."""
    return 1 if q[1].dim() == 2 and q[1].shape[0] == rows else 128


def bind_fp8_quantize(x: torch.Tensor, out) -> DeviceBound:
    rows, hidden = _rows_hidden(x)
    br = _block_rows(out, rows)
    return DeviceBound(load().fc_fp8_quantize,
                       [ctypes.c_void_p(_ptr(x)), _dtype(x, "x"), rows, hidden, br,
                        _fp8(out, rows, hidden, br, "out"), None], 6,
                       keep=(x, *out), device=_one_device(x, *out))


def fp8_quantize(x: torch.Tensor, out, stream=None):
    """Quantize [rows, hidden] bf16 or fp32 to 8-bit out = (codes, scales), in the blocks
    that out was laid out for (alloc_fp8)."""
    _once(bind_fp8_quantize(x, out), stream)


def bind_fp8_dequantize(q, out: torch.Tensor) -> DeviceBound:
    rows, hidden = _rows_hidden(out)
    br = _block_rows(q, rows)
    return DeviceBound(load().fc_fp8_dequantize,
                       [_fp8(q, rows, hidden, br, "q"), rows, hidden, br, ctypes.c_void_p(_ptr(out)),
                        _dtype(out, "out"), None], 6,
                       keep=(*q, out), device=_one_device(*q, out))


def fp8_dequantize(q, out: torch.Tensor, stream=None):
    """out[rows, hidden] (bf16 or fp32) = the values q = (codes, scales) stands for."""
    _once(bind_fp8_dequantize(q, out), stream)


def bind_fp8_matmul(x, w, out: torch.Tensor, d_status: Optional[torch.Tensor] = None) -> DeviceBound:
    rows, features = _rows_hidden(out)
    if w[0].dim() != 2 or w[0].shape[0] != features:
        raise ValueError(f"w's codes must be [{features}, hidden] (got {tuple(w[0].shape)})")
    hidden = w[0].shape[1]
    return DeviceBound(load().fc_fp8_matmul,
                       [_fp8(x, rows, hidden, 1, "x"), _fp8(w, features, hidden, 128, "w"), rows,
                        features, hidden, ctypes.c_void_p(_ptr(out)), _dtype(out, "out"),
                        ctypes.c_void_p(_want(d_status, (2,), torch.int32, "d_status")), None], 8,
                       keep=(*x, *w, out, d_status), device=_one_device(*x, *w, out, d_status))


def fp8_matmul(x, w, out: torch.Tensor, d_status: Optional[torch.Tensor] = None, stream=None):
    """out[rows, features] (bf16 or fp32) = x w^T of two 8-bit tensors: x = (codes, scales)
    of [rows, hidden] with block_rows 1, w of [features, hidden] with block_rows 128."""
    _once(bind_fp8_matmul(x, w, out, d_status), stream)


# ------------------------------------------------- gated feed-forward ------
def bind_gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, out: torch.Tensor,
                   activation: int = ACT_SILU, gate: Optional[torch.Tensor] = None,
                   up: Optional[torch.Tensor] = None,
                   d_status: Optional[torch.Tensor] = None) -> DeviceBound:
    rows, hidden = _rows_hidden(x)
    features, B, P = out.shape[-1], torch.bfloat16, ctypes.c_void_p
    args = [P(_want(x, (rows, hidden), B, "x")), P(_want(w_gate, (features, hidden), B, "w_gate")),
            P(_want(w_up, (features, hidden), B, "w_up")), rows, features, hidden, activation,
            P(_want(out, (rows, features), B, "out")), P(_want(gate, (rows, features), B, "gate")),
            P(_want(up, (rows, features), B, "up")),
            P(_want(d_status, (2,), torch.int32, "d_status")), None]
    keep = (x, w_gate, w_up, out, gate, up, d_status)
    return DeviceBound(load().fc_gated_ffn, args, 11, keep=keep, device=_one_device(*keep))


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, out: torch.Tensor,
              stream=None, **kw):
    """The gated feed-forward block's projections, activation and product in one kernel:
    out[rows, features] = act(x w_gate^T) * (x w_up^T), all bf16, x [rows, hidden], w_gate
    and w_up [features, hidden].  Keywords: activation (ACT_SILU or ACT_GELU_TANH); gate
    and up [rows, features], which receive the two projections for
    gated_ffn_backward; d_status."""
    _once(bind_gated_ffn(x, w_gate, w_up, out, **kw), stream)


def alloc_gated_ffn_workspace(rows: int, features: int, device="cuda", factor_terms: int = 0):
    """Workspace of one gated_ffn_backward call (with these factor_terms) at a time."""
    n = load().fc_gated_ffn_backward_ex_workspace(rows, features, factor_terms)
    return torch.empty(max(n, 32), dtype=torch.uint8, device=device)


def bind_gated_ffn_backward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                            gate: torch.Tensor, up: torch.Tensor, dout: torch.Tensor,
                            workspace: torch.Tensor, dx: Optional[torch.Tensor] = None,
                            dw_gate: Optional[torch.Tensor] = None,
                            dw_up: Optional[torch.Tensor] = None, activation: int = ACT_SILU,
                            d_status: Optional[torch.Tensor] = None,
                            factor_terms: int = 0) -> DeviceBound:
    rows, hidden = _rows_hidden(x)
    features, B, P = dout.shape[-1], torch.bfloat16, ctypes.c_void_p
    need = load().fc_gated_ffn_backward_ex_workspace(rows, features, factor_terms)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    act, weight = (rows, features), (features, hidden)
    args = [P(_want(x, (rows, hidden), B, "x")), P(_want(w_gate, weight, B, "w_gate")),
            P(_want(w_up, weight, B, "w_up")), P(_want(gate, act, B, "gate")),
            P(_want(up, act, B, "up")), P(_want(dout, act, B, "dout")), rows, features, hidden,
            activation, P(_want(dx, (rows, hidden), B, "dx")), P(_want(dw_gate, weight, B, "dw_gate")),
            P(_want(dw_up, weight, B, "dw_up")), P(_ptr(workspace)),
            P(_want(d_status, (2,), torch.int32, "d_status")), None]
    keep = (x, w_gate, w_up, gate, up, dout, dx, dw_gate, dw_up, workspace, d_status)
    if factor_terms == 0:
        return DeviceBound(load().fc_gated_ffn_backward, args, 15, keep=keep, device=_one_device(*keep))
    args.insert(10, factor_terms)
    return DeviceBound(load().fc_gated_ffn_backward_ex, args, 16, keep=keep, device=_one_device(*keep))


def gated_ffn_backward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, gate: torch.Tensor,
                       up: torch.Tensor, dout: torch.Tensor, workspace: torch.Tensor, stream=None,
                       **kw):
    """Gradient of gated_ffn.  gate and up are the projections that the forward pass kept,
    dout the gradient of out.  Keywords: dx and (both or neither) dw_gate and dw_up, bf16,
    which receive the gradients; activation; d_status; factor_terms (0: dg and du in two bf16
    numbers each for up to 128 tokens or 2^19 factors, else in one; 2: always in two).
    workspace from alloc_gated_ffn_workspace, for the same factor_terms."""
    _once(bind_gated_ffn_backward(x, w_gate, w_up, gate, up, dout, workspace, **kw), stream)
