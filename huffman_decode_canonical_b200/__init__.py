"""Python binding of libentro (argument marshalling only).

Every step of the path -- quantization and Huffman coding on the host, decoding,
dequantization and the fused GEMV on the GPU -- runs inside ``libentro.so``;
this module turns numpy / torch objects into pointers and sizes for the C ABI
declared in ``include/entro.h`` and turns return codes into exceptions.
PyTorch is used for device memory and streams only.  There is no fallback:
importing this package fails when the shared library is missing, and device
calls need a CUDA GPU.

The method is EntroLLM ("EntroLLM: Entropy Encoded Weight Compression for
Efficient Large Language Model Inference on Edge Devices", arXiv
2505.02380v4): mixed tensor-level quantization, Huffman coding of the codes and
parallel decoding of chunks; with the lane-interleaved, decode-on-demand
storage of "LazyWeights: Decode-on-Demand Edge LLMs" (arXiv 2611.17108v1).
"""
from __future__ import annotations

import ctypes
import os
from typing import List, NamedTuple, Optional, Sequence, Union

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libentro.so")

OK = 0
E_INVAL, E_LIMIT, E_FORMAT, E_CORRUPT, E_OVERRUN, E_NOMEM, E_CUDA, E_TIMEOUT = -1, -2, -3, -4, -5, -6, -7, -8
QUANT_AUTO, QUANT_UNSIGNED, QUANT_ASYM = 0, 1, 2
SCHEME_UNSIGNED, SCHEME_ASYM = 0, 1
FORMAT_SINGLE, FORMAT_LANES, FORMAT_ROWS, FORMAT_ROWS_CO = 1, 2, 3, 4
GROUP_GEMV, GROUP_BF16 = 1, 2


class EntroError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        detail = f" [{_lib.entro_last_cuda_error().decode()}]" if code == E_CUDA else ""
        super().__init__(f"{what}: {_strerror(code)} ({code}){detail}")


class _Opts(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("quant_mode", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("format", ctypes.c_int32), ("chunk_symbols", ctypes.c_int64), ("threads", ctypes.c_int32),
                ("lanes", ctypes.c_int32)]


class _KVCache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("slots", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("type", ctypes.c_int32)]


class _Info(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("scheme", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("format", ctypes.c_int32), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("n", ctypes.c_int64), ("chunk_symbols", ctypes.c_int64), ("n_chunks", ctypes.c_int64),
                ("scale", ctypes.c_float), ("zero", ctypes.c_int32), ("payload_bytes", ctypes.c_uint64),
                ("index_bytes", ctypes.c_uint64), ("blob_bytes", ctypes.c_uint64), ("coded_bits", ctypes.c_uint64),
                ("max_chunk_words", ctypes.c_uint32), ("lanes", ctypes.c_uint32),
                ("lengths", ctypes.c_uint8 * 256)]


EXPORTS = ["entro_encode", "entro_blob_from_bytes", "entro_blob_bytes", "entro_blob_info", "entro_blob_free",
           "entro_device_bytes", "entro_upload", "entro_tensor_free", "entro_decode_codes",
           "entro_decode_dequant_bf16", "entro_decode_gemv", "entro_group_table_bytes", "entro_group_prepare",
           "entro_group_launch", "entro_group_free", "entro_strerror", "entro_version", "entro_last_cuda_error",
           "entro_decode_gemv_group_static", "entro_set_overlap", "entro_test_stall_tables",
           "entro_quantize_tokens", "entro_unpack_codes", "entro_matmul_i8",
           "entro_kv_append", "entro_kv_read", "entro_kv_attend_workspace", "entro_kv_attend", "entro_attention_prompt"]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python huffman_decode_canonical_b200/build.py` "
                          "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, U64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
    F32 = ctypes.c_float
    PP = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "entro_encode": ([P, I64, I64, ctypes.POINTER(_Opts), PP], I32),
        "entro_blob_from_bytes": ([P, U64, PP], I32),
        "entro_blob_bytes": ([P, PP, ctypes.POINTER(U64)], I32),
        "entro_blob_info": ([P, ctypes.POINTER(_Info)], I32),
        "entro_blob_free": ([P], None),
        "entro_device_bytes": ([P, ctypes.POINTER(U64)], I32),
        "entro_upload": ([P, P, U64, P, PP], I32),
        "entro_tensor_free": ([P], None),
        "entro_decode_codes": ([P, P, P, P], I32),
        "entro_decode_dequant_bf16": ([P, P, P, P], I32),
        "entro_decode_gemv": ([P, P, I32, P, P, P], I32),
        "entro_group_table_bytes": ([I32], U64),
        "entro_group_prepare": ([P, I32, I32, P, P, P, I32, P, U64, P, PP], I32),
        "entro_group_launch": ([P, P, P], I32),
        "entro_group_free": ([P], None),
        "entro_strerror": ([I32], ctypes.c_char_p),
        "entro_version": ([], I32),
        "entro_last_cuda_error": ([], ctypes.c_char_p),
        "entro_decode_gemv_group_static": ([P, P, P, I32, I32, P, P], I32),
        "entro_set_overlap": ([I32], I32),
        "entro_test_stall_tables": ([ctypes.c_uint32], ctypes.c_uint32),
        "entro_kv_append": ([P, P, I64, I64, P, I64, I64, I64, P, P, I64, I32, P, P, I32, P, P], I32),
        "entro_kv_read": ([P, P, I64, I64, P, I64, I64, I64, P, P, I64, I32, P, I32, P, P], I32),
        "entro_kv_attend_workspace": ([P, ctypes.POINTER(U64)], I32),
        "entro_kv_attend": ([P, P, I64, I64, I32, P, I64, I32, P, P, I32, F32, P, I64, I64, P, U64, P, P], I32),
        "entro_attention_prompt": ([I32, I32, P, I64, I64, I32, I64, P, I64, I64, P, I64, I64, I32, I64, P, P, I32, F32, P, I64,
                                    I64, P, P], I32),
        "entro_quantize_tokens": ([P, I32, I64, I64, I64, P, I64, P, P, P], I32),
        "entro_unpack_codes": ([P, I32, I64, I64, P, I64, P], I32),
        "entro_matmul_i8": ([P, I64, P, P, I64, P, I32, I64, I64, I64, P, F32, P, I32, P, I32, I64, P, P], I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def _strerror(code: int) -> str:
    return _lib.entro_strerror(code).decode()


def _check(code: int, what: str):
    if code != OK:
        raise EntroError(code, what)


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> Optional[int]:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dptr(t: Optional[torch.Tensor]) -> Optional[ctypes.c_void_p]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


# ------------------------------------------------------------------ host side

class Blob:
    """One encoded tensor held on the host (library-owned serialized bytes)."""

    def __init__(self, handle: ctypes.c_void_p):
        self._h = handle

    @classmethod
    def encode(cls, w, bits: int = 8, quant_mode: int = QUANT_AUTO, max_len: int = 0,
               fmt: int = FORMAT_LANES, chunk_symbols: int = 0, threads: int = 0, lanes: int = 0) -> "Blob":
        if isinstance(w, torch.Tensor):
            w = w.detach().to("cpu", torch.float32).numpy()
        w = np.ascontiguousarray(w, dtype=np.float32)
        if w.ndim != 2:
            raise ValueError("w must be 2-D [rows, cols]")
        opts = _Opts(bits, quant_mode, max_len, fmt, chunk_symbols, threads, lanes)
        h = ctypes.c_void_p()
        _check(_lib.entro_encode(w.ctypes.data_as(ctypes.c_void_p) if w.size else None, w.shape[0], w.shape[1],
                                 ctypes.byref(opts), ctypes.byref(h)), "entro_encode")
        return cls(h)

    @classmethod
    def from_bytes(cls, data: bytes) -> "Blob":
        buf = np.frombuffer(data, np.uint8)
        h = ctypes.c_void_p()
        _check(_lib.entro_blob_from_bytes(buf.ctypes.data_as(ctypes.c_void_p), buf.size, ctypes.byref(h)),
               "entro_blob_from_bytes")
        return cls(h)

    def to_bytes(self) -> bytes:
        p = ctypes.c_void_p()
        n = ctypes.c_uint64()
        _check(_lib.entro_blob_bytes(self._h, ctypes.byref(p), ctypes.byref(n)), "entro_blob_bytes")
        return ctypes.string_at(p, n.value)

    def info(self) -> dict:
        i = _Info()
        _check(_lib.entro_blob_info(self._h, ctypes.byref(i)), "entro_blob_info")
        d = {f: getattr(i, f) for f, _ in _Info._fields_ if f != "lengths"}
        d["lengths"] = np.frombuffer(bytes(i.lengths), np.uint8).copy()
        return d

    def device_bytes(self) -> int:
        n = ctypes.c_uint64()
        _check(_lib.entro_device_bytes(self._h, ctypes.byref(n)), "entro_device_bytes")
        return n.value

    def close(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.entro_blob_free(self._h)
            self._h = None

    def __del__(self):
        self.close()


def encode(w, **kw) -> Blob:
    return Blob.encode(w, **kw)


# ------------------------------------------------------------------ device side

class DeviceTensor:
    """A blob's decode image in device memory (a torch uint8 buffer) + its handle."""

    def __init__(self, blob: Blob, device: Optional[torch.device] = None,
                 stream: Optional[torch.cuda.Stream] = None):
        device = torch.device(device if device is not None else "cuda")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        info = blob.info()
        self.rows, self.cols, self.n = info["rows"], info["cols"], info["n"]
        self.bits, self.format = info["bits"], info["format"]
        self.chunk_symbols, self.n_chunks = info["chunk_symbols"], info["n_chunks"]
        self.payload_bytes, self.index_bytes = info["payload_bytes"], info["index_bytes"]
        self.info = info
        nbytes = blob.device_bytes()
        with torch.cuda.device(device):
            self.mem = torch.empty(nbytes, dtype=torch.uint8, device=device)
            h = ctypes.c_void_p()
            _check(_lib.entro_upload(blob._h, _dptr(self.mem), nbytes, _stream_ptr(stream), ctypes.byref(h)),
                   "entro_upload")
        self._h = h
        self.device = device

    # output buffers ---------------------------------------------------
    def codes_nbytes(self) -> int:
        return self.n if self.bits == 8 else (self.n + 1) // 2

    def empty_codes(self) -> torch.Tensor:
        return torch.empty(max(self.codes_nbytes(), 1), dtype=torch.uint8, device=self.device)

    def empty_bf16(self) -> torch.Tensor:
        return torch.empty((self.rows, self.cols), dtype=torch.bfloat16, device=self.device)

    # calls ------------------------------------------------------------
    def decode_codes(self, out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        out = self.empty_codes() if out is None else out
        _check(_lib.entro_decode_codes(self._h, _dptr(out), _dptr(status), _stream_ptr(stream)),
               "entro_decode_codes")
        return out

    def decode_dequant_bf16(self, out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        out = self.empty_bf16() if out is None else out
        _check(_lib.entro_decode_dequant_bf16(self._h, _dptr(out), _dptr(status), _stream_ptr(stream)),
               "entro_decode_dequant_bf16")
        return out

    def decode_gemv(self, x: torch.Tensor, y: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        if x.dim() == 1:
            x = x.unsqueeze(0)
        batch = x.shape[0]
        if x.dtype != torch.bfloat16 or not x.is_contiguous() or x.shape[1] != self.cols:
            raise ValueError("x must be a contiguous bf16 [batch, cols] tensor")
        y = torch.empty((batch, self.rows), dtype=torch.float32, device=self.device) if y is None else y
        _check(_lib.entro_decode_gemv(self._h, _dptr(x), batch, _dptr(y), _dptr(status), _stream_ptr(stream)),
               "entro_decode_gemv")
        return y

    def matmul(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
               status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """x @ w.T for any number of tokens (a prompt): x bf16 or fp16 [tokens, cols], or `QuantTokens` that
        several projections share.  The codes are decoded into a buffer of their own for the call, the tokens
        quantized to 8 bits each with its scale, and multiplied in integers (`matmul_i8`)."""
        if not isinstance(x, QuantTokens) and (x.dim() != 2 or x.shape[1] != self.cols):
            raise ValueError("x must be a [tokens, cols] tensor")
        with _on(self.device, stream) as s:
            codes = self.empty_codes()
            _check(_lib.entro_decode_codes(self._h, _dptr(codes), _dptr(status), s), "entro_decode_codes")
            if self.bits == 8 and self.cols % 16 == 0:
                w = codes[:self.n].view(self.rows, self.cols)
            else:
                pitch = _pitch(self.cols)
                w = torch.empty((self.rows, pitch), dtype=torch.uint8, device=self.device)
                _check(_lib.entro_unpack_codes(_dptr(codes), self.bits, self.rows, self.cols, _dptr(w), pitch, s),
                       "entro_unpack_codes")
                w = w[:, :self.cols]
            xq = x if isinstance(x, QuantTokens) else quantize_tokens(x, stream=stream)
            return matmul_i8(xq, w, self.info["scale"], self.info["zero"], out=out, out_dtype=out_dtype, status=status,
                             stream=stream)

    def close(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.entro_tensor_free(self._h)
            self._h = None

    def __del__(self):
        self.close()


def upload(blob: Blob, device=None, stream=None) -> DeviceTensor:
    return DeviceTensor(blob, device, stream)


class Group:
    """One launch over many tensors (fused GEMV of a decode step, or whole-model bf16 decode)."""

    def __init__(self, tensors: Sequence[DeviceTensor], kind: int, xs: Optional[Sequence[torch.Tensor]] = None,
                 ys: Optional[Sequence[torch.Tensor]] = None, outs: Optional[Sequence[torch.Tensor]] = None,
                 batch: int = 1, stream: Optional[torch.cuda.Stream] = None):
        count = len(tensors)
        self.tensors = list(tensors)
        self.xs, self.ys, self.outs = xs, ys, outs       # keep the buffers alive
        dev = tensors[0].device
        nbytes = int(_lib.entro_group_table_bytes(count))
        self.table = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        arr = ctypes.c_void_p * count
        th = arr(*[t._h for t in tensors])
        xp = arr(*[x.data_ptr() for x in xs]) if xs is not None else None
        yp = arr(*[y.data_ptr() for y in ys]) if ys is not None else None
        op = arr(*[o.data_ptr() for o in outs]) if outs is not None else None
        h = ctypes.c_void_p()
        _check(_lib.entro_group_prepare(th, count, kind, xp, yp, op, batch, _dptr(self.table), nbytes,
                                        _stream_ptr(stream), ctypes.byref(h)), "entro_group_prepare")
        self._h = h

    def launch(self, status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        _check(_lib.entro_group_launch(self._h, _dptr(status), _stream_ptr(stream)), "entro_group_launch")

    def close(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.entro_group_free(self._h)
            self._h = None

    def __del__(self):
        self.close()


STATIC_GROUP_MAX = 512


def decode_gemv_group_static(tensors: Sequence[DeviceTensor], xs: Sequence[torch.Tensor],
                             ys: Sequence[torch.Tensor], batch: int = 1, status: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None) -> None:
    """Grouped fused GEMV whose work table lives inside the library (no device allocation)."""
    count = len(tensors)
    if count < 1 or len(xs) != count or len(ys) != count:
        raise ValueError("need one x and one y per tensor")
    for t, x, y in zip(tensors, xs, ys):
        if (x.dtype != torch.bfloat16 or not x.is_contiguous() or x.dim() != 2 or x.shape != (batch, t.cols)
                or x.device != t.device):
            raise ValueError("each x must be a contiguous bf16 [batch, cols] tensor on the tensors' device")
        if (y.dtype != torch.float32 or not y.is_contiguous() or y.dim() != 2 or y.shape != (batch, t.rows)
                or y.device != t.device):
            raise ValueError("each y must be a contiguous fp32 [batch, rows] tensor on the tensors' device")
    arr = ctypes.c_void_p * count
    _check(_lib.entro_decode_gemv_group_static(arr(*[t._h for t in tensors]), arr(*[x.data_ptr() for x in xs]),
                                               arr(*[y.data_ptr() for y in ys]), count, batch, _dptr(status),
                                               _stream_ptr(stream)), "entro_decode_gemv_group_static")


# ------------------------------------------------------------------ around the coded weights

F32, BF16, F16, U8, S8 = range(5)
_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16, torch.uint8: U8, torch.int8: S8}


class _on:
    """The tensors' device as the current one, and new buffers from the pool of the stream that is launched on."""

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        self.guards = []
        if stream is not None:
            if stream.device != device:
                raise ValueError("the stream belongs to another device than the tensors")
            self.guards.append(torch.cuda.stream(stream))
        elif device.index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(device))
        self.device = device

    def __enter__(self) -> int:
        for g in self.guards:
            g.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *e):
        for g in reversed(self.guards):
            g.__exit__(*e)


def _inputs(device: torch.device, **tensors):
    """Refuses what the kernels must not be given: tensors of other devices, or ones that ask for gradients."""
    if device.type != "cuda":
        raise ValueError("expected CUDA tensors")
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient: this call has none (use torch.no_grad())")


def _pitch(cols: int) -> int:
    return (cols + 15) // 16 * 16


class QuantTokens(NamedTuple):
    """Activations in 8 bits: codes int8 [tokens, cols] (rows a multiple of 16 bytes apart), scale fp32 [tokens], sum
    int32 [tokens] (of a token's codes)."""
    codes: torch.Tensor
    scale: torch.Tensor
    sum: torch.Tensor


def quantize_tokens(x: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> QuantTokens:
    """bf16 or fp16 [tokens, cols] (any row stride) to codes 127 x / max|x| of each token, with scale max|x| / 127."""
    if x.dtype not in (torch.bfloat16, torch.float16) or x.dim() != 2 or x.shape[1] < 1 or x.stride(1) != 1:
        raise ValueError("x must be a bf16 or fp16 [tokens, cols] tensor with adjacent columns")
    _inputs(x.device, x=x)
    tokens, cols = x.shape
    pitch = _pitch(cols)
    with _on(x.device, stream) as s:
        codes = torch.empty((tokens, pitch), dtype=torch.int8, device=x.device)
        scale = torch.empty(tokens, dtype=torch.float32, device=x.device)
        total = torch.empty(tokens, dtype=torch.int32, device=x.device)
        _check(_lib.entro_quantize_tokens(x.data_ptr(), _TYPES[x.dtype], tokens, cols, x.stride(0) if tokens > 1 else pitch,
                                          codes.data_ptr(), pitch, scale.data_ptr(), total.data_ptr(), s),
               "entro_quantize_tokens")
    return QuantTokens(codes if pitch == cols else codes[:, :cols], scale, total)


def matmul_i8(x: QuantTokens, w: torch.Tensor, w_scale: Union[float, torch.Tensor], w_zero: Union[None, int, torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
              status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y[t, n] = x.scale[t] * w_scale[n] * sum_k x.codes[t, k] * (w[n, k] - w_zero[n]).

    w uint8 or int8 [rows, cols], adjacent columns, rows a multiple of 16 bytes apart; w_scale a number or fp32 [rows];
    w_zero a whole number, int32 [rows] or None (0).  out: fp32, bf16 or fp16 [tokens, rows] with adjacent columns."""
    q = x.codes
    if w.dtype not in (torch.uint8, torch.int8) or w.dim() != 2 or w.shape[1] < 1 or w.stride(1) != 1:
        raise ValueError("w must be a uint8 or int8 [rows, cols] tensor with adjacent columns")
    rows, cols = w.shape
    tokens = q.shape[0] if q.dim() == 2 else -1
    if q.dtype != torch.int8 or q.dim() != 2 or q.shape[1] != cols or q.stride(1) != 1:
        raise ValueError("x.codes must be an int8 [tokens, cols] tensor with adjacent columns")
    for t, dtype, name in ((x.scale, torch.float32, "x.scale"), (x.sum, torch.int32, "x.sum")):
        if t.dtype != dtype or t.shape != (tokens,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} [tokens] tensor")
    ws, wz = torch.is_tensor(w_scale), torch.is_tensor(w_zero)
    if ws and (w_scale.dtype != torch.float32 or w_scale.shape != (rows,) or not w_scale.is_contiguous()):
        raise ValueError("w_scale must be a number or a contiguous fp32 [rows] tensor")
    if wz and (w_zero.dtype != torch.int32 or w_zero.shape != (rows,) or not w_zero.is_contiguous()):
        raise ValueError("w_zero must be a whole number or a contiguous int32 [rows] tensor")
    if not wz and w_zero is not None and not -2 ** 31 <= w_zero < 2 ** 31:
        raise ValueError("w_zero must fit 32 bits")
    _inputs(w.device, w=w, codes=q, scale=x.scale, sum=x.sum, w_scale=w_scale if ws else None, w_zero=w_zero if wz else None,
            out=out, status=status)
    # a single row's stride says nothing
    ldq, ldw = (q.stride(0) if tokens > 1 else _pitch(cols)), (w.stride(0) if rows > 1 else _pitch(cols))
    if ldq % 16 or ldw % 16 or q.data_ptr() % 16 or w.data_ptr() % 16:
        raise ValueError("x.codes and w must begin on 16 bytes, their rows a multiple of 16 bytes apart")
    with _on(w.device, stream) as s:
        if out is None:
            out = torch.empty((tokens, rows), dtype=out_dtype, device=w.device)
        elif out.shape != (tokens, rows) or (rows > 1 and out.stride(1) != 1) or (tokens > 1 and out.stride(0) < rows):
            raise ValueError("out must be a [tokens, rows] tensor with adjacent columns")
        if out.dtype not in (torch.float32, torch.bfloat16, torch.float16):
            raise ValueError("out must be fp32, bf16 or fp16")
        _check(_lib.entro_matmul_i8(q.data_ptr(), ldq, x.scale.data_ptr(), x.sum.data_ptr(), tokens, w.data_ptr(), _TYPES[w.dtype],
                                    ldw, rows, cols, w_scale.data_ptr() if ws else None, 0.0 if ws else float(w_scale),
                                    w_zero.data_ptr() if wz else None, 0 if wz or w_zero is None else int(w_zero),
                                    out.data_ptr(), _TYPES[out.dtype], out.stride(0) if tokens > 1 else rows,
                                    _dptr(status), s), "entro_matmul_i8")
    return out


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, heads: int, dim: int) -> torch.Tensor:
    """A [tokens, heads, dim] tensor that the kernels can read in 16-byte pieces."""
    if t.dtype != dtype or t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must be a {dtype} [tokens, {heads}, {dim}] tensor")
    s = t.stride()
    if s[2] != 1 or (t.shape[0] > 1 and s[0] % 8) or (heads > 1 and s[1] % 8) or t.data_ptr() % 16:
        raise ValueError(f"{name} must have adjacent channels, strides that are multiples of 8 and begin on 16 bytes")
    return t


def _strides(t: torch.Tensor):
    """Token and head stride; those of a single token or head say nothing."""
    s = t.stride()
    return (s[0] if t.shape[0] > 1 else 0), (s[1] if t.shape[1] > 1 else 0)


def _index(t: torch.Tensor, name: str, shape: tuple):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor")


def attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     cu_keys: Optional[torch.Tensor] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Causal attention over packed prompts: q [tokens, heads, head_dim], k and v [keys, kv_heads, head_dim], bf16 or
    fp16 (slices of one projection's output as they are).  cu_seqlens int32 [batch + 1] says where each sequence's queries
    begin, cu_keys its keys (None: as the queries); a sequence's last query sees its last key, so queries that continue a
    context give their keys with it.  scale: 1 / sqrt(head_dim) by default.  Rows of no sequence are left as they are (give
    `out` to keep theirs)."""
    if q.dtype not in (torch.bfloat16, torch.float16) or q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be bf16 or fp16 [tokens, heads, head_dim] tensors")
    tokens, heads, dim = q.shape
    keys, kv = k.shape[:2]
    if dim not in (64, 96, 128):
        raise ValueError("head_dim must be 64, 96 or 128")
    if kv < 1 or heads < 1 or heads % kv:
        raise ValueError("q's heads must be a multiple of k's")
    _rows(q, "q", q.dtype, heads, dim)
    _rows(k, "k", q.dtype, kv, dim)
    _rows(v, "v", q.dtype, kv, dim)
    if v.shape[0] != keys:
        raise ValueError("k and v must have the same number of tokens")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if (t.shape[0] > 1 and t.stride(0) == 0) or (t.shape[1] > 1 and t.stride(1) == 0):
            raise ValueError(f"{name} must not be expanded")
    batch = cu_seqlens.shape[0] - 1 if cu_seqlens.dim() == 1 else -1
    if batch < 0:
        raise ValueError("cu_seqlens must be an int32 [batch + 1] tensor")
    _index(cu_seqlens, "cu_seqlens", (batch + 1,))
    if cu_keys is not None:
        _index(cu_keys, "cu_keys", (batch + 1,))
    elif keys != tokens:
        raise ValueError("without cu_keys, k and v must have q's tokens")
    if out is not None:
        _rows(out, "out", q.dtype, heads, dim)
        if out.shape[0] != tokens:
            raise ValueError("out must have q's shape")
    scale = dim ** -0.5 if scale is None else float(scale)
    if not 0.0 < scale < 3e38:
        raise ValueError("scale must be above 0 and finite")
    _inputs(q.device, q=q, k=k, v=v, cu_seqlens=cu_seqlens, cu_keys=cu_keys, out=out, status=status)
    with _on(q.device, stream) as s:
        out = torch.empty((tokens, heads, dim), dtype=q.dtype, device=q.device) if out is None else out
        _check(_lib.entro_attention_prompt(_TYPES[q.dtype], dim, q.data_ptr(), *_strides(q), heads, tokens, k.data_ptr(), *_strides(k),
                                           v.data_ptr(), *_strides(v), kv, keys, cu_seqlens.data_ptr(),
                                           cu_keys.data_ptr() if cu_keys is not None else None, batch, scale, out.data_ptr(),
                                           *_strides(out), _dptr(status), s), "entro_attention_prompt")
    return out


class KVCache:
    """Keys and values of one layer in 8 bits, in pages with a scale for each page and head (`entro_kv_cache`).

    Made from the caller's buffers -- codes int8 [pages, kv_heads, page_tokens, head_dim], scales fp32 [pages, kv_heads],
    tails bf16 or fp16 [slots, kv_heads, page_tokens, head_dim] -- or by `KVCache.empty`.  `page_table` int32
    [batch, width] names the pages of each sequence's blocks in order, `lens` int32 [batch] its tokens, `slots` int32
    [batch] its tail slot (None: its place in the batch).  These are read on the GPU: an index out of range is reported in
    `status` (E_INVAL) and skipped."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 k_tail: torch.Tensor, v_tail: torch.Tensor):
        if k_codes.dim() != 4 or k_tail.dim() != 4:
            raise ValueError("codes must be [pages, kv_heads, page_tokens, head_dim], tails [slots, kv_heads, page_tokens, head_dim]")
        pages, kv, page, dim = k_codes.shape
        slots, dtype = k_tail.shape[0], k_tail.dtype
        if page not in (16, 32, 64, 128) or dim not in (64, 96, 128):
            raise ValueError("page_tokens must be 16, 32, 64 or 128 and head_dim 64, 96 or 128")
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("tails must be bf16 or fp16")
        if pages < 1 or slots < 1 or not 1 <= kv <= 65535:
            raise ValueError("a cache has a page, a slot and a key head at least")
        for t, name, want, shape in ((k_codes, "k_codes", torch.int8, (pages, kv, page, dim)), (v_codes, "v_codes", torch.int8, (pages, kv, page, dim)),
                                     (k_scale, "k_scale", torch.float32, (pages, kv)), (v_scale, "v_scale", torch.float32, (pages, kv)),
                                     (k_tail, "k_tail", dtype, (slots, kv, page, dim)), (v_tail, "v_tail", dtype, (slots, kv, page, dim))):
            if t.dtype != want or t.shape != shape or not t.is_contiguous() or t.data_ptr() % 16:
                raise ValueError(f"{name} must be a contiguous {want} {list(shape)} tensor that begins on 16 bytes")
        self.device = k_codes.device
        _inputs(self.device, k_codes=k_codes, v_codes=v_codes, k_scale=k_scale, v_scale=v_scale, k_tail=k_tail, v_tail=v_tail)
        self.k_codes, self.v_codes, self.k_scale, self.v_scale, self.k_tail, self.v_tail = k_codes, v_codes, k_scale, v_scale, k_tail, v_tail
        self.pages, self.kv_heads, self.page_tokens, self.head_dim, self.slots, self.dtype = pages, kv, page, dim, slots, dtype
        self._c = _KVCache(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k_tail.data_ptr(),
                           v_tail.data_ptr(), pages, slots, kv, page, dim, _TYPES[dtype])
        self._ref = ctypes.byref(self._c)
        self._work_bytes = None

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, slots: int = 1,
              dtype: torch.dtype = torch.bfloat16, device=None) -> "KVCache":
        device = torch.device("cuda" if device is None else device)
        codes = [torch.empty((pages, kv_heads, page_tokens, head_dim), dtype=torch.int8, device=device) for _ in range(2)]
        scales = [torch.empty((pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
        tails = [torch.empty((slots, kv_heads, page_tokens, head_dim), dtype=dtype, device=device) for _ in range(2)]
        return cls(*codes, *scales, *tails)

    def _tables(self, page_table: torch.Tensor, slots: Optional[torch.Tensor]) -> int:
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be an int32 [batch, width] tensor with adjacent columns")
        batch = page_table.shape[0]
        if slots is not None:
            _index(slots, "slots", (batch,))
        elif batch > self.slots:
            raise ValueError("more sequences than tail slots")
        return batch

    def append(self, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
               slots: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> None:
        """Packed new tokens k, v [tokens, kv_heads, head_dim] to their sequences; cu_seqlens int32 [batch + 1] says where
        each sequence's begin, lens counts them already.  No page or slot may be written for two sequences."""
        _rows(k, "k", self.dtype, self.kv_heads, self.head_dim)
        _rows(v, "v", self.dtype, self.kv_heads, self.head_dim)
        if k.shape[0] != v.shape[0]:
            raise ValueError("k and v must have the same number of tokens")
        batch = self._tables(page_table, slots)
        _index(cu_seqlens, "cu_seqlens", (batch + 1,))
        _index(lens, "lens", (batch,))
        _inputs(self.device, k=k, v=v, cu_seqlens=cu_seqlens, page_table=page_table, lens=lens, slots=slots, status=status)
        with _on(self.device, stream) as s:
            _check(_lib.entro_kv_append(self._ref, k.data_ptr(), *_strides(k), v.data_ptr(), *_strides(v), k.shape[0],
                                        cu_seqlens.data_ptr(), page_table.data_ptr(), page_table.stride(0) if batch > 1 else page_table.shape[1],
                                        page_table.shape[1], lens.data_ptr(), slots.data_ptr() if slots is not None else None, batch,
                                        _dptr(status), s), "entro_kv_append")

    def read(self, page_table: torch.Tensor, cu_seqlens: torch.Tensor, tokens: int, slots: Optional[torch.Tensor] = None,
             out: Optional[tuple] = None, status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        """(k, v) [tokens, kv_heads, head_dim]: all tokens of the sequences, packed; sequence b holds
        cu_seqlens[b + 1] - cu_seqlens[b] of them."""
        batch = self._tables(page_table, slots)
        _index(cu_seqlens, "cu_seqlens", (batch + 1,))
        if out is not None:
            for t, name in zip(out, ("k", "v")):
                _rows(t, name, self.dtype, self.kv_heads, self.head_dim)
                if t.shape[0] != tokens:
                    raise ValueError(f"{name} must have {tokens} tokens")
        _inputs(self.device, cu_seqlens=cu_seqlens, page_table=page_table, slots=slots, status=status,
                k=out[0] if out is not None else None, v=out[1] if out is not None else None)
        with _on(self.device, stream) as s:
            k, v = out if out is not None else (torch.empty((tokens, self.kv_heads, self.head_dim), dtype=self.dtype, device=self.device)
                                                for _ in range(2))
            _check(_lib.entro_kv_read(self._ref, k.data_ptr(), *_strides(k), v.data_ptr(), *_strides(v), tokens, cu_seqlens.data_ptr(),
                                      page_table.data_ptr(), page_table.stride(0) if batch > 1 else page_table.shape[1], page_table.shape[1],
                                      slots.data_ptr() if slots is not None else None, batch, _dptr(status), s), "entro_kv_read")
        return k, v

    def attend(self, q: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, slots: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Attention of one token of each sequence, q [batch, heads, head_dim] (heads a multiple of kv_heads), over its
        cached tokens; scale: 1 / sqrt(head_dim) by default.  A sequence without tokens gets zeros."""
        heads = q.shape[1] if q.dim() == 3 else 0
        _rows(q, "q", self.dtype, heads, self.head_dim)
        if heads < 1 or heads % self.kv_heads:
            raise ValueError("q's heads must be a multiple of the cache's")
        batch = self._tables(page_table, slots)
        if q.shape[0] != batch:
            raise ValueError("q must have a token for each sequence")
        _index(lens, "lens", (batch,))
        if out is not None:
            _rows(out, "out", self.dtype, heads, self.head_dim)
            if out.shape[0] != batch:
                raise ValueError("out must have q's shape")
        scale = self.head_dim ** -0.5 if scale is None else float(scale)
        if not 0.0 < scale < 3e38:
            raise ValueError("scale must be above 0 and finite")
        _inputs(self.device, q=q, page_table=page_table, lens=lens, slots=slots, out=out, status=status)
        with _on(self.device, stream) as s:
            if self._work_bytes is None:
                n = ctypes.c_uint64()
                _check(_lib.entro_kv_attend_workspace(self._ref, ctypes.byref(n)), "entro_kv_attend_workspace")
                self._work_bytes = n.value
            # a workspace of the call's own, from the pool of the stream it runs on: calls never share one
            work = torch.empty(self._work_bytes, dtype=torch.uint8, device=self.device)
            out = torch.empty((batch, heads, self.head_dim), dtype=self.dtype, device=self.device) if out is None else out
            _check(_lib.entro_kv_attend(self._ref, q.data_ptr(), *_strides(q), heads, page_table.data_ptr(),
                                        page_table.stride(0) if batch > 1 else page_table.shape[1], page_table.shape[1], lens.data_ptr(),
                                        slots.data_ptr() if slots is not None else None, batch, scale, out.data_ptr(), *_strides(out),
                                        work.data_ptr(), self._work_bytes, _dptr(status), s), "entro_kv_attend")
        return out


def test_stall_tables(extra_bytes: int) -> int:
    """Test hook for the bounded waits: later launches wait for `extra_bytes` of table copy that
    never arrive, so each gives up after about a second with E_TIMEOUT in the status word.
    0 turns it off.  Returns the previous value."""
    return int(_lib.entro_test_stall_tables(int(extra_bytes)))


def version() -> int:
    return int(_lib.entro_version())


def set_overlap(enable: bool) -> bool:
    """Launch overlap (programmatic dependent launch) for every later decode call in this
    process: a decode may start while the kernel before it on the stream finishes, reading
    only the tensor's device image until that kernel has completed.  Enable only if no
    kernel launched right before a decode call writes that tensor's device image.
    Returns the previous setting."""
    return bool(_lib.entro_set_overlap(1 if enable else 0))


__all__ = ["Blob", "DeviceTensor", "Group", "EntroError", "encode", "upload", "lib", "version", "set_overlap", "EXPORTS",
           "decode_gemv_group_static", "STATIC_GROUP_MAX", "QuantTokens", "quantize_tokens", "matmul_i8", "attention_prompt", "KVCache",
           "test_stall_tables", "QUANT_AUTO", "QUANT_UNSIGNED", "QUANT_ASYM", "FORMAT_SINGLE", "FORMAT_LANES", "FORMAT_ROWS_CO",
           "FORMAT_ROWS", "GROUP_GEMV",
           "GROUP_BF16", "SCHEME_UNSIGNED", "SCHEME_ASYM"]
