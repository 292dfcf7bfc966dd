"""Python binding of libentro (argument marshalling only).

Every step of the path -- quantization and Huffman coding on the host, decoding,
dequantization and the fused GEMV on the GPU -- runs inside ``libentro.so``;
this module turns numpy / torch objects into pointers and sizes for the C ABI
declared in ``include/entro.h`` and turns return codes into exceptions (the
operators' usual calls do so in ``csrc/binding.cpp``).  PyTorch is used for device memory and streams only.  There is no fallback:
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
import operator
import os
from typing import List, NamedTuple, Optional, Sequence, Union

import numpy as np
import torch
from torch.autograd.forward_ad import unpack_dual

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libentro.so")
BINDING_PATH = os.path.join(_HERE, "_binding.so")

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


class _ProductPlan(ctypes.Structure):
    _fields_ = [("wide", ctypes.c_int32), ("tile_tokens", ctypes.c_int32), ("split", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("row_tiles", ctypes.c_int64), ("token_tiles", ctypes.c_int64)]


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
           "entro_decode_gemv_group_static", "entro_set_overlap", "entro_test_stall_tables", "entro_test_product_plan",
           "entro_quantize_tokens", "entro_unpack_codes", "entro_matmul_i8",
           "entro_kv_append", "entro_kv_read", "entro_kv_attend_workspace", "entro_kv_attend", "entro_attention_prompt"]


def _built(path: str):
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python huffman_decode_canonical_b200/build.py` "
                          "(there is no CPU fallback)")


def _load() -> ctypes.CDLL:
    _built(LIB_PATH)
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
        "entro_test_product_plan": ([I64, I64, I64, I32, P], I32),
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


class _NoFast:
    """In place of the binding's module where torch knows no CUDA: the host side needs none."""

    def __getattr__(self, name):
        return lambda *a: None


def _load_binding():
    """The usual calls of the operators around the coded weights, checked and made without the interpreter's part: each
    returns None for anything that is not the plain valid case, and the function here goes on."""
    if torch.version.cuda is None:
        return _NoFast()
    _built(BINDING_PATH)
    from . import _binding
    _binding.init(*(ctypes.cast(getattr(_lib, f), ctypes.c_void_p).value for f in (
        "entro_quantize_tokens", "entro_matmul_i8", "entro_attention_prompt", "entro_kv_append", "entro_kv_read", "entro_kv_attend")))
    return _binding


_lib = _load()
_fast = _load_binding()


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
        if stream is not None or self.device.index != _current_device():
            with _on(self.device, stream):
                return self.matmul(x, out, out_dtype, status)
        s = _current_stream(self.device.index)
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
        xq = x if isinstance(x, QuantTokens) else quantize_tokens(x)
        return matmul_i8(xq, w, self.info["scale"], self.info["zero"], out=out, out_dtype=out_dtype, status=status)

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


# The current device and its current stream's handle, without the objects that the public calls make of them.
_current_device = getattr(torch._C, "_cuda_getDevice", None)  # (a build of torch without CUDA has neither, and no tensors for them)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _on:
    """The tensors' device as the current one, and `stream` as its current stream: new buffers then come from the pool of
    the stream that is launched on."""

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        if stream is not None and stream.device != device:
            raise ValueError("the stream belongs to another device than the tensors")
        self.guard = torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.guard.__enter__()

    def __exit__(self, *e):
        self.guard.__exit__(*e)


def _check_inputs(index: int, tensors, names):
    """Refuses what the kernels must not be given: tensors of other devices, or ones that ask for gradients (backward or
    forward: a tangent would be lost); a status that is no int32 word (the last one named so); any call of a trace."""
    if index < 0:
        raise ValueError("expected CUDA tensors")
    if torch.jit.is_tracing():
        raise ValueError("this call cannot be traced: its result would be a constant of the trace")
    if names[-1] == "status" and tensors[-1] is not None and (tensors[-1].dtype is not torch.int32 or tensors[-1].numel() < 1):
        raise ValueError("status must be an int32 tensor")
    grad = torch.is_grad_enabled()
    for t in tensors:
        if t is not None and (t.get_device() != index or (grad and t.requires_grad)):
            name = names[[u is t for u in tensors].index(True)]
            if t.get_device() != index:
                raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
            raise ValueError(f"{name} requires a gradient: this call has none (use torch.no_grad())")
        if t is not None and t.is_floating_point() and unpack_dual(t).tangent is not None:
            raise ValueError(f"{names[[u is t for u in tensors].index(True)]} is a dual tensor: this call has no forward-mode gradient")


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
    if stream is None:
        done = _fast.quantize_tokens(x)
        if done is not None:
            return QuantTokens._make(done)
    if x.dtype not in (torch.bfloat16, torch.float16) or x.dim() != 2 or x.shape[1] < 1 or x.stride(1) != 1:
        raise ValueError("x must be a bf16 or fp16 [tokens, cols] tensor with adjacent columns")
    index = x.get_device()
    _check_inputs(index, (x,), ("x",))
    if stream is not None or index != _current_device():
        with _on(x.device, stream):
            return quantize_tokens(x)
    tokens, cols = x.shape
    pitch, device = (cols + 15) // 16 * 16, x.device
    codes = torch.empty((tokens, pitch), dtype=torch.int8, device=device)
    scale = torch.empty(tokens, dtype=torch.float32, device=device)
    total = torch.empty(tokens, dtype=torch.int32, device=device)
    _check(_lib.entro_quantize_tokens(x.data_ptr(), _TYPES[x.dtype], tokens, cols, x.stride(0) if tokens > 1 else pitch,
                                      codes.data_ptr(), pitch, scale.data_ptr(), total.data_ptr(), _current_stream(index)),
           "entro_quantize_tokens")
    return QuantTokens(codes if pitch == cols else codes[:, :cols], scale, total)


def matmul_i8(x: QuantTokens, w: torch.Tensor, w_scale: Union[float, torch.Tensor], w_zero: Union[None, int, torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
              status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y[t, n] = x.scale[t] * w_scale[n] * sum_k x.codes[t, k] * (w[n, k] - w_zero[n]).

    w uint8 or int8 [rows, cols], adjacent columns, rows a multiple of 16 bytes apart; w_scale a number or fp32 [rows];
    w_zero a whole number, int32 [rows] or None (0).  out: fp32, bf16 or fp16 [tokens, rows] with adjacent columns."""
    q, scale, total = x
    if stream is None and out is None:
        done = _fast.matmul_i8(q, scale, total, w, w_scale, w_zero, _TYPES.get(out_dtype), status)
        if done is not None:
            return done
    if w.dtype not in (torch.uint8, torch.int8) or w.dim() != 2 or w.shape[1] < 1 or w.stride(1) != 1:
        raise ValueError("w must be a uint8 or int8 [rows, cols] tensor with adjacent columns")
    rows, cols = w.shape
    if q.dtype is not torch.int8 or q.dim() != 2 or q.shape[1] != cols or q.stride(1) != 1:
        raise ValueError("x.codes must be an int8 [tokens, cols] tensor with adjacent columns")
    tokens = q.shape[0]
    _vector(scale, "x.scale", torch.float32, tokens, "[tokens]")
    _vector(total, "x.sum", torch.int32, tokens, "[tokens]")
    ws, wz = isinstance(w_scale, torch.Tensor), isinstance(w_zero, torch.Tensor)
    if ws:
        _vector(w_scale, "w_scale", torch.float32, rows, "[rows]")
    if wz:
        _vector(w_zero, "w_zero", torch.int32, rows, "[rows]")
    elif w_zero is None:
        w_zero = 0
    else:
        try:
            w_zero = operator.index(w_zero)
        except TypeError:
            raise ValueError("w_zero must be a whole number, an int32 [rows] tensor or None") from None
        if not -2 ** 31 <= w_zero < 2 ** 31:
            raise ValueError("w_zero must fit 32 bits")
    index = w.get_device()
    _check_inputs(index, (w, q, scale, total, w_scale if ws else None, w_zero if wz else None, out, status),
                  ("w", "x.codes", "x.scale", "x.sum", "w_scale", "w_zero", "out", "status"))
    # a single row's stride says nothing
    ldq, ldw = (q.stride(0) if tokens > 1 else _pitch(cols)), (w.stride(0) if rows > 1 else _pitch(cols))
    qp, wp = q.data_ptr(), w.data_ptr()
    if (ldq | ldw | qp | wp) & 15:
        raise ValueError("x.codes and w must begin on 16 bytes, their rows a multiple of 16 bytes apart")
    if stream is not None or index != _current_device():
        with _on(w.device, stream):
            return matmul_i8(x, w, w_scale, w_zero, out, out_dtype, status)
    if out is None:
        out = torch.empty((tokens, rows), dtype=out_dtype, device=w.device)
        ldy = rows
    else:
        if out.shape != (tokens, rows) or (rows > 1 and out.stride(1) != 1) or (tokens > 1 and out.stride(0) < rows):
            raise ValueError("out must be a [tokens, rows] tensor with adjacent columns")
        ldy = out.stride(0) if tokens > 1 else rows
    if out.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise ValueError("out must be fp32, bf16 or fp16")
    _check(_lib.entro_matmul_i8(qp, ldq, scale.data_ptr(), total.data_ptr(), tokens, wp, _TYPES[w.dtype], ldw, rows, cols,
                                w_scale.data_ptr() if ws else None, 0.0 if ws else float(w_scale), w_zero.data_ptr() if wz else None,
                                0 if wz else w_zero, out.data_ptr(), _TYPES[out.dtype], ldy,
                                None if status is None else status.data_ptr(), _current_stream(index)), "entro_matmul_i8")
    return out


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, what: str):
    if t.dtype is not dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {what} tensor")


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, heads: int, dim: int, written: bool = False):
    """Token and head stride of a [tokens, heads, dim] tensor that the kernels can read in 16-byte pieces (those of a
    single token or head say nothing and count as 0); `written`: one whose rows share no elements."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be a {dtype} [tokens, {heads}, {dim}] tensor")
    token, head, channel = t.stride()
    if shape[0] <= 1:
        token = 0
    if heads <= 1:
        head = 0
    if channel != 1 or (token | head) & 7 or t.data_ptr() & 15:
        raise ValueError(f"{name} must have adjacent channels, strides that are multiples of 8 and begin on 16 bytes")
    if written and shape[0] and not any((n <= 1 or s >= dim) and (m <= 1 or r >= (s * (n - 1) if n > 1 else 0) + dim)
                                        for n, s, m, r in ((heads, head, shape[0], token), (shape[0], token, heads, head))):
        raise ValueError(f"{name} must not have rows that share elements")
    return token, head


def attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     cu_keys: Optional[torch.Tensor] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Causal attention over packed prompts: q [tokens, heads, head_dim], k and v [keys, kv_heads, head_dim], bf16 or
    fp16 (slices of one projection's output as they are).  cu_seqlens int32 [batch + 1] says where each sequence's queries
    begin, cu_keys its keys (None: as the queries); a sequence's last query sees its last key, so queries that continue a
    context give their keys with it.  scale: 1 / sqrt(head_dim) by default.  Rows of no sequence are left as they are (give
    `out`, a tensor of its own, to keep theirs)."""
    if stream is None and out is None:
        done = _fast.attention_prompt(q, k, v, cu_seqlens, cu_keys, scale, status)
        if done is not None:
            return done
    if q.dtype not in (torch.bfloat16, torch.float16) or q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be bf16 or fp16 [tokens, heads, head_dim] tensors")
    tokens, heads, dim = q.shape
    keys, kv = k.shape[:2]
    if dim not in (64, 96, 128):
        raise ValueError("head_dim must be 64, 96 or 128")
    if kv < 1 or heads < 1 or heads % kv:
        raise ValueError("q's heads must be a multiple of k's")
    dtype = q.dtype
    qs, ks, vs = _rows(q, "q", dtype, heads, dim), _rows(k, "k", dtype, kv, dim), _rows(v, "v", dtype, kv, dim)
    if v.shape[0] != keys:
        raise ValueError("k and v must have the same number of tokens")
    if (tokens > 1 and qs[0] == 0) or (heads > 1 and qs[1] == 0) or (keys > 1 and 0 in (ks[0], vs[0])) or (kv > 1 and 0 in (ks[1], vs[1])):
        raise ValueError("q, k and v must not be expanded")
    batch = cu_seqlens.shape[0] - 1 if cu_seqlens.dim() == 1 else -1
    if batch < 0:
        raise ValueError("cu_seqlens must be an int32 [batch + 1] tensor")
    _vector(cu_seqlens, "cu_seqlens", torch.int32, batch + 1, "[batch + 1]")
    if cu_keys is not None:
        _vector(cu_keys, "cu_keys", torch.int32, batch + 1, "[batch + 1]")
    elif keys != tokens:
        raise ValueError("without cu_keys, k and v must have q's tokens")
    if out is not None:
        os_ = _rows(out, "out", dtype, heads, dim, written=True)
        if out.shape[0] != tokens:
            raise ValueError("out must have q's shape")
        if tokens and out.data_ptr() in (q.data_ptr(), k.data_ptr(), v.data_ptr()):
            raise ValueError("out must not be q, k or v: they are read while it is written")
    scale = dim ** -0.5 if scale is None else float(scale)
    if not 0.0 < scale <= 2e38:
        raise ValueError("scale must be above 0 and finite")
    index = q.get_device()
    _check_inputs(index, (q, k, v, cu_seqlens, cu_keys, out, status), ("q", "k", "v", "cu_seqlens", "cu_keys", "out", "status"))
    if stream is not None or index != _current_device():
        with _on(q.device, stream):
            return attention_prompt(q, k, v, cu_seqlens, cu_keys, scale, out, status)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=dtype, device=q.device)
        os_ = (heads * dim, dim)
    _check(_lib.entro_attention_prompt(_TYPES[dtype], dim, q.data_ptr(), *qs, heads, tokens, k.data_ptr(), *ks, v.data_ptr(), *vs, kv,
                                       keys, cu_seqlens.data_ptr(), None if cu_keys is None else cu_keys.data_ptr(), batch, scale,
                                       out.data_ptr(), *os_, None if status is None else status.data_ptr(), _current_stream(index)),
           "entro_attention_prompt")
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
        self._index = k_codes.get_device()
        _check_inputs(self._index, (k_codes, v_codes, k_scale, v_scale, k_tail, v_tail),
                      ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail"))
        self._buffers = k_codes, v_codes, k_scale, v_scale, k_tail, v_tail
        self.pages, self.kv_heads, self.page_tokens, self.head_dim, self.slots, self.dtype = pages, kv, page, dim, slots, dtype
        self._c = _KVCache(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k_tail.data_ptr(),
                           v_tail.data_ptr(), pages, slots, kv, page, dim, _TYPES[dtype])
        self._ref = ctypes.byref(self._c)
        self._address = ctypes.addressof(self._c)
        self._work_bytes = None

    # The buffers are the cache's for good: the library holds their addresses.
    k_codes, v_codes, k_scale, v_scale, k_tail, v_tail = (property(lambda self, i=i: self._buffers[i]) for i in range(6))

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, slots: int = 1,
              dtype: torch.dtype = torch.bfloat16, device=None) -> "KVCache":
        device = torch.device("cuda" if device is None else device)
        codes = [torch.empty((pages, kv_heads, page_tokens, head_dim), dtype=torch.int8, device=device) for _ in range(2)]
        scales = [torch.empty((pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
        tails = [torch.empty((slots, kv_heads, page_tokens, head_dim), dtype=dtype, device=device) for _ in range(2)]
        return cls(*codes, *scales, *tails)

    def _tables(self, page_table: torch.Tensor, slots: Optional[torch.Tensor]):
        """(batch, width, row stride) of a page table"""
        if page_table.dtype is not torch.int32 or page_table.dim() != 2:
            raise ValueError("page_table must be an int32 [batch, width] tensor")
        batch, width = page_table.shape
        stride, one = page_table.stride()
        if batch <= 1:
            stride = width
        if (width > 1 and one != 1) or stride < width:
            raise ValueError("page_table must have adjacent columns")
        if slots is not None:
            _vector(slots, "slots", torch.int32, batch, "[batch]")
        elif batch > self.slots:
            raise ValueError("more sequences than tail slots")
        return batch, width, stride

    def append(self, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
               slots: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> None:
        """Packed new tokens k, v [tokens, kv_heads, head_dim] to their sequences; cu_seqlens int32 [batch + 1] says where
        each sequence's begin, lens counts them already.  No page or slot may be written for two sequences."""
        if stream is None and _fast.kv_append(self._address, self._index, k, v, cu_seqlens, page_table, lens, slots, status):
            return
        ks, vs = _rows(k, "k", self.dtype, self.kv_heads, self.head_dim), _rows(v, "v", self.dtype, self.kv_heads, self.head_dim)
        tokens = k.shape[0]
        if tokens != v.shape[0]:
            raise ValueError("k and v must have the same number of tokens")
        batch, width, stride = self._tables(page_table, slots)
        _vector(cu_seqlens, "cu_seqlens", torch.int32, batch + 1, "[batch + 1]")
        _vector(lens, "lens", torch.int32, batch, "[batch]")
        index = self._index
        _check_inputs(index, (k, v, cu_seqlens, page_table, lens, slots, status),
                      ("k", "v", "cu_seqlens", "page_table", "lens", "slots", "status"))
        if stream is not None or index != _current_device():
            with _on(self.device, stream):
                return self.append(k, v, cu_seqlens, page_table, lens, slots, status)
        _check(_lib.entro_kv_append(self._ref, k.data_ptr(), *ks, v.data_ptr(), *vs, tokens, cu_seqlens.data_ptr(), page_table.data_ptr(),
                                    stride, width, lens.data_ptr(), None if slots is None else slots.data_ptr(), batch,
                                    None if status is None else status.data_ptr(), _current_stream(index)), "entro_kv_append")

    def read(self, page_table: torch.Tensor, cu_seqlens: torch.Tensor, tokens: int, slots: Optional[torch.Tensor] = None,
             out: Optional[tuple] = None, status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        """(k, v) [tokens, kv_heads, head_dim]: all tokens of the sequences, packed; sequence b holds
        cu_seqlens[b + 1] - cu_seqlens[b] of them."""
        if stream is None and out is None:
            done = _fast.kv_read(self._address, self._index, page_table, cu_seqlens, tokens, slots, status)
            if done is not None:
                return done
        batch, width, stride = self._tables(page_table, slots)
        _vector(cu_seqlens, "cu_seqlens", torch.int32, batch + 1, "[batch + 1]")
        heads, dim = self.kv_heads, self.head_dim
        k, v = (None, None) if out is None else out
        if out is not None:
            ks, vs = _rows(k, "k", self.dtype, heads, dim, written=True), _rows(v, "v", self.dtype, heads, dim, written=True)
            if k.shape[0] != tokens or v.shape[0] != tokens:
                raise ValueError(f"out must have {tokens} tokens")
            if tokens and k.data_ptr() == v.data_ptr():
                raise ValueError("out's keys and values must be two tensors")
        index = self._index
        _check_inputs(index, (cu_seqlens, page_table, slots, k, v, status), ("cu_seqlens", "page_table", "slots", "k", "v", "status"))
        if stream is not None or index != _current_device():
            with _on(self.device, stream):
                return self.read(page_table, cu_seqlens, tokens, slots, out, status)
        if out is None:
            k = torch.empty((tokens, heads, dim), dtype=self.dtype, device=self.device)
            v = torch.empty((tokens, heads, dim), dtype=self.dtype, device=self.device)
            ks = vs = (heads * dim, dim)
        _check(_lib.entro_kv_read(self._ref, k.data_ptr(), *ks, v.data_ptr(), *vs, tokens, cu_seqlens.data_ptr(), page_table.data_ptr(),
                                  stride, width, None if slots is None else slots.data_ptr(), batch,
                                  None if status is None else status.data_ptr(), _current_stream(index)), "entro_kv_read")
        return k, v

    def attend(self, q: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, slots: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Attention of one token of each sequence, q [batch, heads, head_dim] (heads a multiple of kv_heads), over its
        cached tokens; scale: 1 / sqrt(head_dim) by default.  A sequence without tokens gets zeros."""
        if stream is None and out is None and self._work_bytes is not None:
            done = _fast.kv_attend(self._address, self._index, self._work_bytes, q, page_table, lens, slots, scale, status)
            if done is not None:
                return done
        heads, dim = q.shape[1] if q.dim() == 3 else 0, self.head_dim
        qs = _rows(q, "q", self.dtype, heads, dim)
        if heads < 1 or heads % self.kv_heads:
            raise ValueError("q's heads must be a multiple of the cache's")
        batch, width, stride = self._tables(page_table, slots)
        if q.shape[0] != batch:
            raise ValueError("q must have a token for each sequence")
        _vector(lens, "lens", torch.int32, batch, "[batch]")
        if out is not None:
            os_ = _rows(out, "out", self.dtype, heads, dim, written=True)
            if out.shape[0] != batch:
                raise ValueError("out must have q's shape")
        scale = dim ** -0.5 if scale is None else float(scale)
        if not 0.0 < scale <= 2e38:
            raise ValueError("scale must be above 0 and finite")
        index = self._index
        _check_inputs(index, (q, page_table, lens, slots, out, status), ("q", "page_table", "lens", "slots", "out", "status"))
        if stream is not None or index != _current_device():
            with _on(self.device, stream):
                return self.attend(q, page_table, lens, slots, scale, out, status)
        if self._work_bytes is None:
            n = ctypes.c_uint64()
            _check(_lib.entro_kv_attend_workspace(self._ref, ctypes.byref(n)), "entro_kv_attend_workspace")
            self._work_bytes = n.value
        # a workspace of the call's own, from the pool of the stream it runs on: calls never share one
        work = torch.empty(self._work_bytes, dtype=torch.uint8, device=self.device)
        if out is None:
            out = torch.empty((batch, heads, dim), dtype=self.dtype, device=self.device)
            os_ = (heads * dim, dim)
        _check(_lib.entro_kv_attend(self._ref, q.data_ptr(), *qs, heads, page_table.data_ptr(), stride, width, lens.data_ptr(),
                                    None if slots is None else slots.data_ptr(), batch, scale, out.data_ptr(), *os_, work.data_ptr(),
                                    self._work_bytes, None if status is None else status.data_ptr(), _current_stream(index)),
               "entro_kv_attend")
        return out


def test_stall_tables(extra_bytes: int) -> int:
    """Test hook for the bounded waits: later launches wait for `extra_bytes` of table copy that
    never arrive, so each gives up after about a second with E_TIMEOUT in the status word.
    0 turns it off.  Returns the previous value."""
    return int(_lib.entro_test_stall_tables(int(extra_bytes)))


def test_product_plan(tokens: int, rows: int, cols: int, sms: int = 148) -> dict:
    """Test hook: how `matmul_i8` takes a call of these sizes on a device of `sms` SMs (`entro_test_product_plan`)."""
    plan = _ProductPlan()
    _check(_lib.entro_test_product_plan(tokens, rows, cols, sms, ctypes.byref(plan)), "entro_test_product_plan")
    return {f: getattr(plan, f) for f, _ in _ProductPlan._fields_}


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
           "test_stall_tables", "test_product_plan", "QUANT_AUTO", "QUANT_UNSIGNED", "QUANT_ASYM", "FORMAT_SINGLE", "FORMAT_LANES", "FORMAT_ROWS_CO",
           "FORMAT_ROWS", "GROUP_GEMV",
           "GROUP_BF16", "SCHEME_UNSIGNED", "SCHEME_ASYM"]
