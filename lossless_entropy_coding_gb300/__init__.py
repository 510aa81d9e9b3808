"""Python binding of libecc_gb300: lossless fixed-codebook coding of e4m3
byte tensors on GB300 (Quad Length Codes and single-stage canonical Huffman),
and the language-model operators next to the coders (layer norm, the matrix
product with a fused epilogue, token log probabilities, and their gradients).

Argument marshalling only.  Every entry point has the name of the C function
it calls (see include/ecc.h and include/ecc_lm.h for the contract); PyTorch supplies device memory
and the current CUDA stream.  All coding work runs in the library's CUDA
kernels or its host codebook builders -- there is no other code path: if the
shared library has not been built, importing the binding still works but
every call raises.
"""
from __future__ import annotations

import ctypes as ct
import functools
import os
import struct
import threading
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libecc_gb300.so")

OK, ERR_ARG, ERR_CAPACITY, ERR_CORRUPT, ERR_CODEBOOK, ERR_TIMEOUT, ERR_CUDA, ERR_CHECK = range(8)
FAMILY_QLC, FAMILY_HUFFMAN, FAMILY_ESCAPE = 1, 2, 3
MAX_CODE_LEN = 48
BASE_WIDTHS = (3, 3, 3, 3, 3, 4, 5, 8)

# Layout of ecc_codebook (C struct in include/ecc.h), naturally aligned.
CODEBOOK_DTYPE = np.dtype([
    ("magic", "<u4"), ("family", "<u4"), ("max_len", "<u4"), ("min_len", "<u4"),
    ("n_coded", "<u4"), ("prefix_bits", "<u4"), ("reserved", "<u4", (2,)),
    ("code", "<u8", (256,)), ("first", "<u8", (64,)),
    ("enc_code", "<u4", (256,)), ("enc_mul", "<u4", (256,)), ("area", "<u4", (8,)), ("dec", "<u2", (16384,)),
    ("count", "<u2", (64,)), ("index", "<u2", (64,)),
    ("area_start", "<u2", (8,)), ("area_size", "<u2", (8,)),
    ("width", "u1", (8,)), ("len", "u1", (256,)), ("rank", "u1", (256,)),
    ("by_rank", "u1", (256,)), ("sorted", "u1", (256,)),
], align=True)


class EccError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {_status_name(code)} ({code})")
        self.code = code


class _Desc(ct.Structure):
    _fields_ = [("in_", ct.c_void_p), ("out", ct.c_void_p), ("n", ct.c_uint64), ("cap", ct.c_uint64),
                ("chunk_off", ct.c_void_p), ("sub_bits", ct.c_void_p), ("total_bits", ct.c_void_p),
                ("cb", ct.c_void_p), ("status", ct.c_void_p), ("t_done_ns", ct.c_void_p),
                ("C", ct.c_uint32), ("S", ct.c_uint32)]


_lock = threading.Lock()
_lib = None


def _load():
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libecc_gb300 is not built ({LIB_PATH} missing): run "
                               "`python -m lossless_entropy_coding_gb300.build`")
        lib = ct.CDLL(LIB_PATH)
        P, Z, U32, U64, I32, D = ct.c_void_p, ct.c_size_t, ct.c_uint32, ct.c_uint64, ct.c_int32, ct.c_double
        F = ct.c_float
        sig = {
            "ecc_codebook_bytes": (Z, []),
            "qlc_build_tables": (I32, [P, P, P]),
            "qlc_search_widths": (I32, [P, U32, U32, P, P]),
            "huff_build_canonical": (I32, [P, U32, P]),
            "escape_build_tables": (I32, [P, P]),
            "gqlc_build_tables": (I32, [P, U32, P, P]),
            "gqlc_search_widths": (I32, [P, U32, U32, U32, P, P]),
            "huff_build_limited": (I32, [P, U32, P]),
            "ecc_entropy_bits": (D, [P]),
            "ecc_kl_bits": (D, [P, P]),
            "ecc_code_bits": (I32, [P, P, P]),
            "ecc_num_chunks": (Z, [Z, U32]),
            "ecc_num_subblocks": (Z, [Z, U32]),
            "ecc_max_encoded_bytes": (Z, [Z, U32, U32]),
            "ecc_encode_workspace_bytes": (Z, [Z, U32]),
            "e4m3_histogram": (I32, [P, Z, P, P]),
            "huff_build_device": (I32, [P, U64, U32, P, P, P]),
            "ecc_encode": (I32, [P, Z, P, U32, U32, P, Z, P, P, P, P, Z, P, P]),
            "ecc_decode": (I32, [P, Z, P, P, Z, U32, U32, P, P, P, P]),
            "ecc_batched_workspace_bytes": (Z, [P, U32]),
            "ecc_encode_batched": (I32, [P, U32, P, Z, P, P]),
            "ecc_decode_batched": (I32, [P, U32, P, Z, P, P]),
            "ecc_selftest_wait": (I32, [P, U64, U64, U64, P, P, P]),
            "ecc_encode_static": (I32, [P, Z, P, U32, U32, P, Z, P, P, P, P, P]),
            "ecc_status_string": (ct.c_char_p, [I32]),
            "bf16_escape_table_sigma": (I32, [ct.c_double, P]),
            "bf16_escape_table_counts": (I32, [P, P]),
            "bf16_exponent_histogram": (I32, [P, Z, P, P]),
            "bf16_escape_max_encoded_bytes": (Z, [Z, U32]),
            "bf16_escape_encode": (I32, [P, Z, P, U32, U32, P, Z, P, P, P, P, Z, P, P]),
            "bf16_escape_decode": (I32, [P, Z, P, P, Z, U32, U32, P, P, P, P]),
            "ecc_layer_norm": (I32, [P, U64, U32, P, P, U32, U64, U64, F, P, U64, U32, F, P, P, P]),
            "ecc_layer_norm_grad_workspace_bytes": (Z, [U64, U64]),
            "ecc_layer_norm_grad": (I32, [P, U64, P, U64, U32, P, U32, P, P, U64, U64, P, U64, P, P, P, Z, P]),
            "ecc_linear_workspace_bytes": (Z, [P]),
            "ecc_linear": (I32, [P, P, Z, P, P]),
            "ecc_linear_grad_workspace_bytes": (Z, [P]),
            "ecc_linear_grad": (I32, [P, P, Z, P, P]),
            "ecc_token_logprob": (I32, [P, U64, U32, P, U64, U64, F, U32, P, P, P, P, P, P]),
            "ecc_token_logprob_grad": (I32, [P, U64, U32, P, U64, U64, F, P, P, P, P, P, U64, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
        return lib


def lib():
    """The loaded ctypes library (raises if it has not been built)."""
    return _load()


def _status_name(code: int) -> str:
    try:
        return _load().ecc_status_string(code).decode()
    except Exception:  # library missing: fall back to the number
        return "status"


def _check(code: int, what: str):
    if code != OK:
        raise EccError(code, what)


def _np_ptr(a: np.ndarray):
    return a.ctypes.data_as(ct.c_void_p)


def _u64(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a).astype(np.uint64, copy=False))


def _u8(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a).astype(np.uint8, copy=False))


# ------------------------------------------------------------------ host builders

def codebook_bytes() -> int:
    return int(_load().ecc_codebook_bytes())


def qlc_build_tables(count, width=BASE_WIDTHS) -> np.ndarray:
    """Host QLC codebook (raw ecc_codebook bytes)."""
    count, width = _u64(count), _u8(width)
    out = np.zeros(codebook_bytes(), np.uint8)
    _check(_load().qlc_build_tables(_np_ptr(count), _np_ptr(width), _np_ptr(out)), "qlc_build_tables")
    return out


def qlc_search_widths(count, max_distinct: int = 4, require_full: bool = False):
    count = _u64(count)
    w = np.zeros(8, np.uint8)
    cost = np.zeros(1, np.uint64)
    _check(_load().qlc_search_widths(_np_ptr(count), max_distinct, int(bool(require_full)), _np_ptr(w),
                                     _np_ptr(cost)), "qlc_search_widths")
    return w, int(cost[0])


def huff_build_canonical(weight, max_len: int = MAX_CODE_LEN) -> np.ndarray:
    """Host canonical Huffman codebook (raw ecc_codebook bytes)."""
    weight = _u64(weight)
    out = np.zeros(codebook_bytes(), np.uint8)
    _check(_load().huff_build_canonical(_np_ptr(weight), max_len, _np_ptr(out)), "huff_build_canonical")
    return out


def codebook_view(cb: np.ndarray):
    """Structured view of raw codebook bytes (fields of ecc_codebook)."""
    return np.frombuffer(np.ascontiguousarray(cb, np.uint8).tobytes(), CODEBOOK_DTYPE)[0]


def entropy_bits(count) -> float:
    return float(_load().ecc_entropy_bits(_np_ptr(_u64(count))))


def kl_bits(p_count, q_count) -> float:
    return float(_load().ecc_kl_bits(_np_ptr(_u64(p_count)), _np_ptr(_u64(q_count))))


def code_bits(count, cb: np.ndarray) -> int:
    out = np.zeros(1, np.uint64)
    cbb = _u8(cb)
    _check(_load().ecc_code_bits(_np_ptr(_u64(count)), _np_ptr(cbb), _np_ptr(out)), "ecc_code_bits")
    return int(out[0])


def num_chunks(n: int, C: int) -> int:
    return int(_load().ecc_num_chunks(n, C))


def num_subblocks(n: int, S: int) -> int:
    return int(_load().ecc_num_subblocks(n, S))


def max_encoded_bytes(n: int, C: int, max_len: int) -> int:
    return int(_load().ecc_max_encoded_bytes(n, C, max_len))


def encode_workspace_bytes(n: int, C: int) -> int:
    return int(_load().ecc_encode_workspace_bytes(n, C))


def _register_path(cb) -> bool:
    """Whether the decoder reads codes of codebook cb through its prefix
    register path (QLC with a 3-bit prefix and codes of at most 11 bits)
    rather than through its first-level table.  cb: host codebook bytes, a
    device codebook made by to_device, or None (taken as the register
    path)."""
    if cb is None:
        return True
    tag = getattr(cb, "_ecc_register_path", None)
    if tag is not None:
        return bool(tag)
    if not isinstance(cb, np.ndarray):  # a device tensor of unknown origin
        return True
    v = codebook_view(cb)
    return int(v["family"]) == FAMILY_QLC and int(v["prefix_bits"]) == 3 and int(v["max_len"]) <= 11


def default_subblock(C: int, cb=None) -> int:
    """Sub-block size used when none is given.

    A QLC codebook the decoder reads through its prefix registers (or no
    codebook given): C/64, clamped to [64, 256].  Any other codebook (Huffman,
    the escape code, a length-limited Huffman or a QLC of fewer areas):
    C/128, clamped to [64, 128].  Its decoder waits on dependent table
    lookups, and sub-blocks of 128 symbols give each lane two independent
    streams at the same number of warps (1 GiB gradient tensor, Huffman
    decode: 1.14 -> 1.03 ms at 16 KiB chunks, 1.15 -> 1.04 ms at 64 KiB,
    for 1/64 byte a symbol more of sub-block counts); the QLC decoder is
    issue-bound and gains nothing.  Larger sub-blocks cost the decoder
    occupancy: a warp stages 32 sub-blocks or more, so with S > 256 fewer
    warps fit an SM."""
    if _register_path(cb):
        return int(min(256, max(64, C // 64)))
    return int(min(128, max(64, C // 128)))


# ------------------------------------------------------------------ device calls

def _torch():
    import torch
    return torch


def _stream_ptr(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ct.c_void_p(s.cuda_stream)


def _dptr(t):
    return ct.c_void_p(t.data_ptr()) if t is not None else ct.c_void_p(0)


def gqlc_build_tables(count, width, prefix_bits: int) -> np.ndarray:
    """Host QLC codebook with 2^prefix_bits areas (raw ecc_codebook bytes)."""
    count = _u64(count)
    w = np.zeros(8, np.uint8)
    w[:len(width)] = _u8(width)
    out = np.zeros(codebook_bytes(), np.uint8)
    _check(_load().gqlc_build_tables(_np_ptr(count), int(prefix_bits), _np_ptr(w), _np_ptr(out)),
           "gqlc_build_tables")
    return out


def gqlc_search_widths(count, prefix_bits: int, max_distinct: int = 4, require_full: bool = False):
    """Best widths of the 2^prefix_bits areas; returns (width, cost_bits)."""
    count = _u64(count)
    w = np.zeros(8, np.uint8)
    cost = np.zeros(1, np.uint64)
    _check(_load().gqlc_search_widths(_np_ptr(count), int(prefix_bits), int(max_distinct), int(bool(require_full)),
                                      _np_ptr(w), _np_ptr(cost)), "gqlc_search_widths")
    return w[:1 << prefix_bits].copy(), int(cost[0])


def huff_build_limited(weight, max_len: int) -> np.ndarray:
    """Host canonical Huffman codebook with lengths of at most max_len
    (package-merge; raw ecc_codebook bytes)."""
    weight = _u64(weight)
    out = np.zeros(codebook_bytes(), np.uint8)
    _check(_load().huff_build_limited(_np_ptr(weight), int(max_len), _np_ptr(out)), "huff_build_limited")
    return out


def escape_build_tables(count) -> np.ndarray:
    """Host escape-code codebook (raw ecc_codebook bytes): top-7 e4m3
    exponents in 3 bits, others 000 + exponent, sign and mantissa kept."""
    count = _u64(count)
    out = np.zeros(codebook_bytes(), np.uint8)
    _check(_load().escape_build_tables(_np_ptr(count), _np_ptr(out)), "escape_build_tables")
    return out


def to_device(cb: np.ndarray, device="cuda"):
    """Copy raw codebook bytes to a device tensor (what the kernels read).
    The tensor remembers which decoder path the codebook takes, for
    default_subblock."""
    torch = _torch()
    t = torch.from_numpy(np.ascontiguousarray(cb, np.uint8)).to(device)
    t._ecc_register_path = _register_path(cb)
    return t


def e4m3_histogram(x, count=None, stream=None):
    """Add the byte histogram of device tensor x to count (int64[256] on the
    device, zero-initialised when not given) and return count."""
    torch = _torch()
    if count is None:
        count = torch.zeros(256, dtype=torch.int64, device=x.device)
    _check(_load().e4m3_histogram(_dptr(x), x.numel(), _dptr(count), _stream_ptr(stream)), "e4m3_histogram")
    return count


def huff_build_device(count, add: int = 1, max_len: int = MAX_CODE_LEN, out=None, status=None, stream=None):
    """Build the canonical Huffman codebook of weights count + add on the
    device (count: int64[256] device tensor, e.g. from e4m3_histogram).
    Returns (codebook uint8 device tensor, status int32[1] device tensor);
    nothing is synchronised, read status after the stream reaches the call."""
    torch = _torch()
    dev = count.device
    if out is None:
        out = torch.empty(codebook_bytes(), dtype=torch.uint8, device=dev)
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=dev)
    _check(_load().huff_build_device(_dptr(count), int(add), int(max_len), _dptr(out), _dptr(status),
                                     _stream_ptr(stream)), "huff_build_device")
    return out, status


@dataclass
class Encoded:
    """Device tensors of one encoded container (payload holds out_cap bytes;
    the used part is payload[:chunk_off[-1]])."""
    payload: object
    chunk_off: object
    sub_bits: object
    total_bits: object
    status: object
    n: int
    C: int
    S: int


def ecc_encode(x, dev_cb, C: int = 16384, S: int | None = None, max_len: int = MAX_CODE_LEN, out=None,
               chunk_off=None, sub_bits=None, total_bits=None, ws=None, status=None, stream=None) -> Encoded:
    """Encode device bytes x with device codebook dev_cb (no synchronisation;
    read .status after the stream reaches this point)."""
    torch = _torch()
    dev = x.device
    n = x.numel()
    S = default_subblock(C, dev_cb) if S is None else S
    if out is None:
        out = torch.empty(max(16, max_encoded_bytes(n, C, max_len)), dtype=torch.uint8, device=dev)
    nch = num_chunks(n, C)
    if chunk_off is None:
        chunk_off = torch.empty(nch + 1, dtype=torch.int64, device=dev)
    if sub_bits is None:
        sub_bits = torch.empty(max(1, num_subblocks(n, S)), dtype=torch.int16, device=dev)
    if total_bits is None:
        total_bits = torch.empty(1, dtype=torch.int64, device=dev)
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=dev)
    if ws is None:
        ws = torch.empty(encode_workspace_bytes(n, C), dtype=torch.uint8, device=dev)
    _check(_load().ecc_encode(_dptr(x), n, _dptr(dev_cb), C, S, _dptr(out), out.numel(), _dptr(chunk_off),
                              _dptr(sub_bits), _dptr(total_bits), _dptr(ws), ws.numel(), _dptr(status),
                              _stream_ptr(stream)), "ecc_encode")
    return Encoded(out, chunk_off, sub_bits, total_bits, status, n, C, S)


def ecc_decode(enc: Encoded, dev_cb, out=None, status=None, stream=None):
    """Decode a container into device bytes (returns (out, status))."""
    torch = _torch()
    dev = enc.payload.device
    if out is None:
        out = torch.empty(max(16, enc.n), dtype=torch.uint8, device=dev)
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=dev)
    _check(_load().ecc_decode(_dptr(enc.payload), enc.payload.numel(), _dptr(enc.chunk_off), _dptr(enc.sub_bits),
                              enc.n, enc.C, enc.S, _dptr(dev_cb), _dptr(out), _dptr(status), _stream_ptr(stream)),
           "ecc_decode")
    return out, status


def make_descs(items) -> ct.Array:
    """ecc_desc array from dicts with keys in, out, n, cap, chunk_off,
    sub_bits, total_bits, cb, status, t_done_ns, C, S (tensors or None)."""
    arr = (_Desc * len(items))()
    for d, it in zip(arr, items):
        d.in_ = it["in"].data_ptr()
        d.out = it["out"].data_ptr()
        d.n = int(it["n"])
        d.cap = int(it["cap"])
        d.chunk_off = it["chunk_off"].data_ptr()
        d.sub_bits = it["sub_bits"].data_ptr()
        d.total_bits = it["total_bits"].data_ptr() if it.get("total_bits") is not None else 0
        d.cb = it["cb"].data_ptr()
        d.status = it["status"].data_ptr()
        d.t_done_ns = it["t_done_ns"].data_ptr() if it.get("t_done_ns") is not None else 0
        d.C = int(it["C"])
        d.S = int(it["S"])
    return arr


def batched_workspace_bytes(descs) -> int:
    return int(_load().ecc_batched_workspace_bytes(ct.cast(descs, ct.c_void_p), len(descs)))


def ecc_encode_batched(descs, ws, t_start=None, stream=None):
    _check(_load().ecc_encode_batched(ct.cast(descs, ct.c_void_p), len(descs), _dptr(ws), ws.numel(),
                                      _dptr(t_start), _stream_ptr(stream)), "ecc_encode_batched")


def ecc_decode_batched(descs, ws, t_start=None, stream=None):
    _check(_load().ecc_decode_batched(ct.cast(descs, ct.c_void_p), len(descs), _dptr(ws), ws.numel(),
                                      _dptr(t_start), _stream_ptr(stream)), "ecc_decode_batched")


def ecc_selftest_wait(flags, chunk: int, aggregate: int, timeout_ns: int, prefix, status, stream=None):
    _check(_load().ecc_selftest_wait(_dptr(flags), chunk, aggregate, timeout_ns, _dptr(prefix), _dptr(status),
                                     _stream_ptr(stream)), "ecc_selftest_wait")


STATIC_MAX_CHUNKS = 65536


def ecc_encode_static(x, dev_cb, C: int = 16384, S: int | None = None, max_len: int = MAX_CODE_LEN, out=None,
                      chunk_off=None, sub_bits=None, total_bits=None, status=None, stream=None) -> Encoded:
    """ecc_encode with the library's built-in scratch array instead of a
    caller workspace (for callers that cannot allocate device memory on
    their call path).  Calls that may overlap on the GPU must be ordered by
    the caller: they share the scratch array."""
    torch = _torch()
    dev = x.device
    n = x.numel()
    S = default_subblock(C, dev_cb) if S is None else S
    if out is None:
        out = torch.empty(max(16, max_encoded_bytes(n, C, max_len)), dtype=torch.uint8, device=dev)
    if chunk_off is None:
        chunk_off = torch.empty(num_chunks(n, C) + 1, dtype=torch.int64, device=dev)
    if sub_bits is None:
        sub_bits = torch.empty(max(1, num_subblocks(n, S)), dtype=torch.int16, device=dev)
    if total_bits is None:
        total_bits = torch.empty(1, dtype=torch.int64, device=dev)
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=dev)
    _check(_load().ecc_encode_static(_dptr(x), n, _dptr(dev_cb), C, S, _dptr(out), out.numel(), _dptr(chunk_off),
                                     _dptr(sub_bits), _dptr(total_bits), _dptr(status), _stream_ptr(stream)),
           "ecc_encode_static")
    return Encoded(out, chunk_off, sub_bits, total_bits, status, n, C, S)


# ---------------------------------------------------------------- BF16 exponent escape code

def bf16_escape_table_sigma(sigma: float) -> np.ndarray:
    """The 7-exponent table of N(0, sigma^2) in BF16 (uint8[7], rank order)."""
    top = np.zeros(7, np.uint8)
    _check(_load().bf16_escape_table_sigma(float(sigma), _np_ptr(top)), "bf16_escape_table_sigma")
    return top


def bf16_escape_table_counts(count) -> np.ndarray:
    """The 7 most frequent exponent fields of a count vector (uint8[7])."""
    count = _u64(count)
    top = np.zeros(7, np.uint8)
    _check(_load().bf16_escape_table_counts(_np_ptr(count), _np_ptr(top)), "bf16_escape_table_counts")
    return top


def bf16_exponent_histogram(x, count=None, stream=None):
    """Device exponent-field counts of BF16 values (x: uint16/int16/bfloat16
    device tensor), added to count (int64[256], allocated if None)."""
    torch = _torch()
    if count is None:
        count = torch.zeros(256, dtype=torch.int64, device=x.device)
    _check(_load().bf16_exponent_histogram(_dptr(x), x.numel(), _dptr(count), _stream_ptr(stream)),
           "bf16_exponent_histogram")
    return count


def bf16_escape_max_encoded_bytes(n: int, C: int) -> int:
    return int(_load().bf16_escape_max_encoded_bytes(n, C))


def bf16_escape_encode(x, top7, C: int = 4096, S: int | None = None, out=None, chunk_off=None, sub_bits=None,
                       total_bits=None, ws=None, status=None, stream=None) -> Encoded:
    """Encode device BF16 values (2-byte elements) with the escape code and
    the host table top7."""
    torch = _torch()
    dev = x.device
    n = x.numel()
    S = default_subblock(C) if S is None else S
    top7 = np.ascontiguousarray(top7, dtype=np.uint8)
    if out is None:
        out = torch.empty(max(16, bf16_escape_max_encoded_bytes(n, C)), dtype=torch.uint8, device=dev)
    if chunk_off is None:
        chunk_off = torch.empty(num_chunks(n, C) + 1, dtype=torch.int64, device=dev)
    if sub_bits is None:
        sub_bits = torch.empty(max(1, num_subblocks(n, S)), dtype=torch.int16, device=dev)
    if total_bits is None:
        total_bits = torch.empty(1, dtype=torch.int64, device=dev)
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=dev)
    if ws is None:
        ws = torch.empty(encode_workspace_bytes(n, C), dtype=torch.uint8, device=dev)
    _check(_load().bf16_escape_encode(_dptr(x), n, _np_ptr(top7), C, S, _dptr(out), out.numel(), _dptr(chunk_off),
                                      _dptr(sub_bits), _dptr(total_bits), _dptr(ws), ws.numel(), _dptr(status),
                                      _stream_ptr(stream)), "bf16_escape_encode")
    return Encoded(out, chunk_off, sub_bits, total_bits, status, n, C, S)


def bf16_escape_decode(enc: Encoded, top7, out=None, status=None, stream=None):
    """Decode a BF16 escape-code container (returns (values int16, status))."""
    torch = _torch()
    dev = enc.payload.device
    top7 = np.ascontiguousarray(top7, dtype=np.uint8)
    if out is None:
        out = torch.empty(max(8, enc.n), dtype=torch.int16, device=dev)
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=dev)
    _check(_load().bf16_escape_decode(_dptr(enc.payload), enc.payload.numel(), _dptr(enc.chunk_off),
                                      _dptr(enc.sub_bits), enc.n, enc.C, enc.S, _np_ptr(top7), _dptr(out),
                                      _dptr(status), _stream_ptr(stream)), "bf16_escape_decode")
    return out, status


# ---------------------------------------------------------------- language-model operators
# Matrices are torch tensors [..., columns] whose last dimension is contiguous
# and whose leading dimensions collapse to rows of one stride.  e4m3 tensors
# are uint8 (the coders' bytes) or torch.float8_e4m3fn.  A call on another
# stream than the current one allocates its outputs and scratch for that
# stream; the caller orders the streams, as for the coding calls.

F32, BF16, F16, E4M3 = range(4)
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
MAX_TOP = 32

_types = {}  # torch element type -> C code, filled by _bind
_empty = _empty_strided = _empty_like = _raw_stream = _current_device = _f32 = _i32 = _i64 = _u8t = None


def _bind():
    """Look up once what every call below needs."""
    global _empty, _empty_strided, _empty_like, _raw_stream, _current_device, _f32, _i32, _i64, _u8t
    torch = _torch()
    _types.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16, torch.float8_e4m3fn: E4M3,
                   torch.uint8: E4M3})
    _empty, _f32, _i32, _i64, _u8t = torch.empty, torch.float32, torch.int32, torch.int64, torch.uint8
    _empty_strided, _empty_like = torch.empty_strided, torch.empty_like
    torch.cuda.init()
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _load()


def _refuse(what: str):
    raise EccError(ERR_ARG, what)


def _new(shape, dtype, device):
    """A contiguous tensor (torch.empty takes twice as long over a shape that is a tuple)."""
    n = len(shape)
    if n == 1:
        return _empty(shape[0], dtype=dtype, device=device)
    if n == 2:
        return _empty_strided(shape, (shape[1] or 1, 1), dtype=dtype, device=device)
    return _empty(shape, dtype=dtype, device=device)


def _type(t, what: str) -> int:
    code = _types.get(t)
    return _refuse(what + ": element type") if code is None else code


def _matrix(t, what: str):
    """(rows, columns, leading dimension) of a tensor of rows."""
    shape, stride = t.shape, t.stride()
    n = len(shape)
    if n == 0 or (stride[-1] != 1 and shape[-1] > 1):
        _refuse(what + ": rows are not contiguous")
    cols = shape[-1]
    if n == 2:
        rows = shape[0]
        return rows, cols, stride[0] if rows > 1 else cols
    rows, ld = 1, cols
    for i in range(n - 2, -1, -1):
        if shape[i] == 1:
            continue
        if rows == 1:
            ld = stride[i]
        elif shape[i] and stride[i] != rows * ld:
            _refuse(what + ": leading dimensions do not collapse")
        rows *= shape[i]
    return rows, cols, ld


def _vector(t, n: int, dev: int, what: str, dtype=None):
    """Pointer of a contiguous tensor of n elements (0 for None)."""
    if t is None:
        return 0
    if t.numel() != n or not t.is_contiguous() or t.get_device() != dev or (dtype is not None and t.dtype != dtype):
        _refuse(what)
    return t.data_ptr()


def _on_stream(f):
    """Run f with the device of its first tensor current and, where a stream is
    given, with that stream current (so that what f allocates belongs to it);
    f gets the stream's handle."""
    @functools.wraps(f)
    def call(x, *args, stream=None, **kw):
        if _empty is None:
            _bind()
        dev = x.get_device()
        if dev < 0:
            _refuse(f.__name__ + ": needs CUDA tensors")
        if stream is None and dev == _current_device():
            kw["stream"] = _raw_stream(dev)
            return f(x, *args, **kw)
        torch = _torch()
        with torch.cuda.device(dev):
            s = torch.cuda.current_stream() if stream is None else stream
            with torch.cuda.stream(s):
                return f(x, *args, stream=s.cuda_stream, **kw)
    return call


@_on_stream
def ecc_layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, out_dtype=None, out_scale: float = 1.0,
                   mean=None, rstd=None, stream=None):
    """Layer norm over the last dimension of device tensor x; returns (out,
    mean, rstd).  out_dtype: x's type (default), or uint8 / float8_e4m3fn for
    e4m3 values of out * out_scale.  weight, bias: of x's type or float32."""
    dev, device, shape, dtype = x.get_device(), x.device, x.shape, x.dtype
    rows, cols, ldx = _matrix(x, "ecc_layer_norm: x")
    if out is None:
        out = _new(shape, out_dtype or dtype, device)
        ldy = cols
    elif out.shape != shape or out.get_device() != dev:
        _refuse("ecc_layer_norm: out")
    else:
        ldy = _matrix(out, "ecc_layer_norm: out")[2]
    lead = (rows,) if len(shape) == 2 else shape[:-1]
    if mean is None:
        mean = _new(lead, _f32, device)
        pmean = mean.data_ptr()
    else:
        pmean = _vector(mean, rows, dev, "ecc_layer_norm: mean", _f32)
    if rstd is None:
        rstd = _new(lead, _f32, device)
        prstd = rstd.data_ptr()
    else:
        prstd = _vector(rstd, rows, dev, "ecc_layer_norm: rstd", _f32)
    p_dtype = weight.dtype if weight is not None else bias.dtype if bias is not None else dtype
    code = _lib.ecc_layer_norm(
        x.data_ptr(), ldx, _type(dtype, "ecc_layer_norm"), _vector(weight, cols, dev, "ecc_layer_norm: weight"),
        _vector(bias, cols, dev, "ecc_layer_norm: bias", p_dtype), _type(p_dtype, "ecc_layer_norm"), rows, cols, eps,
        out.data_ptr(), ldy, _type(out.dtype, "ecc_layer_norm"), out_scale, pmean, prstd, stream)
    if code:
        _check(code, "ecc_layer_norm")
    return out, mean, rstd


def layer_norm_grad_workspace_bytes(rows: int, cols: int) -> int:
    return int(_load().ecc_layer_norm_grad_workspace_bytes(rows, cols))


@_on_stream
def ecc_layer_norm_grad(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, ws=None, stream=None):
    """Backward pass of ecc_layer_norm; returns (dx, dweight, dbias), the last
    two float32.  weight None: ones (dweight and dbias are still summed)."""
    dev = dy.get_device()
    rows, cols, ldx = _matrix(x, "ecc_layer_norm_grad: x")
    if x.shape != dy.shape or x.dtype != dy.dtype or x.get_device() != dev:
        _refuse("ecc_layer_norm_grad: x")
    _, _, lddy = _matrix(dy, "ecc_layer_norm_grad: dy")
    if dx is None:
        dx = _new(x.shape, x.dtype, x.device)
    elif dx.shape != x.shape or dx.dtype != x.dtype or dx.get_device() != dev:
        _refuse("ecc_layer_norm_grad: dx")
    _, _, lddx = _matrix(dx, "ecc_layer_norm_grad: dx")
    if dweight is None:
        dweight = _empty(cols, dtype=_f32, device=x.device)
    if dbias is None:
        dbias = _empty(cols, dtype=_f32, device=x.device)
    lib = _lib
    if ws is None:
        ws = _empty(lib.ecc_layer_norm_grad_workspace_bytes(rows, cols), dtype=_u8t, device=x.device)
    if mean is None or rstd is None:
        _refuse("ecc_layer_norm_grad: mean and rstd")
    _check(lib.ecc_layer_norm_grad(
        dy.data_ptr(), lddy, x.data_ptr(), ldx, _type(x.dtype, "ecc_layer_norm_grad"),
        _vector(weight, cols, dev, "ecc_layer_norm_grad: weight"),
        _type(x.dtype if weight is None else weight.dtype, "ecc_layer_norm_grad"),
        _vector(mean, rows, dev, "ecc_layer_norm_grad: mean", _f32),
        _vector(rstd, rows, dev, "ecc_layer_norm_grad: rstd", _f32), rows, cols, dx.data_ptr(), lddx,
        _vector(dweight, cols, dev, "ecc_layer_norm_grad: dweight", _f32),
        _vector(dbias, cols, dev, "ecc_layer_norm_grad: dbias", _f32), ws.data_ptr(), ws.numel(), stream),
        "ecc_layer_norm_grad")
    return dx, dweight, dbias


_LINEAR_JOB = struct.Struct("@6P8Q2f6I")        # ecc_linear_job
_LINEAR_GRAD_JOB = struct.Struct("@7P9Qf5I")    # ecc_linear_grad_job


def _activation(act: str, what: str) -> int:
    code = ACTIVATIONS.get(act)
    return _refuse(what + ": activation") if code is None else code


def _operand(t, rows: int, cols: int, dev: int, what: str):
    """(pointer, leading dimension, type) of a [rows, cols] tensor (zeros for None)."""
    if t is None:
        return 0, 0, 0
    r, c, ld = _matrix(t, what)
    if r != rows or c != cols or t.get_device() != dev:
        _refuse(what + ": shape or device")
    return t.data_ptr(), ld, _type(t.dtype, what)


@_on_stream
def ecc_linear(x, w, bias=None, residual=None, act: str = "none", scale: float = 1.0, out=None, out_dtype=None,
               out_scale: float = 1.0, pre=None, ws=None, status=None, stream=None):
    """act(scale * x w^T + bias) + residual of device tensors x [..., K] and
    w [N, K] (bfloat16, float16 or e4m3); returns (out [..., N], status).
    out_dtype: x's type by default, bfloat16 for e4m3 operands; uint8 or
    float8_e4m3fn: e4m3 values of out * out_scale.  pre: a tensor [..., N]
    that receives the activation's argument, for ecc_linear_grad."""
    dev = x.get_device()
    M, K, ldx = _matrix(x, "ecc_linear: x")
    in_type = _type(x.dtype, "ecc_linear: x")
    if w.dim() != 2:
        _refuse("ecc_linear: w")
    N = w.shape[0]
    pw, ldw, w_type = _operand(w, N, K, dev, "ecc_linear: w")
    if w_type != in_type:
        _refuse("ecc_linear: x and w of different types")
    if out is None:
        shape = (M, N) if x.dim() == 2 else (*x.shape[:-1], N)
        out = _new(shape, out_dtype or (_torch().bfloat16 if in_type == E4M3 else x.dtype), x.device)
    if status is None:
        status = _empty(1, dtype=_i32, device=x.device)
    pout, ldout, out_type = _operand(out, M, N, dev, "ecc_linear: out")
    pres, ldres, res_type = _operand(residual, M, N, dev, "ecc_linear: residual")
    ppre, ldpre, pre_type = _operand(pre, M, N, dev, "ecc_linear: pre")
    job = _LINEAR_JOB.pack(x.data_ptr(), pw, _vector(bias, N, dev, "ecc_linear: bias"), pres, pout, ppre, M, N, K, ldx,
                           ldw, ldres, ldout, ldpre, scale, out_scale, in_type,
                           0 if bias is None else _type(bias.dtype, "ecc_linear: bias"), res_type, out_type, pre_type,
                           _activation(act, "ecc_linear"))
    lib = _lib
    if ws is None:
        need = lib.ecc_linear_workspace_bytes(job)
        ws = _empty(need, dtype=_u8t, device=x.device) if need else None
    _check(lib.ecc_linear(job, 0 if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(),
                          _vector(status, 1, dev, "ecc_linear: status", _i32), stream), "ecc_linear")
    return out, status


@_on_stream
def ecc_linear_grad(dy, x, w, pre=None, act: str = "none", scale: float = 1.0, dx=None, dw=None, dbias=None,
                    dw_dtype=None, want=("dx", "dw", "dbias"), ws=None, status=None, stream=None):
    """Backward pass of ecc_linear's product; returns (dx, dw, dbias, status),
    None for what `want` leaves out.  pre: the activation's argument (needed
    unless act is "none").  dw_dtype: x's type (default) or float32; dbias is
    float32."""
    dev = dy.get_device()
    M, N, lddy = _matrix(dy, "ecc_linear_grad: dy")
    in_type = _type(dy.dtype, "ecc_linear_grad: dy")
    K = x.shape[-1]
    px, ldx, x_type = _operand(x, M, K, dev, "ecc_linear_grad: x")
    pw, ldw, w_type = _operand(w, N, K, dev, "ecc_linear_grad: w")
    if x_type != in_type or w_type != in_type:
        _refuse("ecc_linear_grad: dy, x and w of different types")
    ppre, ldpre, pre_type = _operand(pre, M, N, dev, "ecc_linear_grad: pre")
    if dx is None and "dx" in want:
        dx = _new(x.shape, x.dtype, x.device)
    if dw is None and "dw" in want:
        dw = _new((N, K), dw_dtype or x.dtype, x.device)
    if dbias is None and "dbias" in want:
        dbias = _empty(N, dtype=_f32, device=x.device)
    if status is None:
        status = _empty(1, dtype=_i32, device=x.device)
    pdx, lddx, dx_type = _operand(dx, M, K, dev, "ecc_linear_grad: dx")
    if dx is not None and dx_type != in_type:
        _refuse("ecc_linear_grad: dx")
    pdw, lddw, dw_type = _operand(dw, N, K, dev, "ecc_linear_grad: dw")
    job = _LINEAR_GRAD_JOB.pack(dy.data_ptr(), px, pw, ppre, pdx, pdw,
                                _vector(dbias, N, dev, "ecc_linear_grad: dbias", _f32), M, N, K, lddy, ldx,
                                ldw, ldpre, lddx, lddw, scale, in_type, pre_type, dw_type,
                                _activation(act, "ecc_linear_grad"), 0)
    lib = _lib
    if ws is None:
        need = lib.ecc_linear_grad_workspace_bytes(job)
        ws = _empty(need, dtype=_u8t, device=x.device) if need else None
    _check(lib.ecc_linear_grad(job, 0 if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(),
                               _vector(status, 1, dev, "ecc_linear_grad: status", _i32), stream),
           "ecc_linear_grad")
    return dx, dw, dbias, status


@dataclass
class TokenLogprob:
    """Device tensors of ecc_token_logprob (None where not asked for), in nats."""
    logprob: object
    entropy: object
    lse: object
    top_logprob: object
    top_index: object


@_on_stream
def ecc_token_logprob(logits, tokens=None, top: int = 0, scale: float = 1.0, stream=None) -> TokenLogprob:
    """Log probabilities of tokens (int64 [...], negative: none) under softmax
    of scale * logits [..., vocab], with each row's entropy, log partition and
    `top` most probable tokens (at most 32)."""
    dev = logits.get_device()
    rows, vocab, ld = _matrix(logits, "ecc_token_logprob: logits")
    lead = (rows,) if logits.dim() == 2 else logits.shape[:-1]
    if not 0 <= top <= MAX_TOP:
        _refuse("ecc_token_logprob: top")
    ptok = _vector(tokens, rows, dev, "ecc_token_logprob: tokens", _i64)
    device = logits.device
    logprob = _new(lead, _f32, device) if tokens is not None else None
    entropy = _new(lead, _f32, device)
    lse = _new(lead, _f32, device)
    top_logprob = top_index = None
    if top:
        top_logprob = _new((*lead, top), _f32, device)
        top_index = _new((*lead, top), _i32, device)
    _check(_lib.ecc_token_logprob(
        logits.data_ptr(), ld, _type(logits.dtype, "ecc_token_logprob"), ptok, rows, vocab, scale, top,
        0 if logprob is None else logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), top_logprob.data_ptr() if top else 0,
        top_index.data_ptr() if top else 0, stream), "ecc_token_logprob")
    return TokenLogprob(logprob, entropy, lse, top_logprob, top_index)


@_on_stream
def ecc_token_logprob_grad(logits, tokens, lse, entropy=None, dlogprob=None, dentropy=None, scale: float = 1.0,
                           dlogits=None, stream=None):
    """Gradient with respect to the logits of sum(dlogprob * logprob +
    dentropy * entropy); returns dlogits (which may be given as logits
    itself)."""
    dev = logits.get_device()
    rows, vocab, ld = _matrix(logits, "ecc_token_logprob_grad: logits")
    if dlogits is None:
        dlogits = _new(logits.shape, logits.dtype, logits.device)
    elif dlogits.shape != logits.shape or dlogits.dtype != logits.dtype or dlogits.get_device() != dev:
        _refuse("ecc_token_logprob_grad: dlogits")
    _, _, ldd = _matrix(dlogits, "ecc_token_logprob_grad: dlogits")
    f = _f32
    _check(_lib.ecc_token_logprob_grad(
        logits.data_ptr(), ld, _type(logits.dtype, "ecc_token_logprob_grad"),
        _vector(tokens, rows, dev, "ecc_token_logprob_grad: tokens", _i64), rows, vocab, scale,
        _vector(lse, rows, dev, "ecc_token_logprob_grad: lse", f),
        _vector(entropy, rows, dev, "ecc_token_logprob_grad: entropy", f),
        _vector(dlogprob, rows, dev, "ecc_token_logprob_grad: dlogprob", f),
        _vector(dentropy, rows, dev, "ecc_token_logprob_grad: dentropy", f), dlogits.data_ptr(), ldd, stream),
        "ecc_token_logprob_grad")
    return dlogits
