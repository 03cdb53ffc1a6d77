"""Python binding of libdflash.so: argument marshalling only.

Every function here checks tensor placement, dtype and contiguity, turns
tensors into raw device pointers and calls the C ABI of the same name
(``include/dflash.h``) on the current HIP stream.  All arithmetic of the path
runs in the library's HIP kernels.  Importing this package fails if the
library has not been built (``python block_draft_select_amd/build.py``).
"""

import ctypes
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdflash.so")

F32 = 0
BF16 = 1
K_MAX, L_MAX, R_MAX, V_MAX, CHUNK = 16, 16, 256, 2097152, 4096
STATIC_SCRATCH_BYTES = 8 << 20
ROWS_MAX, DISTILL_K_MAX = 4194304, 1024
LOGPROBS_M_MAX, TOP_MAX, H_MAX = 1024, 32, 65536

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = 0, 1, 2, 3, 4

KERNELS = ("topk", "gate", "scores", "trace", "stats", "finalize", "cycle_stream", "cycle_scores",
           "cycle_finalize", "conv2tap", "trace_viterbi", "topk_merge", "shard_stats", "shard_finalize", "sample",
           "filter", "distill", "distill_grad", "quant_i8", "linear_i8", "logprobs", "logprobs_grad")


class dflash_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "L", "V", "K", "r", "hidden", "logit_dtype", "param_dtype")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class dflash_rows(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("stride", ctypes.c_int64), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class dflash_filters(ctypes.Structure):
    _fields_ = [("T", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p), ("group", ctypes.c_int32)]


class dflash_linear(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("xq_stride", ctypes.c_int64), ("wq_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("N", ctypes.c_int32), ("H", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class DFlashError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{message} (status {status})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python block_draft_select_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, U64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t
    I64, F64 = ctypes.c_int64, ctypes.c_double
    D, W, F = ctypes.POINTER(dflash_dims), ctypes.POINTER(dflash_rows), ctypes.POINTER(dflash_filters)
    L = ctypes.POINTER(dflash_linear)
    sig = {
        "dflash_abi_version": (I32, []),
        "dflash_status_string": (ctypes.c_char_p, [I32]),
        "dflash_last_error": (ctypes.c_char_p, []),
        "dflash_workspace_bytes": (I32, [D, ctypes.POINTER(SZ)]),
        "dflash_workspace_init": (I32, [P, SZ, P]),
        "dflash_topk": (I32, [D, P, P, P, P, SZ, P]),
        "dflash_pair_scores": (I32, [D, P, P, P, P, P, P, P, P, SZ, P]),
        "dflash_trace": (I32, [D, P, P, P, P, U64, P, P, P, P]),
        "dflash_verify": (I32, [D, P, P, P, P, P, P, U64, P, P, P, SZ, P]),
        "dflash_cycle": (I32, [D, P, P, P, P, P, P, P, P, U64, P, P, P, P, P, P, P, P, P, SZ, P]),
        "dflash_cycle_maxsum": (I32, [D, P, P, P, P, P, P, P, P, U64, P, P, P, P, P, P, P, P, P, SZ, P]),
        "dflash_cycle_static": (I32, [D, P, P, P, P, P, P, P, P, U64, P, P, P, P, P, P, P, P, P]),
        "dflash_conv2tap": (I32, [D, P, P, P, P, P]),
        "dflash_trace_viterbi": (I32, [D, P, P, P, P, P, P]),
        "dflash_topk_merge": (I32, [D, I32, ctypes.POINTER(I32), P, P, P, P, P]),
        "dflash_shard_stats_bytes": (I32, [D, I32, ctypes.POINTER(I32), ctypes.POINTER(SZ)]),
        "dflash_shard_stats": (I32, [D, I32, ctypes.POINTER(I32), I32, P, P, P, P]),
        "dflash_verify_shards": (I32, [D, I32, ctypes.POINTER(I32), ctypes.POINTER(P), P, P, P, P, P, P, U64, P, P,
                                       P]),
        "dflash_rows_workspace_bytes": (I32, [W, ctypes.POINTER(SZ)]),
        "dflash_sample": (I32, [W, P, F, P, P, P, P, P, SZ, P]),
        "dflash_filter": (I32, [W, P, F, ctypes.c_float, P, I64, P, P, SZ, P]),
        "dflash_distill": (I32, [W, P, I32, F64, P, P, P, P, P, P, P, P, SZ, P]),
        "dflash_distill_grad": (I32, [W, P, I32, F64, P, P, P, P, P, P, P, P, I64, P]),
        "dflash_logprobs": (I32, [W, P, P, I32, I32, P, P, P, P, I32, P, P, P, SZ, P]),
        "dflash_logprobs_grad": (I32, [W, P, P, I32, I32, P, P, P, P, P, P, I64, P]),
        "dflash_quant_i8": (I32, [W, P, P, I64, P, P]),
        "dflash_linear_i8": (I32, [L, P, P, P, P, P, P]),
        "dflash_read_probe": (I32, [P, SZ, P, P]),
        "dflash_copy_probe": (I32, [P, P, SZ, P]),
        "dflash_kernel_name": (ctypes.c_char_p, [I32]),
        "dflash_profile_enable": (I32, [I32]),
        "dflash_profile_collect": (I32, [I32, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_double)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _check(status):
    if status != OK:
        raise DFlashError(status, lib.dflash_last_error().decode())


# ------------------------------------------------------------------ helpers

def dims(B, L, V, K, r, hidden, logit_dtype, param_dtype):
    """A ``dflash_dims`` value (dtypes: F32 / BF16 or the strings 'f32'/'bf16')."""
    conv = {"f32": F32, "bf16": BF16, F32: F32, BF16: BF16}
    return dflash_dims(int(B), int(L), int(V), int(K), int(r), int(hidden),
                       conv[logit_dtype], conv[param_dtype])


def workspace_bytes(d):
    n = ctypes.c_size_t(0)
    _check(lib.dflash_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def workspace(d, device="cuda"):
    """A zero-filled workspace tensor large enough for every entry point."""
    return torch.zeros(max(workspace_bytes(d), 16), dtype=torch.uint8, device=device)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_TORCH_LOGIT = {F32: torch.float32, BF16: torch.bfloat16}


def _ptr(t, name, dtype=None, numel=None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    return ctypes.c_void_p(t.data_ptr())


# ------------------------------------------------------------------ entry points

def dflash_topk(d, U, cand_idx, cand_logit, ws, stream=None):
    R = d.B * d.L
    _check(lib.dflash_topk(ctypes.byref(d), _ptr(U, "U", _TORCH_LOGIT[d.logit_dtype], R * d.V),
                           _ptr(cand_idx, "cand_idx", torch.int32, R * d.K),
                           _ptr(cand_logit, "cand_logit", torch.float32, R * d.K),
                           _ptr(ws, "ws", torch.uint8), ws.numel(), _stream(stream)))


def dflash_pair_scores(d, x0, cand_idx, cand_logit, E, W_g, h, S, ws, stream=None):
    R, pt = d.B * d.L, _TORCH_LOGIT[d.param_dtype]
    _check(lib.dflash_pair_scores(ctypes.byref(d), _ptr(x0, "x0", torch.int32, d.B),
                                  _ptr(cand_idx, "cand_idx", torch.int32, R * d.K),
                                  _ptr(cand_logit, "cand_logit", torch.float32, R * d.K),
                                  _ptr(E, "E", pt, d.V * d.r), _ptr(W_g, "W_g", pt, d.hidden * d.r),
                                  _ptr(h, "h", pt, R * d.hidden), _ptr(S, "S", torch.float32, R * d.K * d.K),
                                  _ptr(ws, "ws", torch.uint8), ws.numel(), _stream(stream)))


def dflash_trace(d, S, cand_idx, T, seed, cycle, path_rank, draft_tok, q, stream=None):
    R = d.B * d.L
    _check(lib.dflash_trace(ctypes.byref(d), _ptr(S, "S", torch.float32, R * d.K * d.K),
                            _ptr(cand_idx, "cand_idx", torch.int32, R * d.K),
                            _ptr(T, "T", torch.float32, d.B), _ptr(seed, "seed", torch.int64, d.B),
                            ctypes.c_uint64(int(cycle) & 0xFFFFFFFFFFFFFFFF),
                            _ptr(path_rank, "path_rank", torch.int32, R),
                            _ptr(draft_tok, "draft_tok", torch.int32, R),
                            _ptr(q, "q", torch.float32, R * d.K), _stream(stream)))


def dflash_verify(d, Z, cand_idx, path_rank, q, T, seed, cycle, accept_len, out_tok, ws, stream=None):
    R = d.B * d.L
    _check(lib.dflash_verify(ctypes.byref(d),
                             _ptr(Z, "Z", _TORCH_LOGIT[d.logit_dtype], d.B * (d.L + 1) * d.V),
                             _ptr(cand_idx, "cand_idx", torch.int32, R * d.K),
                             _ptr(path_rank, "path_rank", torch.int32, R),
                             _ptr(q, "q", torch.float32, R * d.K),
                             _ptr(T, "T", torch.float32, d.B), _ptr(seed, "seed", torch.int64, d.B),
                             ctypes.c_uint64(int(cycle) & 0xFFFFFFFFFFFFFFFF),
                             _ptr(accept_len, "accept_len", torch.int32, d.B),
                             _ptr(out_tok, "out_tok", torch.int32, d.B * (d.L + 1)),
                             _ptr(ws, "ws", torch.uint8), ws.numel(), _stream(stream)))


def _cycle_call(fn, d, U, Z, x0, E, W_g, h, T, seed, cycle, accept_len, out_tok, ws,
                cand_idx, cand_logit, S, path_rank, draft_tok, q, stream):
    R, lt, pt = d.B * d.L, _TORCH_LOGIT[d.logit_dtype], _TORCH_LOGIT[d.param_dtype]
    _check(fn(
        ctypes.byref(d), _ptr(U, "U", lt, R * d.V), _ptr(Z, "Z", lt, d.B * (d.L + 1) * d.V),
        _ptr(x0, "x0", torch.int32, d.B), _ptr(E, "E", pt, d.V * d.r),
        _ptr(W_g, "W_g", pt, d.hidden * d.r), _ptr(h, "h", pt, R * d.hidden),
        _ptr(T, "T", torch.float32, d.B), _ptr(seed, "seed", torch.int64, d.B),
        ctypes.c_uint64(int(cycle) & 0xFFFFFFFFFFFFFFFF),
        _ptr(accept_len, "accept_len", torch.int32, d.B),
        _ptr(out_tok, "out_tok", torch.int32, d.B * (d.L + 1)),
        _ptr(cand_idx, "cand_idx", torch.int32, R * d.K, optional=True),
        _ptr(cand_logit, "cand_logit", torch.float32, R * d.K, optional=True),
        _ptr(S, "S", torch.float32, R * d.K * d.K, optional=True),
        _ptr(path_rank, "path_rank", torch.int32, R, optional=True),
        _ptr(draft_tok, "draft_tok", torch.int32, R, optional=True),
        _ptr(q, "q", torch.float32, R * d.K, optional=True),
        _ptr(ws, "ws", torch.uint8), ws.numel(), _stream(stream)))


def dflash_cycle(d, U, Z, x0, E, W_g, h, T, seed, cycle, accept_len, out_tok, ws,
                 cand_idx=None, cand_logit=None, S=None, path_rank=None, draft_tok=None, q=None,
                 stream=None):
    _cycle_call(lib.dflash_cycle, d, U, Z, x0, E, W_g, h, T, seed, cycle, accept_len, out_tok, ws,
                cand_idx, cand_logit, S, path_rank, draft_tok, q, stream)


def dflash_cycle_maxsum(d, U, Z, x0, E, W_g, h, T, seed, cycle, accept_len, out_tok, ws,
                        cand_idx=None, cand_logit=None, S=None, path_rank=None, draft_tok=None, q=None,
                        stream=None):
    _cycle_call(lib.dflash_cycle_maxsum, d, U, Z, x0, E, W_g, h, T, seed, cycle, accept_len, out_tok, ws,
                cand_idx, cand_logit, S, path_rank, draft_tok, q, stream)


def dflash_cycle_static(d, U, Z, x0, E, W_g, h, T, seed, cycle, accept_len, out_tok,
                        cand_idx=None, cand_logit=None, S=None, path_rank=None, draft_tok=None, q=None,
                        stream=None):
    """dflash_cycle on the library's own static scratch (no workspace argument)."""
    R, lt, pt = d.B * d.L, _TORCH_LOGIT[d.logit_dtype], _TORCH_LOGIT[d.param_dtype]
    _check(lib.dflash_cycle_static(
        ctypes.byref(d), _ptr(U, "U", lt, R * d.V), _ptr(Z, "Z", lt, d.B * (d.L + 1) * d.V),
        _ptr(x0, "x0", torch.int32, d.B), _ptr(E, "E", pt, d.V * d.r),
        _ptr(W_g, "W_g", pt, d.hidden * d.r), _ptr(h, "h", pt, R * d.hidden),
        _ptr(T, "T", torch.float32, d.B), _ptr(seed, "seed", torch.int64, d.B),
        ctypes.c_uint64(int(cycle) & 0xFFFFFFFFFFFFFFFF),
        _ptr(accept_len, "accept_len", torch.int32, d.B),
        _ptr(out_tok, "out_tok", torch.int32, d.B * (d.L + 1)),
        _ptr(cand_idx, "cand_idx", torch.int32, R * d.K, optional=True),
        _ptr(cand_logit, "cand_logit", torch.float32, R * d.K, optional=True),
        _ptr(S, "S", torch.float32, R * d.K * d.K, optional=True),
        _ptr(path_rank, "path_rank", torch.int32, R, optional=True),
        _ptr(draft_tok, "draft_tok", torch.int32, R, optional=True),
        _ptr(q, "q", torch.float32, R * d.K, optional=True), _stream(stream)))


def dflash_topk_merge(d, shard_begin, cand_idx_parts, cand_logit_parts, cand_idx, cand_logit, stream=None):
    """``shard_begin``: a Python sequence of the shards' first token indices."""
    R, n = d.B * d.L, len(shard_begin)
    begins = (ctypes.c_int32 * n)(*[int(v) for v in shard_begin])
    _check(lib.dflash_topk_merge(ctypes.byref(d), n, begins,
                                 _ptr(cand_idx_parts, "cand_idx_parts", torch.int32, n * R * d.K),
                                 _ptr(cand_logit_parts, "cand_logit_parts", torch.float32, n * R * d.K),
                                 _ptr(cand_idx, "cand_idx", torch.int32, R * d.K),
                                 _ptr(cand_logit, "cand_logit", torch.float32, R * d.K), _stream(stream)))


def _begins(shard_begin):
    n = len(shard_begin)
    return n, (ctypes.c_int32 * n)(*[int(v) for v in shard_begin])


def shard_stats_bytes(d, shard_begin):
    n, begins = _begins(shard_begin)
    out = ctypes.c_size_t(0)
    _check(lib.dflash_shard_stats_bytes(ctypes.byref(d), n, begins, ctypes.byref(out)))
    return out.value


def dflash_shard_stats(d, shard_begin, shard, Z_shard, T, stats, stream=None):
    """Statistics of shard ``shard`` (its rows ``Z_shard`` [B, L+1, width])
    into its columns of ``stats`` (a uint8 tensor of shard_stats_bytes)."""
    n, begins = _begins(shard_begin)
    hi = shard_begin[shard + 1] if shard + 1 < n else d.V
    width = int(hi) - int(shard_begin[shard])
    _check(lib.dflash_shard_stats(ctypes.byref(d), n, begins, int(shard),
                                  _ptr(Z_shard, "Z_shard", _TORCH_LOGIT[d.logit_dtype], d.B * (d.L + 1) * width),
                                  _ptr(T, "T", torch.float32, d.B), _ptr(stats, "stats", torch.uint8),
                                  _stream(stream)))


def dflash_verify_shards(d, shard_begin, Z_shards, stats, cand_idx, path_rank, q, T, seed, cycle, accept_len,
                         out_tok, stream=None):
    """``Z_shards``: one [B, L+1, width] tensor per shard."""
    n, begins = _begins(shard_begin)
    R = d.B * d.L
    zp = (ctypes.c_void_p * n)(*[_ptr(z, "Z_shards[]", _TORCH_LOGIT[d.logit_dtype]).value for z in Z_shards])
    _check(lib.dflash_verify_shards(ctypes.byref(d), n, begins, zp, _ptr(stats, "stats", torch.uint8),
                                    _ptr(cand_idx, "cand_idx", torch.int32, R * d.K),
                                    _ptr(path_rank, "path_rank", torch.int32, R),
                                    _ptr(q, "q", torch.float32, R * d.K),
                                    _ptr(T, "T", torch.float32, d.B), _ptr(seed, "seed", torch.int64, d.B),
                                    ctypes.c_uint64(int(cycle) & 0xFFFFFFFFFFFFFFFF),
                                    _ptr(accept_len, "accept_len", torch.int32, d.B),
                                    _ptr(out_tok, "out_tok", torch.int32, d.B * (d.L + 1)), _stream(stream)))


def dflash_trace_viterbi(d, S, cand_idx, path_rank, draft_tok, q, stream=None):
    R = d.B * d.L
    _check(lib.dflash_trace_viterbi(ctypes.byref(d), _ptr(S, "S", torch.float32, R * d.K * d.K),
                                    _ptr(cand_idx, "cand_idx", torch.int32, R * d.K),
                                    _ptr(path_rank, "path_rank", torch.int32, R),
                                    _ptr(draft_tok, "draft_tok", torch.int32, R),
                                    _ptr(q, "q", torch.float32, R * d.K), _stream(stream)))


def dflash_conv2tap(d, x, x0, Wt, y, stream=None):
    R, pt = d.B * d.L, _TORCH_LOGIT[d.param_dtype]
    _check(lib.dflash_conv2tap(ctypes.byref(d), _ptr(x, "x", pt, R * d.hidden), _ptr(x0, "x0", pt, d.B * d.hidden),
                               _ptr(Wt, "Wt", pt, 2 * d.hidden * d.hidden),
                               _ptr(y, "y", torch.float32, R * d.hidden), _stream(stream)))


# ------------------------------------------------------------------ rows of vocabulary logits

_ROWS_DTYPE = {torch.float32: F32, torch.bfloat16: BF16}


def rows(t):
    """A ``dflash_rows`` value describing a tensor of logits [..., V]: the
    leading dimensions must step evenly (any stride), the last one by 1."""
    if t.dtype not in _ROWS_DTYPE:
        raise TypeError(f"logits must be torch.float32 or torch.bfloat16, got {t.dtype}")
    if t.dim() < 1:
        raise ValueError("logits must have at least one dimension")
    V, R, stride = t.shape[-1], 1, None
    if V > 1 and t.stride(-1) != 1:
        raise ValueError("the elements of a logit row must be adjacent")
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * R and R != 0:
            raise ValueError("the rows of the logits must step evenly")
        R *= n
    return dflash_rows(R, V if stride is None else stride, V, _ROWS_DTYPE[t.dtype])


def rows_workspace_bytes(r):
    n = ctypes.c_size_t(0)
    _check(lib.dflash_rows_workspace_bytes(ctypes.byref(r), ctypes.byref(n)))
    return n.value


def rows_workspace(r, device="cuda"):
    """A workspace tensor large enough for any operator on these rows."""
    return torch.empty(max(rows_workspace_bytes(r), 16), dtype=torch.uint8, device=device)


def _row_tensor(t, name, r, device, stride=None):
    """Pointer and row stride of a tensor of rows ``r`` (``stride``: the row
    stride it must have)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() == 2:  # the usual case without the walk over dimensions
        (n, V), (st, step) = t.shape, t.stride()
        if (step == 1 and n == r.R and V == r.V and n > 0 and (n == 1 or stride is None or st == stride)
                and _ROWS_DTYPE.get(t.dtype) == r.dtype and t.get_device() == device.index):
            return t.data_ptr(), st if n > 1 else V
    own = rows(t)
    own_R, own_V, own_stride, own_dtype = own.R, own.V, own.stride, own.dtype
    if own_R != r.R or own_V != r.V or own_dtype != r.dtype:
        raise ValueError(f"{name} must hold {r.R} rows of {r.V} logits of the rows' dtype")
    if stride is not None and own_R > 1 and own_stride != stride:
        raise ValueError(f"{name} must have the row stride {stride}, got {own_stride}")
    if t.get_device() != device.index:
        _on(t, name, device)
    return t.data_ptr(), own_stride


def _on(t, name, device):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the rows are on {device}")


def _vec(t, name, dtype, numel, device, optional=False):
    if t is None and optional:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and (numel is None or t.numel() == numel)
            and t.get_device() == device.index and t.is_contiguous()):
        return t.data_ptr()
    _ptr(t, name, dtype, numel, optional)  # raises what is wrong with it
    _on(t, name, device)


# the current stream's handle without the stream object around it, which takes 1 us of a call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(fn, device, stream, *args):
    """Call an entry point on ``stream`` (None: the current stream of the
    tensors' device), with that device current."""
    if stream is None:
        raw = _raw_stream(device.index)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the rows are on {device}")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == device.index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status:
        _check(status)


def _groups(r, group):
    if group == 1 and type(group) is int:
        return 1, r.R
    group = operator.index(group)  # the arrays' lengths are checked against it: neither rounded nor wrapped
    if not 1 <= group < 1 << 31:
        raise ValueError(f"group must lie in [1, 2^31), got {group}")
    return group, -(-r.R // group)


def _filters(r, device, T, top_k, top_p, min_p, group):
    group, n = _groups(r, group)
    return dflash_filters(_vec(T, "T", torch.float32, n, device, True), _vec(top_k, "top_k", torch.int32, n, device, True),
                          _vec(top_p, "top_p", torch.float32, n, device, True),
                          _vec(min_p, "min_p", torch.float32, n, device, True), group)


def dflash_sample(r, Z, u, token, ws, T=None, top_k=None, top_p=None, min_p=None, group=1, prob=None, kept=None,
                  stream=None):
    """One token per row of ``Z`` (described by ``r = rows(Z)``) into
    ``token``, by the uniforms ``u`` [R] (float64) under the settings T,
    top_k, top_p, min_p (one value per ``group`` rows; None: off)."""
    dev = Z.device
    f = _filters(r, dev, T, top_k, top_p, min_p, group)
    _call(lib.dflash_sample, dev, stream, r, _row_tensor(Z, "Z", r, dev, r.stride)[0], f,
          _vec(u, "u", torch.float64, r.R, dev), _vec(token, "token", torch.int32, r.R, dev),
          _vec(prob, "prob", torch.float32, r.R, dev, True), _vec(kept, "kept", torch.int32, r.R, dev, True),
          _vec(ws, "ws", torch.uint8, None, dev), ws.numel())


def dflash_filter(r, Z, out, ws, fill=None, T=None, top_k=None, top_p=None, min_p=None, group=1, kept=None, stream=None):
    """``out`` = the rows ``Z`` with the tokens that the settings remove set
    to ``fill`` (None: the lowest finite value of Z's type); ``out`` may be
    ``Z``."""
    dev = Z.device
    if fill is None:
        fill = torch.finfo(Z.dtype).min
    f = _filters(r, dev, T, top_k, top_p, min_p, group)
    po, so = _row_tensor(out, "out", r, dev)
    _call(lib.dflash_filter, dev, stream, r, _row_tensor(Z, "Z", r, dev, r.stride)[0], f, float(fill), po, so,
          _vec(kept, "kept", torch.int32, r.R, dev, True), _vec(ws, "ws", torch.uint8, None, dev), ws.numel())


def _distill_list(r, t_idx, t_logit, device):
    if t_idx is None and t_logit is None:
        return 0, None, None
    if t_idx is None or t_logit is None or t_idx.shape != t_logit.shape:
        raise ValueError("t_idx and t_logit must be given together, with one shape [R, K]")
    K = t_idx.shape[-1]
    return K, _vec(t_idx, "t_idx", torch.int32, r.R * K, device), _vec(t_logit, "t_logit", torch.float32, r.R * K, device)


def dflash_distill(r, S, t_idx, t_logit, loss, lse, ws, tau=1.0, t_lse=None, weight=None, lse_rest=None, stream=None):
    """The loss of each student row against the teacher's listed logits
    (``t_idx``, ``t_logit`` [R, K]; both None: K = 0, ``lse`` alone)."""
    dev = S.device
    K, pi, pt = _distill_list(r, t_idx, t_logit, dev)
    _call(lib.dflash_distill, dev, stream, r, _row_tensor(S, "S", r, dev, r.stride)[0], K, float(tau), pi, pt,
          _vec(t_lse, "t_lse", torch.float64, r.R, dev, True), _vec(weight, "weight", torch.float32, r.R, dev, True),
          _vec(loss, "loss", torch.float32, r.R, dev, True), _vec(lse, "lse", torch.float64, r.R, dev),
          _vec(lse_rest, "lse_rest", torch.float64, r.R, dev, True), _vec(ws, "ws", torch.uint8, None, dev), ws.numel())


def dflash_distill_grad(r, S, t_idx, t_logit, lse, dS, tau=1.0, t_lse=None, weight=None, grad_loss=None, lse_rest=None,
                        stream=None):
    """The gradient of dflash_distill's loss with respect to ``S`` into
    ``dS`` (may be ``S``)."""
    dev = S.device
    K, pi, pt = _distill_list(r, t_idx, t_logit, dev)
    pd, sd = _row_tensor(dS, "dS", r, dev)
    _call(lib.dflash_distill_grad, dev, stream, r, _row_tensor(S, "S", r, dev, r.stride)[0], K, float(tau), pi, pt,
          _vec(t_lse, "t_lse", torch.float64, r.R, dev, True), _vec(weight, "weight", torch.float32, r.R, dev, True),
          _vec(grad_loss, "grad_loss", torch.float32, r.R, dev, True), _vec(lse, "lse", torch.float64, r.R, dev),
          _vec(lse_rest, "lse_rest", torch.float64, r.R, dev, True), pd, sd)


def _given(r, tok, values, name, device):
    if tok is None and values is None:
        return 0, None, None
    if tok is None or values is None or tok.shape != values.shape or tok.dim() < 1:
        raise ValueError(f"tok and {name} must be given together, with one shape [R, M]")
    M = tok.shape[-1] if r.R == 0 or tok.numel() != r.R else 1  # [R] as well as [R, 1]
    return M, _vec(tok, "tok", torch.int32, r.R * M, device), _vec(values, name, torch.float32, r.R * M, device)


def dflash_logprobs(r, Z, tok, logp, norm, ws, T=None, group=1, entropy=None, top_idx=None, top_logp=None, stream=None):
    """Log probabilities ``logp`` of the tokens ``tok`` [R, M] (both None: M =
    0) in the rows ``Z``, ``norm`` [R, 2] for the gradient, and, if given,
    ``entropy`` [R] and the largest alternatives ``top_idx``, ``top_logp``
    [R, N].  ``T``: a temperature per ``group`` rows (None: 1)."""
    dev = Z.device
    group, n = _groups(r, group)
    M, pk, pl = _given(r, tok, logp, "logp", dev)
    N, pi, pv = 0, None, None
    if top_idx is not None or top_logp is not None:
        if top_idx is None or top_logp is None or top_idx.shape != top_logp.shape or top_idx.dim() < 1:
            raise ValueError("top_idx and top_logp must be given together, with one shape [R, N]")
        N = top_idx.shape[-1]
        pi, pv = _vec(top_idx, "top_idx", torch.int32, r.R * N, dev), _vec(top_logp, "top_logp", torch.float32, r.R * N, dev)
    _call(lib.dflash_logprobs, dev, stream, r, _row_tensor(Z, "Z", r, dev, r.stride)[0],
          _vec(T, "T", torch.float32, n, dev, True), group, M, pk, pl, _vec(norm, "norm", torch.float32, 2 * r.R, dev),
          _vec(entropy, "entropy", torch.float32, r.R, dev, True), N, pi, pv, _vec(ws, "ws", torch.uint8, None, dev),
          ws.numel())


def dflash_logprobs_grad(r, Z, tok, grad_logp, norm, dZ, T=None, group=1, entropy=None, grad_entropy=None, stream=None):
    """The gradient of dflash_logprobs's ``logp`` and ``entropy`` with respect
    to ``Z`` into ``dZ`` (may be ``Z``)."""
    dev = Z.device
    group, n = _groups(r, group)
    M, pk, pg = _given(r, tok, grad_logp, "grad_logp", dev)
    pd, sd = _row_tensor(dZ, "dZ", r, dev)
    _call(lib.dflash_logprobs_grad, dev, stream, r, _row_tensor(Z, "Z", r, dev, r.stride)[0],
          _vec(T, "T", torch.float32, n, dev, True), group, M, pk, pg,
          _vec(grad_entropy, "grad_entropy", torch.float32, r.R, dev, True), _vec(norm, "norm", torch.float32, 2 * r.R, dev),
          _vec(entropy, "entropy", torch.float32, r.R, dev, True), pd, sd)


# ------------------------------------------------------------------ rows in 8 bits

def i8_rows(R, H, device="cuda"):
    """An int8 tensor [R, H] whose rows lie as the 8-bit operators take them:
    a multiple of 16 bytes apart, from a 16-byte aligned address on."""
    return torch.empty(R, -(-H // 16) * 16, dtype=torch.int8, device=device)[:, :H]


def _i8(t, name, rows_, H, device, stride=None):
    """Pointer and row stride of an int8 tensor of ``rows_`` rows of H."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.int8:
        raise TypeError(f"{name} must be torch.int8, got {t.dtype}")
    if t.shape != (rows_, H):
        raise ValueError(f"{name} must have the shape [{rows_}, {H}], got {list(t.shape)}")
    st, step = t.stride()
    if step != 1 and H > 1:
        raise ValueError(f"the elements of a row of {name} must be adjacent")
    if rows_ <= 1:
        st = -(-H // 16) * 16
    elif stride is not None and st != stride:
        raise ValueError(f"{name} must have the row stride {stride}, got {st}")
    if t.get_device() != device.index:
        _on(t, name, device)
    if H % 16 and rows_ and t.storage_offset() + (rows_ - 1) * st + -(-H // 16) * 16 > t.untyped_storage().nbytes():
        raise ValueError(f"the last row of {name} must lie in a multiple of 16 bytes (i8_rows makes such tensors)")
    return t.data_ptr(), st


def dflash_quant_i8(r, X, q, scale, stream=None):
    """The rows ``X`` (described by ``r = rows(X)``) as 8-bit integers ``q``
    [R, H] (``i8_rows``) with the scales ``scale`` [R]."""
    dev = X.device
    pq, sq = _i8(q, "q", r.R, r.V, dev)
    _call(lib.dflash_quant_i8, dev, stream, r, _row_tensor(X, "X", r, dev, r.stride)[0], pq, sq,
          _vec(scale, "scale", torch.float32, r.R, dev))


def linear_i8(xq, wq, y):
    """A ``dflash_linear`` value describing ``y`` [..., N] = ``xq`` [R, H] times
    ``wq`` [N, H]."""
    ry = rows(y)
    if xq.dim() != 2 or wq.dim() != 2 or xq.shape[1] != wq.shape[1]:
        raise ValueError(f"xq and wq must have the shapes [R, H] and [N, H], got {list(xq.shape)} and {list(wq.shape)}")
    if ry.R != xq.shape[0] or ry.V != wq.shape[0]:
        raise ValueError(f"y must hold {xq.shape[0]} rows of {wq.shape[0]}, got {ry.R} of {ry.V}")
    pitch = -(-xq.shape[1] // 16) * 16
    return dflash_linear(ry.R, xq.stride(0) if xq.shape[0] > 1 else pitch, wq.stride(0) if wq.shape[0] > 1 else pitch,
                         ry.stride, ry.V, xq.shape[1], ry.dtype)


def dflash_linear_i8(d, xq, xs, wq, ws, y, stream=None):
    """``y`` = the 8-bit rows ``xq`` (scales ``xs``) times ``wq`` (scales
    ``ws``), as ``d = linear_i8(xq, wq, y)`` describes them."""
    dev = xq.device
    if y.shape != (d.R, d.N) or y.stride() != (d.y_stride, 1) or _ROWS_DTYPE.get(y.dtype) != d.dtype or y.get_device() != dev.index:
        _row_tensor(y, "y", dflash_rows(d.R, d.y_stride, d.N, d.dtype), dev, d.y_stride)  # other forms of the same rows, or what is wrong
    _call(lib.dflash_linear_i8, dev, stream, d, _i8(xq, "xq", d.R, d.H, dev, d.xq_stride)[0],
          _vec(xs, "xs", torch.float32, d.R, dev), _i8(wq, "wq", d.N, d.H, dev, d.wq_stride)[0],
          _vec(ws, "ws", torch.float32, d.N, dev), y.data_ptr())


def dflash_workspace_init(ws, stream=None):
    _check(lib.dflash_workspace_init(_ptr(ws, "ws", torch.uint8), ws.numel(), _stream(stream)))


def dflash_read_probe(buf, sink, stream=None):
    _check(lib.dflash_read_probe(_ptr(buf, "buf"), buf.numel() * buf.element_size(),
                                 _ptr(sink, "sink", torch.int32), _stream(stream)))


def dflash_copy_probe(dst, src, stream=None):
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < n:
        raise ValueError("dst smaller than src")
    _check(lib.dflash_copy_probe(_ptr(dst, "dst"), _ptr(src, "src"), n, _stream(stream)))


def dflash_profile_enable(on):
    _check(lib.dflash_profile_enable(1 if on else 0))


def dflash_profile_collect(kernel):
    """(launches, total_ms) of the recorded launches of a kernel (name or id)."""
    kid = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    n, ms = ctypes.c_int64(0), ctypes.c_double(0.0)
    _check(lib.dflash_profile_collect(kid, ctypes.byref(n), ctypes.byref(ms)))
    return n.value, ms.value
