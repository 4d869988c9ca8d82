"""Python binding of the MSA C ABI (include/msa.h): argument marshalling only.

Every computation runs in libmsa.so's CUDA kernels. PyTorch supplies device memory
(outputs and workspace) and the current stream. There is no fallback: if the library
is missing or a call fails, these functions raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa.so")

MSA_OK = 0
STATUS = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARG", 2: "MSA_ERR_UNSUPPORTED", 3: "MSA_ERR_WORKSPACE",
          4: "MSA_ERR_CUDA", 5: "MSA_ERR_TIMEOUT", 6: "MSA_ERR_DEVICE_BOUNDS"}
MODE_PREFILL, MODE_DECODE = 0, 1

# Every symbol include/msa.h declares.
EXPORTS = ("msa_index_select_workspace", "msa_index_select", "msa_sparse_attn_workspace", "msa_sparse_attn",
           "msa_forward_workspace", "msa_forward", "msa_get_device_error", "msa_status_string",
           "msa_last_error_detail", "msa_profile_start", "msa_profile_stop", "msa_index_select_static",
           "msa_forward_host_device_bytes", "msa_forward_host", "msa_index_kl_workspace", "msa_index_kl",
           "msa_set_wait_limit_ns", "msa_rope", "msa_paged_append", "msa_paged_decode_workspace",
           "msa_paged_decode")


class MsaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


class MsaParams(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("hq", ctypes.c_int32), ("g", ctypes.c_int32),
                ("d", ctypes.c_int32), ("d_idx", ctypes.c_int32), ("bk", ctypes.c_int32),
                ("k", ctypes.c_int32), ("scale", ctypes.c_float), ("n", ctypes.c_int64),
                ("lmax", ctypes.c_int64), ("seqlens", ctypes.c_void_p), ("query_chunk", ctypes.c_int64),
                ("lse_out", ctypes.c_void_p)]


class MsaRopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("x_token_stride", ctypes.c_int64),
                ("x_head_stride", ctypes.c_int64), ("y_token_stride", ctypes.c_int64), ("y_head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


class MsaRopeParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("backward", ctypes.c_int32), ("scale", ctypes.c_float), ("positions_i64", ctypes.c_int32),
                ("freqs", ctypes.c_void_p), ("positions", ctypes.c_void_p)]


class MsaPagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_idx", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("k_page_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64), ("k_idx_page_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("g", ctypes.c_int32), ("d", ctypes.c_int32), ("d_idx", ctypes.c_int32)]


class MsaPagedAppendParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("rot", ctypes.c_int32), ("idx_rot", ctypes.c_int32),
                ("scale", ctypes.c_float), ("table_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("seqlens", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p), ("freqs", ctypes.c_void_p),
                ("idx_freqs", ctypes.c_void_p)]


class MsaPagedDecodeParams(ctypes.Structure):
    _fields_ = [("hq", ctypes.c_int32), ("batch", ctypes.c_int32), ("n_new", ctypes.c_int32), ("bk", ctypes.c_int32),
                ("k", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_prefix_pages", ctypes.c_int32),
                ("scale", ctypes.c_float), ("table_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("seqlens", ctypes.c_void_p), ("prefix_pages", ctypes.c_void_p)]


class MsaKernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_int32), ("total_ms", ctypes.c_double)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmsa.so and declare its signatures. Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} (run block_sparse_long_tcgen05_b200/build.py)")
    lib = ctypes.CDLL(path)
    c_i32, c_i64, c_sz, c_p, c_f = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    pp = ctypes.POINTER(MsaParams)
    sig = {
        "msa_index_select_workspace": (c_sz, [c_i64, c_i32, c_i32, c_i32, c_i32]),
        "msa_index_select": (c_i32, [c_p, c_p, c_i64, c_i32, c_i32, c_i32, c_i32, c_p, c_p, c_sz, c_p]),
        "msa_sparse_attn_workspace": (c_sz, [c_i64, c_i32, c_i32, c_i32, c_i32, c_i32]),
        "msa_sparse_attn": (c_i32, [c_p, c_p, c_p, c_p, c_i64, c_i32, c_i32, c_i32, c_i32, c_i32, c_f, c_p,
                                    c_p, c_sz, c_p]),
        "msa_forward_workspace": (c_sz, [pp]),
        "msa_forward": (c_i32, [pp, c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_sz, c_p]),
        "msa_get_device_error": (c_i32, [c_p]),
        "msa_status_string": (ctypes.c_char_p, [c_i32]),
        "msa_last_error_detail": (ctypes.c_char_p, []),
        "msa_profile_start": (c_i32, []),
        "msa_profile_stop": (c_i32, [ctypes.POINTER(MsaKernelStat), c_i32]),
        "msa_index_select_static": (c_i32, [c_p, c_p, c_i64, c_i32, c_i32, c_i32, c_i32, c_p, c_p]),
        "msa_forward_host_device_bytes": (c_sz, [pp]),
        "msa_forward_host": (c_i32, [pp, c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_sz, c_p]),
        "msa_index_kl_workspace": (c_sz, [pp]),
        "msa_index_kl": (c_i32, [pp, c_p, c_p, c_p, c_p, c_p, c_p, c_f, c_p, c_p, c_sz, c_p]),
        "msa_set_wait_limit_ns": (c_i32, [ctypes.c_uint64]),
        "msa_rope": (c_i32, [ctypes.POINTER(MsaRopeParams), ctypes.POINTER(MsaRopeTensor), c_i32, c_i64, c_p]),
        "msa_paged_append": (c_i32, [ctypes.POINTER(MsaPagedCache), ctypes.POINTER(MsaPagedAppendParams)]
                             + [ctypes.POINTER(MsaRopeTensor)] * 5 + [c_i64, c_p]),
        "msa_paged_decode_workspace": (c_sz, [ctypes.POINTER(MsaPagedCache), ctypes.POINTER(MsaPagedDecodeParams)]),
        "msa_paged_decode": (c_i32, [ctypes.POINTER(MsaPagedCache), ctypes.POINTER(MsaPagedDecodeParams), c_p, c_p, c_p,
                                     c_p, c_p, c_sz, c_p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != MSA_OK:
        lib = load_library()
        raise MsaError(status, lib.msa_last_error_detail().decode())


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _bf16(t: torch.Tensor, name: str) -> int:
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    return _ptr(t)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(nbytes: int, device, workspace: torch.Tensor | None) -> torch.Tensor:
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def msa_index_select_workspace(n: int, g: int, d_idx: int, k: int, bk: int = 128) -> int:
    return load_library().msa_index_select_workspace(n, g, d_idx, bk, k)


def msa_index_select(q_idx: torch.Tensor, k_idx: torch.Tensor, k: int, bk: int = 128,
                     block_ids: torch.Tensor | None = None, workspace: torch.Tensor | None = None
                     ) -> torch.Tensor:
    """Index Branch: q_idx, k_idx [N, G, d_idx] bf16 -> block_ids [N, G, k] int32."""
    lib = load_library()
    N, G, d_idx = q_idx.shape
    if tuple(k_idx.shape) != (N, G, d_idx):
        raise ValueError("k_idx shape must equal q_idx shape")
    if block_ids is None:
        block_ids = torch.empty(N, G, k, dtype=torch.int32, device=q_idx.device)
    need = lib.msa_index_select_workspace(N, G, d_idx, bk, k)
    ws = _workspace(need, q_idx.device, workspace)
    _check(lib.msa_index_select(_bf16(q_idx, "q_idx"), _bf16(k_idx, "k_idx"), N, G, d_idx, bk, k,
                                _ptr(block_ids), _ptr(ws), ws.numel(), _stream(q_idx.device)))
    return block_ids


def msa_sparse_attn_workspace(n: int, hq: int, g: int, d: int, k: int, bk: int = 128) -> int:
    return load_library().msa_sparse_attn_workspace(n, hq, g, d, bk, k)


def msa_sparse_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_ids: torch.Tensor,
                    bk: int = 128, scale: float = 0.0, o: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Main Branch (KV-outer): q [N,Hq,d], k/v [N,G,d], block_ids [N,G,k] -> o [N,Hq,d]."""
    lib = load_library()
    N, Hq, d = q.shape
    G = k.shape[1]
    topk = block_ids.shape[2]
    if block_ids.dtype != torch.int32:
        raise ValueError("block_ids must be int32")
    if o is None:
        o = torch.empty_like(q)
    need = lib.msa_sparse_attn_workspace(N, Hq, G, d, bk, topk)
    ws = _workspace(need, q.device, workspace)
    _check(lib.msa_sparse_attn(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _ptr(block_ids), N, Hq, G, d, bk,
                               topk, scale, _ptr(o), _ptr(ws), ws.numel(), _stream(q.device)))
    return o


def prefill_params(N: int, Hq: int, G: int, d: int, d_idx: int, k: int, bk: int = 128, scale: float = 0.0,
                   query_chunk: int = 0) -> MsaParams:
    return MsaParams(mode=MODE_PREFILL, hq=Hq, g=G, d=d, d_idx=d_idx, bk=bk, k=k, scale=scale, n=N, lmax=0,
                     seqlens=None, query_chunk=query_chunk)


def decode_params(B: int, Lmax: int, seqlens: torch.Tensor, Hq: int, G: int, d: int, d_idx: int, k: int,
                  bk: int = 128, scale: float = 0.0) -> MsaParams:
    return MsaParams(mode=MODE_DECODE, hq=Hq, g=G, d=d, d_idx=d_idx, bk=bk, k=k, scale=scale, n=B, lmax=Lmax,
                     seqlens=_ptr(seqlens), query_chunk=0)


def msa_forward_workspace(p: MsaParams) -> int:
    return load_library().msa_forward_workspace(ctypes.byref(p))


def msa_forward(p: MsaParams, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_idx: torch.Tensor,
                k_idx: torch.Tensor, o: torch.Tensor | None = None, block_ids: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Both branches (prefill or decode, per p.mode); returns o. See include/msa.h."""
    lib = load_library()
    if o is None:
        o = torch.empty_like(q)
    need = lib.msa_forward_workspace(ctypes.byref(p))
    if need == 0:
        raise MsaError(1, "unsupported or invalid msa_params")
    ws = _workspace(need, q.device, workspace)
    _check(lib.msa_forward(ctypes.byref(p), _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _bf16(q_idx, "q_idx"),
                           _bf16(k_idx, "k_idx"), _ptr(block_ids), _ptr(o), _ptr(ws), ws.numel(),
                           _stream(q.device)))
    return o


def _host(t: torch.Tensor | None, name: str, dtype=torch.bfloat16) -> int | None:
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} host tensor")
    return t.data_ptr()


def msa_forward_host_device_bytes(p: MsaParams) -> int:
    return load_library().msa_forward_host_device_bytes(ctypes.byref(p))


def forward_host(p: MsaParams, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_idx: torch.Tensor,
                 k_idx: torch.Tensor, o: torch.Tensor, block_ids: torch.Tensor | None = None,
                 device_buf: torch.Tensor | None = None, device=None) -> torch.Tensor:
    """Prefill with host tensors in and out (page-locked for the copies to overlap the
    kernels); see msa_forward_host in include/msa.h. Enqueued on the current stream of
    `device`: o (and block_ids) are complete once that stream is."""
    lib = load_library()
    device = torch.device("cuda") if device is None else torch.device(device)
    need = lib.msa_forward_host_device_bytes(ctypes.byref(p))
    if need == 0:
        raise MsaError(1, "unsupported or invalid msa_params for msa_forward_host")
    buf = _workspace(need, device, device_buf)
    _check(lib.msa_forward_host(ctypes.byref(p), _host(q, "q"), _host(k, "k"), _host(v, "v"), _host(q_idx, "q_idx"),
                                _host(k_idx, "k_idx"), _host(block_ids, "block_ids", torch.int32), _host(o, "o"),
                                _ptr(buf), buf.numel() * buf.element_size(), _stream(device)))
    return o


def prefill(q, k, v, q_idx, k_idx, topk: int, bk: int = 128, scale: float = 0.0, query_chunk: int = 0,
            block_ids: torch.Tensor | None = None, o: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, lse: torch.Tensor | None = None) -> torch.Tensor:
    """Both branches of one sequence; with `lse` (float32 [N, Hq]) also the log-sum-exp of
    every (query, head)'s logits over its selected tokens, as index_kl takes it."""
    N, Hq, d = q.shape
    G, d_idx = q_idx.shape[1], q_idx.shape[2]
    p = prefill_params(N, Hq, G, d, d_idx, topk, bk, scale, query_chunk)
    if lse is not None:
        if lse.dtype != torch.float32 or tuple(lse.shape) != (N, Hq):
            raise ValueError("lse must be float32 [N, Hq]")
        p.lse_out = _ptr(lse)
    return msa_forward(p, q, k, v, q_idx, k_idx, o=o, block_ids=block_ids, workspace=workspace)


def index_kl(q, k, q_idx, k_idx, block_ids: torch.Tensor, lse: torch.Tensor, bk: int = 128, scale: float = 0.0,
             idx_scale: float = 0.0, query_chunk: int = 0, kl: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Index-branch KL loss forward (msa_index_kl): KL(P_main || P_idx) per (query, group) ->
    float32 [N, G]; block_ids and lse as the prefill forward produced them."""
    lib = load_library()
    N, Hq, d = q.shape
    G, d_idx = q_idx.shape[1], q_idx.shape[2]
    topk = block_ids.shape[2]
    if block_ids.dtype != torch.int32 or lse.dtype != torch.float32:
        raise ValueError("block_ids must be int32 and lse float32")
    p = prefill_params(N, Hq, G, d, d_idx, topk, bk, scale, query_chunk)
    if kl is None:
        kl = torch.empty(N, G, dtype=torch.float32, device=q.device)
    need = lib.msa_index_kl_workspace(ctypes.byref(p))
    if need == 0:
        raise MsaError(2, "unsupported shape for msa_index_kl")
    ws = _workspace(need, q.device, workspace)
    _check(lib.msa_index_kl(ctypes.byref(p), _bf16(q, "q"), _bf16(k, "k"), _bf16(q_idx, "q_idx"),
                            _bf16(k_idx, "k_idx"), _ptr(block_ids), _ptr(lse), idx_scale, _ptr(kl), _ptr(ws),
                            ws.numel(), _stream(q.device)))
    return kl


def decode(q, k_cache, v_cache, q_idx, k_idx_cache, seqlens, topk: int, bk: int = 128, scale: float = 0.0,
           block_ids: torch.Tensor | None = None, o: torch.Tensor | None = None,
           workspace: torch.Tensor | None = None) -> torch.Tensor:
    B, Hq, d = q.shape
    Lmax, G = k_cache.shape[1], k_cache.shape[2]
    d_idx = q_idx.shape[2]
    if seqlens.dtype != torch.int32:
        raise ValueError("seqlens must be int32")
    p = decode_params(B, Lmax, seqlens, Hq, G, d, d_idx, topk, bk, scale)
    return msa_forward(p, q, k_cache, v_cache, q_idx, k_idx_cache, o=o, block_ids=block_ids,
                       workspace=workspace)


# ------------------------------------------------------------------------------------ serving
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"
                     ) -> tuple[torch.Tensor, float]:
    """(freqs, scale) for rope and paged_append: radians a position of each of the rot / 2 pairs
    (float64), and what cos and sin are multiplied with.

    scaling, for contexts `factor` times as long as the trained ones: "none"; "linear", positions
    divided by factor; "ntk", the base raised so that the slowest pair is stretched by factor;
    "yarn", pairs that turn more than beta_fast times in trained_length kept, those that turn less
    than beta_slow times stretched by factor, a linear ramp over the pairs between, and cos and sin
    scaled by 0.1 ln(factor) + 1."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be a positive even number")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    scale = 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if not beta_fast > beta_slow > 0.0 or trained_length < 1:
            raise ValueError("yarn wants beta_fast > beta_slow > 0 and a trained length")
        pair = lambda turns: rot * math.log(trained_length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo = max(math.floor(pair(beta_fast)), 0)
        hi = min(math.ceil(pair(beta_slow)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r} (none, linear, ntk, yarn)")
    return f.to(device), scale


# The serving calls are made once a layer and step, on tensors that a GPU is done with in a few
# microseconds: their parameter structures are packed directly (the layouts of the ctypes
# structures above), and each tensor is looked at once.
_PACK_TENSOR = struct.Struct("@PPqqqqii").pack
_PACK_ROPE = struct.Struct("@iiiifiPP").pack
_PACK_APPEND = struct.Struct("@iiiiiifqPPPPP").pack
_PACK_DECODE = struct.Struct("@iiiiiiifqPPP").pack
_fast = None
_forward_ad = torch.autograd.forward_ad
_current_device = getattr(torch._C, "_cuda_getDevice", None)          # absent in builds without CUDA
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _serving():
    """The serving entry points, taking packed structures."""
    global _fast
    if _fast is None:
        lib = load_library()
        c_i32, c_i64, c_sz, c_p = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
        out = []
        for name, res, args in (("msa_rope", c_i32, [c_p, c_p, c_i32, c_i64, c_p]),
                                ("msa_paged_append", c_i32, [c_p] * 7 + [c_i64, c_p]),
                                ("msa_paged_decode_workspace", c_sz, [c_p, c_p]),
                                ("msa_paged_decode", c_i32, [c_p] * 7 + [c_sz, c_p])):
            fn = lib[name]
            fn.restype, fn.argtypes = res, args
            out.append(fn)
        _fast = out
    return _fast


def _no_tangent(*tensors: torch.Tensor | None) -> None:
    if any(t is not None and _forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise ValueError("the result would carry no tangent; call this on the primals (the rotation is linear: the tangent's "
                         "rotation is the result's tangent)")


def _dual() -> bool:
    """Whether tensors may carry tangents: a dual_level is open."""
    return getattr(_forward_ad, "_current_level", 0) >= 0


def _heads(x: torch.Tensor, name: str, n: int, index: int, dtype, y: torch.Tensor | None = None, y_dtype=None) -> bytes:
    """Checks a tensor of heads (and the one its result goes to) and packs its msa_rope_tensor."""
    shape, sx = x.shape, x.stride()
    if len(shape) != 3 or shape[0] != n:
        raise ValueError(f"{name} must be [{n}, heads, dim]")
    if x.dtype is not dtype or x.get_device() != index:
        raise ValueError(f"{name} must be {dtype} on device {index}")
    if sx[2] != 1 and shape[2] != 1:
        raise ValueError(f"{name}: the elements of a head must lie side by side")
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: the result would carry no gradient; call this under torch.no_grad() "
                         "(rope(..., backward=True) takes gradients back)")
    if y is None:
        return _PACK_TENSOR(x.data_ptr(), 0, sx[0], sx[1], 0, 0, shape[1], shape[2])
    sy = y.stride()
    if y.dtype is not y_dtype or y.shape != shape or y.get_device() != index or (sy[2] != 1 and shape[2] != 1):
        raise ValueError(f"{name}: its result must be {y_dtype} {list(shape)} on device {index}, heads' elements side by side")
    return _PACK_TENSOR(x.data_ptr(), y.data_ptr(), sx[0], sx[1], sy[0], sy[1], shape[1], shape[2])


def _small(t: torch.Tensor, name: str, index: int, dtype, shape) -> int:
    """Address of a contiguous tensor of known shape, type and device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} on device {index}")
    return t.data_ptr()


def _freqs(t: torch.Tensor, name: str, index: int) -> tuple[int, int]:
    shape = t.shape
    if t.dtype is not torch.float64 or len(shape) != 1 or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float64 [rot / 2] on device {index}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: frequencies get no gradient here; detach them")
    return t.data_ptr(), 2 * shape[0]


def _launch(index: int, fn, *args) -> None:
    """fn(*args, stream) on the tensors' device, whichever device is the current one."""
    if index == _current_device():
        st = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _current_stream(index))
    if st != MSA_OK:
        _check(st)


def rope(x, positions: torch.Tensor, freqs: torch.Tensor, interleaved: bool = False, scale: float = 1.0,
         backward: bool = False, out=None):
    """Rotary positions (msa_rope): x [N, heads, dim], or up to four such tensors of the same N
    tokens (other head counts and dims), bf16, fp16 or fp32; positions [N] int32 or int64; freqs
    float64 [rot / 2] (rope_frequencies). The first rot elements of every head are rotated, in halves
    or interleaved pairs, the rest copied. backward=True: the gradient of the result to that of x
    (same freqs, positions and scale). out: where the results go (x itself: in place)."""
    many = isinstance(x, (tuple, list))
    xs = tuple(x) if many else (x,)
    if not 1 <= len(xs) <= 4:
        raise ValueError("rope takes one to four tensors")
    dtype, index, n = xs[0].dtype, xs[0].get_device(), xs[0].shape[0]
    if index < 0:
        raise ValueError("expected CUDA tensors")
    if dtype not in _DTYPES:
        raise ValueError(f"rope takes bfloat16, float16 and float32, not {dtype}")
    if _dual():
        _no_tangent(freqs, *xs)
    if positions.dtype != torch.int64 and positions.dtype != torch.int32:
        raise ValueError("positions must be int32 or int64")
    if out is None:
        outs = tuple(torch.empty(t.shape, dtype=dtype, device=t.device) for t in xs)
    else:
        outs = tuple(out) if many else (out,)
        if len(outs) != len(xs):
            raise ValueError("out must match x")
    f, rot = _freqs(freqs, "freqs", index)
    p = _PACK_ROPE(_DTYPES[dtype], rot, bool(interleaved), bool(backward), scale, positions.dtype == torch.int64, f,
                   _small(positions, "positions", index, positions.dtype, (n,)))
    tensors = b"".join([_heads(a, "x", n, index, dtype, b, dtype) for a, b in zip(xs, outs)])
    _launch(index, _serving()[0], p, tensors, len(xs), n)
    return outs if many else outs[0]


class PagedCache:
    """Handle of a paged cache: k_pages, v_pages [pages, page_size, G, d] and k_idx_pages
    [pages, page_size, G, d_idx], bf16 (see msa_paged_cache in include/msa.h). Pages may lie apart
    (slices of a larger tensor); a page itself is contiguous. The handle keeps the tensors alive."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_idx_pages: torch.Tensor):
        load_library()
        if k_pages.dim() != 4 or k_idx_pages.dim() != 4 or v_pages.shape != k_pages.shape \
                or k_idx_pages.shape[:3] != k_pages.shape[:3]:
            raise ValueError("pages must be [pages, page_size, G, dim] of one geometry")
        if 0 in k_pages.shape or 0 in k_idx_pages.shape:
            raise ValueError("a cache has at least one page, and pages at least one row")
        self.device = k_pages.device
        if self.device.type != "cuda":
            raise ValueError("expected CUDA tensors")
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages"), (k_idx_pages, "k_idx_pages")):
            if t.dtype != torch.bfloat16 or t.device != self.device:
                raise ValueError(f"{name} must be bfloat16 on {self.device}")
            if not t[0].is_contiguous():
                raise ValueError(f"{name}: a page must be contiguous")
        self.k_pages, self.v_pages, self.k_idx_pages = k_pages, v_pages, k_idx_pages
        self.num_pages, self.page_size, self.G, self.d = k_pages.shape
        self.d_idx = k_idx_pages.shape[3]
        stride = lambda t: t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t[0].numel())  # noqa: E731
        self.index = self.device.index
        self.c = MsaPagedCache(k_pages.data_ptr(), v_pages.data_ptr(), k_idx_pages.data_ptr(), self.num_pages,
                               stride(k_pages), stride(v_pages), stride(k_idx_pages), self.page_size, self.G, self.d,
                               self.d_idx)
        self.address = ctypes.addressof(self.c)
        self.workspaces = {}   # bytes that paged_decode needs, by the call's sizes


def _table(page_table: torch.Tensor, index: int, batch: int) -> tuple[int, int, int]:
    """(address, columns, stride of rows) of a page table."""
    shape, st = page_table.shape, page_table.stride()
    if page_table.dtype != torch.int32 or len(shape) != 2 or page_table.get_device() != index or shape[0] != batch \
            or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"page_table must be int32 [{batch}, pages] on device {index}, its rows contiguous")
    return page_table.data_ptr(), shape[1], max(st[0], shape[1]) if batch == 1 else st[0]


def paged_append(cache: PagedCache, page_table: torch.Tensor, seqlens: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 k_idx: torch.Tensor, cu_seqlens: torch.Tensor | None = None, freqs: torch.Tensor | None = None,
                 idx_freqs: torch.Tensor | None = None, rotate_index: bool = True, interleaved: bool = False,
                 rope_scale: float = 1.0, q: torch.Tensor | None = None, q_idx: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None, q_idx_out: torch.Tensor | None = None
                 ) -> tuple[torch.Tensor | None, torch.Tensor | None]:
    """Writes new tokens into the cache (msa_paged_append): k, v [N, G, d], k_idx [N, G, d_idx] in bf16,
    fp16 or fp32, keys rotated by their positions on the way (freqs given; index keys by idx_freqs, or by
    freqs, unless rotate_index is False). seqlens [B] int32 counts the new tokens; cu_seqlens [B + 1] int32
    says which rows are whose (None: N / B each; rows of positions below 0, as all of an empty sequence of a
    padded batch, then have no token); rows behind cu_seqlens[B] are padding. q [N, Hq, d] and
    q_idx [N, G, d_idx] are rotated in the same launch into q_out / q_idx_out (bf16; allocated if None,
    padding rows then undefined). Returns (q_out, q_idx_out)."""
    index, dtype, n, batch = cache.index, k.dtype, k.shape[0], seqlens.shape[0]
    if dtype not in _DTYPES:
        raise ValueError(f"paged_append takes bfloat16, float16 and float32, not {dtype}")
    if _dual():
        _no_tangent(k, v, k_idx, q, q_idx, freqs, idx_freqs)
    table, columns, stride = _table(page_table, index, batch)
    if (q is None and q_out is not None) or (q_idx is None and q_idx_out is not None):
        raise ValueError("q_out or q_idx_out without its input")
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if q_idx is not None and q_idx_out is None:
        q_idx_out = torch.empty(q_idx.shape, dtype=torch.bfloat16, device=q_idx.device)
    f, rot = (0, 0) if freqs is None else _freqs(freqs, "freqs", index)
    fi, irot = (f, rot) if rotate_index else (0, 0)
    if idx_freqs is not None:
        fi, irot = _freqs(idx_freqs, "idx_freqs", index)
    cu = 0 if cu_seqlens is None else _small(cu_seqlens, "cu_seqlens", index, torch.int32, (batch + 1,))
    p = _PACK_APPEND(_DTYPES[dtype], batch, columns, bool(interleaved), rot, irot, rope_scale, stride, table,
                     _small(seqlens, "seqlens", index, torch.int32, (batch,)), cu, f, fi)
    _launch(index, _serving()[1], cache.address, p, _heads(k, "k", n, index, dtype), _heads(v, "v", n, index, dtype),
            _heads(k_idx, "k_idx", n, index, dtype), None if q is None else _heads(q, "q", n, index, dtype, q_out, torch.bfloat16),
            None if q_idx is None else _heads(q_idx, "q_idx", n, index, dtype, q_idx_out, torch.bfloat16), n)
    return q_out, q_idx_out


def paged_decode_workspace(cache: PagedCache, batch: int, max_pages: int, hq: int, topk: int, bk: int = 128,
                           n_new: int = 1) -> int:
    """Bytes of workspace of paged_decode for page tables of max_pages columns."""
    p = MsaPagedDecodeParams(hq, batch, n_new, bk, topk, max_pages, 0, 0.0, max_pages, None, None, None)
    need = load_library().msa_paged_decode_workspace(cache.c, p)
    if need == 0:   # the call itself, refused for the same sizes, says which kind of refusal it is
        _check(load_library().msa_paged_decode(cache.c, p, None, None, None, None, None, 0, None))
    return need


def paged_decode(cache: PagedCache, page_table: torch.Tensor, seqlens: torch.Tensor, q: torch.Tensor, q_idx: torch.Tensor,
                 topk: int, bk: int = 128, scale: float = 0.0, prefix_pages: torch.Tensor | None = None,
                 block_ids: torch.Tensor | None = None, o: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Decode over a paged cache (msa_paged_decode). q [B, Hq, d] and q_idx [B, G, d_idx] are the newest
    token's of every sequence, or with a second dimension of 1 to 8 the newest tokens'; their keys are
    in the cache already (paged_append). page_table [B, pages], seqlens [B] int32. prefix_pages int32
    [n]: the first n pages of every sequence, where the batch shares a prefix; it is scored once for all.
    block_ids int32 [..., G, topk] takes the selection. Returns o, shaped as q; rows without a token are 0."""
    index, shape = cache.index, q.shape
    if len(shape) not in (3, 4) or shape[-1] != cache.d:
        raise ValueError(f"q must be [B, Hq, {cache.d}] or [B, tokens, Hq, {cache.d}]")
    batch, hq = shape[0], shape[-2]
    S = 1 if len(shape) == 3 else shape[1]
    kp, vp = cache.k_pages, cache.v_pages
    if torch.is_grad_enabled() and (q.requires_grad or q_idx.requires_grad or kp.requires_grad or vp.requires_grad):
        raise ValueError("the result would carry no gradient; call this under torch.no_grad()")
    if _dual():
        _no_tangent(q, q_idx, kp, vp)
    table, columns, stride = _table(page_table, index, batch)
    lens = _small(seqlens, "seqlens", index, torch.int32, (batch,))
    bf16, lead = torch.bfloat16, shape[:-2]
    qp = _small(q, "q", index, bf16, shape)
    qip = _small(q_idx, "q_idx", index, bf16, lead + (cache.G, cache.d_idx))
    idp = None if block_ids is None else _small(block_ids, "block_ids", index, torch.int32, lead + (cache.G, topk))
    if o is None:
        o = torch.empty_like(q)
    op = _small(o, "o", index, bf16, shape)
    pp, shared = 0, 0
    if prefix_pages is not None:
        shared = prefix_pages.shape[0]
        pp = _small(prefix_pages, "prefix_pages", index, torch.int32, (shared,))
    p = _PACK_DECODE(hq, batch, S, bk, topk, columns, shared, scale, stride, table, lens, pp)
    fns = _serving()
    sizes = (batch, S, hq, columns, topk, bk)
    need = cache.workspaces.get(sizes)
    if need is None:
        need = fns[2](cache.address, p)
        if need == 0:   # refused: by the call itself with its status
            _check(fns[3](cache.address, p, qp, qip, idp, op, None, 0, None))
        cache.workspaces[sizes] = need
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on device {index}")
    _launch(index, fns[3], cache.address, p, qp, qip, idp, op, workspace.data_ptr(), workspace.nbytes)
    return o


def msa_get_device_error(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device error status."""
    lib = load_library()
    dev = device if device is not None else torch.cuda.current_device()
    return lib.msa_get_device_error(_stream(dev))


def check_device_error(device=None) -> None:
    st = msa_get_device_error(device)
    if st != MSA_OK:
        raise MsaError(st, load_library().msa_last_error_detail().decode())


def set_wait_limit_ns(ns: int) -> None:
    """Time limit of the kernels' gating waits on the current device (0: the 2 s default)."""
    _check(load_library().msa_set_wait_limit_ns(int(ns)))


def msa_profile_start() -> None:
    """Start recording CUDA events around every launch of the library."""
    _check(load_library().msa_profile_start())


def msa_profile_stop() -> dict:
    """Stop recording; {kernel name: (launches, total device ms)} since msa_profile_start."""
    lib = load_library()
    buf = (MsaKernelStat * 32)()
    n = lib.msa_profile_stop(buf, 32)
    if n < 0:
        raise MsaError(4, "profile events failed")
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms)) for i in range(min(n, 32))}
