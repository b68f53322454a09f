"""Ternary-weight linear layer for MI355X (gfx950): thin binding over libternary.so.

    y = x @ (q * s)^T,  q in {-1, 0, +1} packed 4 codes per byte (2 bits each,
    00 -> 0, 01 -> +1, 10 -> -1, 11 -> 0, first weight in the lowest bits),
    s an fp16 scale per output channel or per group of 32, 64, 128 or 256
    consecutive K weights.

The format is the one stated on trdm.cn "三元量化模型接入vLLM：从逆向加载到Kernel优化的完整实战"
(§3.1) and m.nxbn.cn/news/169761 (§2.2); the layer's interface (x, weight,
scale) -> y follows m.nxbn.cn/news/169761 §5.2.

Everything here only marshals arguments: shapes, dtypes and the current HIP
stream are read from torch tensors and passed to the C ABI of
``include/ternary.h``.  Every step of the computation runs in the HIP kernels.
If the library is not built this module raises on first use; there is no
CPU fallback.
"""

from __future__ import annotations

import ctypes
import functools
from pathlib import Path
from typing import NamedTuple

import torch

__all__ = [
    "TernaryError", "lib", "pack", "unpack", "linear", "linear_batch", "select_path", "gemv_max_m",
    "PATHS", "BF16", "FP16", "abi_version", "shutdown", "LIB_PATH", "probe_read", "probe_copy",
    "probe_mfma", "probe_mfma_flops", "probe_lib", "PROBE_LIB_PATH", "quantize",
    "linear_batch_noalloc", "tile", "untile",
    "tiled_bytes", "LAYOUTS", "fp8_quantize", "fp8_linear", "route", "Routing", "linear_experts",
    "combine", "sort_slots", "dispatch", "dispatch_backward", "combine_backward", "linear_adapters",
    "linear_adapters_backward",
]

LIB_PATH = Path(__file__).resolve().parent / "libternary.so"
# Measurement probes (include/ternary_probe.h) live in a library of their own.
PROBE_LIB_PATH = Path(__file__).resolve().parent / "libternary_probe.so"

BF16, FP16 = 0, 1
PATHS = {"auto": 0, "gemv": 1, "gemm": 2, "simple": 3, "gemv_f4": 4, "gemv_b16": 5,
         "gemv_valu": 6, "few": 7, "gemm_zskip": 8}
LAYOUTS = {"rows": 0, "tiled": 1}

# Every symbol include/ternary.h declares.
EXPORTS = (
    "ternary_pack", "ternary_unpack", "ternary_linear", "ternary_linear_ex",
    "ternary_linear_batch", "ternary_select_path", "ternary_gemv_max_m",
    "ternary_status_string", "ternary_abi_version", "ternary_shutdown", "ternary_quantize",
    "ternary_linear_batch_noalloc", "ternary_tile", "ternary_untile", "ternary_tiled_bytes",
    "ternary_linear_tiled", "ternary_fp8_quantize", "ternary_fp8_linear", "ternary_route",
    "ternary_route_workspace", "ternary_linear_experts", "ternary_combine",
    "ternary_sort_slots", "ternary_sort_slots_workspace", "ternary_dispatch",
    "ternary_dispatch_backward", "ternary_combine_backward", "ternary_linear_adapters",
    "ternary_linear_adapters_workspace", "ternary_linear_adapters_backward",
    "ternary_linear_adapters_backward_workspace",
)
# Every symbol include/ternary_probe.h declares (measurement probes).
PROBE_EXPORTS = ("ternary_probe_read", "ternary_probe_read_nt", "ternary_probe_copy",
                 "ternary_probe_mfma")
MAX_BATCH = 8
PROBE_THREADS = 256


class Problem(ctypes.Structure):
    """ternary_problem of include/ternary.h."""
    _fields_ = [("x", ctypes.c_void_p), ("packed", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("M", ctypes.c_int64), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("group_size", ctypes.c_int64),
                ("layout", ctypes.c_int64)]

_lib = None


class TernaryError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not LIB_PATH.exists():
        raise RuntimeError(
            f"{LIB_PATH} is missing: build the HIP library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(str(LIB_PATH))
    i64, p, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    L.ternary_pack.argtypes = [p, i64, i64, p, p, p]
    L.ternary_unpack.argtypes = [p, i64, i64, p, p]
    L.ternary_linear.argtypes = [p, i32, i64, i64, i64, p, p, i64, p, p]
    L.ternary_linear_ex.argtypes = [p, i32, i64, i64, i64, p, p, i64, p, i32, p]
    L.ternary_linear_tiled.argtypes = [p, i32, i64, i64, i64, p, p, i64, p, i32, p]
    L.ternary_tile.argtypes = [p, i64, i64, p, p]
    L.ternary_untile.argtypes = [p, i64, i64, p, p]
    L.ternary_tiled_bytes.argtypes = [i64, i64]
    L.ternary_tiled_bytes.restype = i64
    L.ternary_linear_batch.argtypes = [p, i32, i32, p]
    L.ternary_linear_batch_noalloc.argtypes = [p, i32, i32, p]
    L.ternary_quantize.argtypes = [p, i32, i64, i64, i64, p, p, p]
    f32 = ctypes.c_float
    L.ternary_fp8_quantize.argtypes = [p, i32, i64, i64, i64, i32, i32, p, p, p]
    L.ternary_fp8_linear.argtypes = [p, p, p, p, i64, i64, i64, p, i32, p]
    L.ternary_route.argtypes = [p, i32, i64, i64, p, i32, i32, i32, i32, i32, f32, p, p, p, p, p, p, p]
    L.ternary_route_workspace.argtypes = [i64, i64]
    L.ternary_route_workspace.restype = i64
    L.ternary_linear_experts.argtypes = [p, p, i64, p, p, i64, i64, i64, i64, p, p, i64, i32, i32, p,
                                         i32, p]
    L.ternary_combine.argtypes = [p, i32, i64, i64, p, p, i64, i32, p, p, p]
    L.ternary_sort_slots.argtypes = [p, i64, i32, i64, p, p, p, p, p, p]
    L.ternary_dispatch.argtypes = [p, i32, i64, i64, p, p, i32, i64, p, p]
    L.ternary_dispatch_backward.argtypes = [p, i32, i64, i64, p, p, i64, i32, p, p, p, p, p]
    L.ternary_combine_backward.argtypes = [p, p, i32, i64, i64, p, p, i64, i32, p, p, p]
    L.ternary_linear_adapters.argtypes = [p, i32, i64, i64, i64, i64, p, p, i64, p, p, p, p, p, p, p, p, p]
    L.ternary_linear_adapters_backward.argtypes = [p, p, p, i32, i64, i64, i64, i64, p, p, i64, p, p, p, p,
                                                   p, p, p, p, p, p]
    L.ternary_sort_slots_workspace.argtypes = [i64, i32, i64]
    for nm in ("ternary_linear_adapters_workspace", "ternary_linear_adapters_backward_workspace"):
        getattr(L, nm).argtypes = [i64, i64, i64, i64, i64]
    for nm in ("ternary_sort_slots_workspace", "ternary_linear_adapters_workspace",
               "ternary_linear_adapters_backward_workspace"):
        getattr(L, nm).restype = i64
    L.ternary_select_path.argtypes = [i64, i64, i64, i64]
    L.ternary_status_string.argtypes = [i32]
    L.ternary_status_string.restype = ctypes.c_char_p
    for nm in ("ternary_pack", "ternary_unpack", "ternary_linear", "ternary_linear_ex",
               "ternary_linear_batch", "ternary_select_path", "ternary_gemv_max_m",
               "ternary_abi_version", "ternary_shutdown", "ternary_quantize",
               "ternary_linear_batch_noalloc", "ternary_linear_tiled", "ternary_tile",
               "ternary_untile", "ternary_fp8_quantize", "ternary_fp8_linear", "ternary_route",
               "ternary_linear_experts", "ternary_combine", "ternary_sort_slots", "ternary_dispatch",
               "ternary_dispatch_backward", "ternary_combine_backward", "ternary_linear_adapters",
               "ternary_linear_adapters_backward"):
        getattr(L, nm).restype = i32
    _lib = L
    return L


_probe_lib = None


def probe_lib() -> ctypes.CDLL:
    """The measurement-probe library (bench and its tests only); raises if it
    has not been built."""
    global _probe_lib
    if _probe_lib is not None:
        return _probe_lib
    if not PROBE_LIB_PATH.exists():
        raise RuntimeError(f"{PROBE_LIB_PATH} is missing: build the HIP libraries first")
    L = ctypes.CDLL(str(PROBE_LIB_PATH))
    i64, p, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    L.ternary_probe_read.argtypes = [p, i64, i32, p, p]
    L.ternary_probe_read_nt.argtypes = [p, i64, i32, p, p]
    L.ternary_probe_copy.argtypes = [p, p, i64, i32, p]
    L.ternary_probe_mfma.argtypes = [i32, i32, p, p]
    for nm in PROBE_EXPORTS:
        getattr(L, nm).restype = i32
    _probe_lib = L
    return L


def status_string(status: int) -> str:
    return lib().ternary_status_string(int(status)).decode()


def abi_version() -> int:
    return int(lib().ternary_abi_version())


def shutdown() -> None:
    """Free the library's per-stream workspaces (ternary_shutdown)."""
    _check(int(lib().ternary_shutdown()), "ternary_shutdown")


def gemv_max_m() -> int:
    return int(lib().ternary_gemv_max_m())


def select_path(M: int, N: int, K: int, group_size: int) -> str:
    r = int(lib().ternary_select_path(M, N, K, group_size))
    if r < 0:
        raise TernaryError(r, "ternary_select_path")
    return {v: k for k, v in PATHS.items()}[r]


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor):
    """The current HIP stream of t's device (what torch would launch on)."""
    if _raw_stream is not None:
        return _raw_stream(t.device.index)
    return torch.cuda.current_stream(t.device).cuda_stream


def _check(status: int, where: str):
    if status != 0:
        raise TernaryError(status, where)


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def pack(q: torch.Tensor, invalid_count: torch.Tensor | None = None) -> torch.Tensor:
    """int8 [N, K] in {-1,0,1} -> uint8 [N, K/4].  Values outside {-1,0,1} are
    written as 0 and, if ``invalid_count`` (int32 device scalar) is given,
    added to it."""
    _dev(q, "q")
    if q.dtype != torch.int8 or q.dim() != 2:
        raise ValueError("q must be a 2-D int8 tensor")
    N, K = q.shape
    out = torch.empty((N, K // 4), dtype=torch.uint8, device=q.device)
    cnt = None
    if invalid_count is not None:
        _dev(invalid_count, "invalid_count")
        if invalid_count.dtype != torch.int32 or invalid_count.numel() != 1:
            raise ValueError("invalid_count must be a one-element int32 tensor")
        cnt = invalid_count.data_ptr()
    _check(lib().ternary_pack(q.data_ptr(), N, K, out.data_ptr(), cnt, _stream(q)), "ternary_pack")
    return out


def unpack(packed: torch.Tensor, K: int | None = None) -> torch.Tensor:
    """uint8 (or int8 reinterpreted) [N, K/4] -> int8 [N, K].  ``K``, if given,
    must be the row length the packed bytes hold (4 codes per byte)."""
    if packed.dtype == torch.int8:
        packed = packed.view(torch.uint8)
    if packed.dtype != torch.uint8 or packed.dim() != 2:
        raise ValueError("packed must be a 2-D uint8/int8 tensor")
    N = packed.shape[0]
    if K is not None and K != packed.shape[1] * 4:
        raise ValueError(f"K={K} does not match the packed rows ({packed.shape[1]} bytes hold "
                         f"K={packed.shape[1] * 4})")
    K = packed.shape[1] * 4
    _dev(packed, "packed")
    out = torch.empty((N, K), dtype=torch.int8, device=packed.device)
    _check(lib().ternary_unpack(packed.data_ptr(), N, K, out.data_ptr(), _stream(packed)),
           "ternary_unpack")
    return out


_ACT = {torch.bfloat16: BF16, torch.float16: FP16}


def tiled_bytes(N: int, K: int) -> int:
    """Bytes of the tiled layout of an [N, K] code matrix (ternary_tiled_bytes)."""
    r = int(lib().ternary_tiled_bytes(N, K))
    if r < 0:
        raise TernaryError(r, "ternary_tiled_bytes")
    return r


def tile(packed: torch.Tensor) -> torch.Tensor:
    """Row-major codes uint8 [N, K/4] -> the library's tiled layout, a uint8
    tensor [ceil(N/16), ceil(K/256), 1024] (one kilobyte per block of 16 rows x
    256 codes; include/ternary.h gives the byte order)."""
    if packed.dtype == torch.int8:
        packed = packed.view(torch.uint8)
    if packed.dtype != torch.uint8 or packed.dim() != 2:
        raise ValueError("packed must be a 2-D uint8/int8 tensor")
    _dev(packed, "packed")
    N, K = packed.shape[0], packed.shape[1] * 4
    out = torch.empty(((N + 15) // 16, (K + 255) // 256, 1024), dtype=torch.uint8,
                      device=packed.device)
    assert out.numel() == tiled_bytes(N, K)
    _check(lib().ternary_tile(packed.data_ptr(), N, K, out.data_ptr(), _stream(packed)),
           "ternary_tile")
    return out


def untile(tiled: torch.Tensor, N: int, K: int) -> torch.Tensor:
    """The inverse of tile(): tiled codes of an [N, K] matrix -> uint8 [N, K/4]."""
    _dev(tiled, "tiled")
    if tiled.dtype != torch.uint8 or tiled.numel() != tiled_bytes(N, K):
        raise ValueError(f"tiled must be uint8 with {tiled_bytes(N, K)} bytes for N={N}, K={K}")
    out = torch.empty((N, K // 4), dtype=torch.uint8, device=tiled.device)
    _check(lib().ternary_untile(tiled.data_ptr(), N, K, out.data_ptr(), _stream(tiled)),
           "ternary_untile")
    return out


def quantize(w: torch.Tensor, group_size: int = 128):
    """bf16/fp16 weights [N, K] -> (packed uint8 [N, K/4], fp16 scales [N] or
    [N, K/group_size]) by ternary_quantize: per group s = max|w| (fp16),
    q = round(w / s) in {-1, 0, +1}."""
    _dev(w, "w")
    dt = _ACT.get(w.dtype)
    if dt is None or w.dim() != 2:
        raise ValueError("w must be a 2-D bfloat16 or float16 tensor")
    N, K = w.shape
    packed = torch.empty((N, K // 4), dtype=torch.uint8, device=w.device)
    sshape = (N,) if group_size == -1 else (N, K // group_size if group_size > 0 else 0)
    scale = torch.empty(sshape, dtype=torch.float16, device=w.device)
    _check(int(lib().ternary_quantize(w.data_ptr(), dt, N, K, group_size, packed.data_ptr(),
                                      scale.data_ptr(), _stream(w))), "ternary_quantize")
    return packed, scale


def _check_problem(x, packed, scale, group_size, out, layout="rows"):
    """Shapes/dtypes of one problem checked against each other -> (dt, M, N, K, g, packed, out).
    Row-major codes are [N, K/4]; tiled ones any uint8 tensor of tiled_bytes(N, K)
    bytes, N then being taken from the scale's first dimension."""
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {tuple(LAYOUTS)}")
    dt = _ACT.get(x.dtype)
    if dt is None:
        raise ValueError("x must be bfloat16 or float16")
    if packed.dtype == torch.int8:
        packed = packed.view(torch.uint8)
    xs, ps, ss = x.shape, packed.shape, scale.shape
    if len(xs) != 2:
        raise ValueError("x must be 2-D [M, K] (flatten leading dimensions first)")
    if scale.dtype != torch.float16:
        raise ValueError("scale must be float16")
    M, K = xs
    if layout == "tiled":
        if packed.dtype != torch.uint8 or not len(ss):
            raise ValueError("tiled codes must be a uint8 tensor; scale gives N")
        N = ss[0]
        if packed.numel() != tiled_bytes(N, K):
            raise ValueError(f"tiled codes hold {packed.numel()} bytes, N={N}, K={K} needs "
                             f"{tiled_bytes(N, K)}")
    else:
        if packed.dtype != torch.uint8 or len(ps) != 2:
            raise ValueError("packed must be a 2-D uint8/int8 tensor")
        N = ps[0]
        if ps[1] * 4 != K:
            raise ValueError(f"packed has {ps[1]} bytes per row, K={K} needs {K // 4}")
    if group_size is None:
        group_size = -1 if len(ss) == 1 else (K // ss[1] if ss[1] else 0)
    if group_size == -1:
        ok = tuple(ss) == (N,)
    else:
        ok = len(ss) == 2 and group_size > 0 and ss[0] == N and ss[1] * group_size == K
    if not ok:
        raise ValueError(f"scale shape {tuple(ss)} does not match N={N}, K={K}, "
                         f"group_size={group_size}")
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    elif out.dtype != x.dtype or tuple(out.shape) != (M, N) or not out.is_contiguous():
        raise ValueError("out must be contiguous, match x's dtype and have shape [M, N]")
    for t in (x, packed, scale, out):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous device tensors")
    return dt, M, N, K, group_size, packed, out


def linear(x: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor,
           group_size: int | None = None, path: str = "auto",
           out: torch.Tensor | None = None, layout: str = "rows") -> torch.Tensor:
    """y [M, N] = x [M, K] @ (q * s)^T in x's dtype (bf16 or fp16).

    ``scale`` is fp16 [N] (per channel) or [N, K/group_size]; ``group_size`` is
    inferred from its shape when not given.  ``path`` forces a kernel
    ("gemv", "gemm", "simple", "gemv_f4", "gemv_b16"); "auto" picks by M.
    ``layout`` is "rows" (packed [N, K/4]) or "tiled" (packed from tile()).
    Shapes are checked here against each other, so the sizes passed to the C
    ABI match the tensors.
    """
    dt, M, N, K, group_size, packed, out = _check_problem(x, packed, scale, group_size, out,
                                                          layout)
    fn = lib().ternary_linear_tiled if layout == "tiled" else lib().ternary_linear_ex
    st = fn(x.data_ptr(), dt, M, N, K, packed.data_ptr(), scale.data_ptr(), group_size,
            out.data_ptr(), PATHS[path], _stream(x))
    if st:
        raise TernaryError(st, "ternary_linear_tiled" if layout == "tiled" else "ternary_linear")
    return out


def linear_batch(problems, noalloc: bool = False) -> list:
    """Several projections in as few launches as possible (one for all decode
    shapes).  ``problems`` is a sequence of (x, packed, scale, group_size, out)
    tuples, optionally with a sixth element, the layout ("rows" or "tiled");
    group_size and out may be None; returns the outputs.  With
    ``noalloc`` the call goes to ternary_linear_batch_noalloc (split-K scratch
    in the library's static array; no device memory is allocated by the
    library; the outputs are allocated here unless given)."""
    n = len(problems)
    if not 1 <= n <= MAX_BATCH:
        raise ValueError(f"1..{MAX_BATCH} problems per batch")
    arr = (Problem * n)()
    outs = []
    dts = set()
    for i, prob in enumerate(problems):
        x, packed, scale, g, out = prob[:5]
        layout = prob[5] if len(prob) > 5 else "rows"
        dt, M, N, K, g, packed, out = _check_problem(x, packed, scale, g, out, layout)
        dts.add(dt)
        arr[i] = Problem(x.data_ptr(), packed.data_ptr(), scale.data_ptr(), out.data_ptr(),
                         M, N, K, g, LAYOUTS[layout])
        outs.append(out)
    if len(dts) != 1:
        raise ValueError("all problems of a batch share one activation dtype")
    fn = lib().ternary_linear_batch_noalloc if noalloc else lib().ternary_linear_batch
    st = fn(arr, n, dts.pop(), _stream(problems[0][0]))
    if st:
        raise TernaryError(st, "ternary_linear_batch_noalloc" if noalloc else "ternary_linear_batch")
    return outs


def linear_batch_noalloc(problems) -> list:
    """linear_batch through ternary_linear_batch_noalloc."""
    return linear_batch(problems, noalloc=True)


# ---------------------------------------------------------------- 8-bit layers and experts

_OUT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_FP8 = (torch.float8_e4m3fn, torch.uint8)
BLOCKS = {"row": 0, "tile": 1}
ACTS = {"none": 0, "swiglu": 1}
SCORES = {"softmax": 0, "sigmoid": 1}
ROWS = {"tokens": 0, "sorted": 1}
FP8_BLOCK = 128


def _same_device(first: torch.Tensor, *rest) -> int:
    """The device index of contiguous tensors that all live on one device."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("all tensors must be device tensors")
    for t in rest:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous and on one device")
    return dev


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_fns: dict = {}


def _call(name: str, dev: int, *args) -> None:
    """Calls a library function on the current stream of device `dev`."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    if dev == _current_device():
        st = fn(*args, _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    if st:
        raise TernaryError(st, name)


def _choice(table: dict, value, name: str) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {tuple(table)}")
    return table[value]


def _output(out, shape, dtype, dev, like):
    """`out` checked, or a new tensor where `like` is."""
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    if out.shape != shape or out.dtype not in _OUT or not out.is_contiguous() \
            or out.get_device() != dev:
        raise ValueError(f"out must be a contiguous bfloat16, float16 or float32 tensor of shape {shape} "
                         "on the inputs' device")
    return out


def fp8_quantize(x: torch.Tensor, block: str = "row", act: str = "none"):
    """bf16/fp16/fp32 [M, K] -> (float8_e4m3fn [M, Kp], float32 scales), Kp = K rounded
    up to a multiple of 128 (filled with zeros), by ternary_fp8_quantize: a scale
    for 128 values of a row (``block="row"``, scales [M, Kp/128]: activations) or
    for 128 rows x 128 values (``"tile"``, scales [ceil(M/128), Kp/128]: weights).
    ``act="swiglu"`` takes [M, 2K] and quantises silu(x[:, :K]) * x[:, K:].
    Rows may be strided (x.stride(1) == 1)."""
    dt = _OUT.get(x.dtype)
    if dt is None or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16, float16 or float32 tensor")
    b, a = _choice(BLOCKS, block, "block"), _choice(ACTS, act, "act")
    dev = _same_device(x)
    M, width = x.shape
    if width == 0 or (a and width % 2):
        raise ValueError("x must have columns (an even number of them for swiglu)")
    ld = x.stride(0) if M > 1 else width
    if (x.stride(1) != 1 and width > 1) or ld < width:
        raise ValueError("the rows of x must be contiguous and must not overlap")
    K = width // 2 if a else width
    kb = (K + 127) // 128
    q = torch.empty((M, kb * 128), dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty(((M + 127) // 128 if b else M, kb), dtype=torch.float32, device=x.device)
    _call("ternary_fp8_quantize", dev, x.data_ptr(), dt, M, K, ld, b, a, q.data_ptr(), scale.data_ptr())
    return q, scale


def fp8_linear(xq: torch.Tensor, x_scale: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
               dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """y [M, N] = (xq * x_scale) @ (wq * w_scale)^T of block-scaled 8-bit matrices
    (fp8_quantize with ``block="row"`` for x [M, K] and ``"tile"`` for w [N, K]), in
    ``dtype`` (bfloat16, float16 or float32; that of ``out`` if given)."""
    if xq.dtype not in _FP8 or wq.dtype not in _FP8 or xq.dim() != 2 or wq.dim() != 2:
        raise ValueError("xq and wq must be 2-D float8_e4m3fn (or uint8) tensors")
    (M, K), N = xq.shape, wq.shape[0]
    if K == 0 or K % 128 or wq.shape[1] != K:
        raise ValueError(f"xq [{M}, {K}] and wq {tuple(wq.shape)} must share K, a multiple of 128")
    if x_scale.dtype != torch.float32 or w_scale.dtype != torch.float32 \
            or x_scale.shape != (M, K // 128) or w_scale.shape != ((N + 127) // 128, K // 128):
        raise ValueError(f"scales must be float32 [{M}, {K // 128}] and [{(N + 127) // 128}, {K // 128}]")
    dev = _same_device(xq, xq, x_scale, wq, w_scale)
    if dtype not in _OUT:
        raise ValueError("dtype must be bfloat16, float16 or float32")
    out = _output(out, (M, N), dtype, dev, x_scale)
    _call("ternary_fp8_linear", dev, xq.data_ptr(), x_scale.data_ptr(), wq.data_ptr(), w_scale.data_ptr(),
          M, N, K, out.data_ptr(), _OUT[out.dtype])
    return out


class Routing(NamedTuple):
    """What route() gives, and linear_experts() and combine() take (ternary_route)."""
    ids: torch.Tensor      # int32 [T, top_k]: a token's experts, best first; -1: none
    weights: torch.Tensor  # float32 [T, top_k]: their weights
    offsets: torch.Tensor  # int32 [E + 1]: expert e's places are offsets[e] .. offsets[e + 1] - 1
    order: torch.Tensor    # int32 [T * top_k]: the slot t * top_k + j at each place; -1: none
    slots: torch.Tensor    # int32 [T, top_k]: each slot's place; -1: none


def route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor | None = None,
          groups: int = 1, top_groups: int | None = None, renormalize: bool = True,
          scale: float = 1.0) -> Routing:
    """Each token's ``top_k`` experts by softmax or sigmoid scores of logits [T, E]
    (bf16/fp16/fp32), their weights, and the slots sorted by expert.  ``bias``
    (float32 [E]) is added for the choice only; with ``groups`` > 1 only experts of
    the ``top_groups`` groups with the largest sums of their two best scores are
    chosen.  Weights are divided by their sum (``renormalize``) and multiplied
    by ``scale``.  An expert whose logit is -inf is never chosen; a token
    without any (a padded row of -inf) takes no slots."""
    dt = _OUT.get(logits.dtype)
    if dt is None or logits.dim() != 2:
        raise ValueError("logits must be a 2-D bfloat16, float16 or float32 tensor")
    sc = _choice(SCORES, score, "score")
    T, E = logits.shape
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (E,)):
        raise ValueError(f"bias must be a float32 tensor [{E}]")
    dev = _same_device(logits, logits, bias)
    if top_groups is None:
        top_groups = groups
    L = _lib or lib()
    need = L.ternary_route_workspace(T, E)
    if need < 0 or not 1 <= top_k <= 32:
        raise TernaryError(min(need, 0) or -2, "ternary_route")
    d = logits.device
    ids = torch.empty((T, top_k), dtype=torch.int32, device=d)
    weights = torch.empty((T, top_k), dtype=torch.float32, device=d)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=d)
    order = torch.empty(T * top_k, dtype=torch.int32, device=d)
    slots = torch.empty_like(ids)
    # (held until the launches are enqueued: freed before, another thread's call could get it between them)
    ws = torch.empty(need, dtype=torch.uint8, device=d) if need else None
    _call("ternary_route", dev, logits.data_ptr(), dt, T, E, bias.data_ptr() if bias is not None else None,
          sc, groups, top_groups, top_k, 1 if renormalize else 0, scale, ids.data_ptr(),
          weights.data_ptr(), offsets.data_ptr(), order.data_ptr(), slots.data_ptr(),
          ws.data_ptr() if need else None)
    return Routing(ids, weights, offsets, order, slots)


def _check_routing(r: Routing):
    ids, weights, offsets, order, slots = r
    i32, shape = torch.int32, ids.shape
    T, k = shape
    if ids.dtype is not i32 or offsets.dtype is not i32 or order.dtype is not i32 or slots.dtype is not i32 \
            or weights.dtype is not torch.float32 or order.shape != (T * k,) or slots.shape != shape \
            or weights.shape != shape:
        raise ValueError("routing must hold int32 ids and slots [T, k], offsets [E + 1], order [T * k] "
                         "and float32 weights [T, k]")
    return T, k


def linear_experts(xq: torch.Tensor, x_scale: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor,
                   routing: Routing, K: int | None = None, rows: str = "tokens",
                   dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """y [T * top_k, N]: at each place of ``routing.order`` the row of x times its
    expert's ternary weights.  xq [rows, Kp], x_scale [rows, Kp/128] from
    fp8_quantize hold the tokens (``rows="tokens"``) or one row for each place
    (``"sorted"``); ``packed`` holds the experts' tiled codes, uint8
    [E, ...] with tiled_bytes(N, K) bytes each (stacked tile() results); ``scale``
    is float16 [E, N], or [E, N, K/128] or [E, N, K/256] for groups.  ``K`` need only be
    given where it is not Kp.  Rows of places that hold no slot (from
    offsets[E] on) are not written."""
    if xq.dtype not in _FP8 or xq.dim() != 2 or x_scale.dtype != torch.float32:
        raise ValueError("xq must be 2-D float8_e4m3fn (or uint8) and x_scale float32")
    T, k = _check_routing(routing)
    R, (n, Kp) = T * k, xq.shape
    if K is None:
        K = Kp
    if Kp != (K + 127) // 128 * 128 or x_scale.shape != (n, Kp // 128):
        raise ValueError(f"xq [{n}, {Kp}] and x_scale {tuple(x_scale.shape)} do not match K={K}")
    by = _choice(ROWS, rows, "rows")
    if n != (R if by else T):
        raise ValueError(f"xq must hold {R if by else T} rows ({rows})")
    if scale.dtype != torch.float16 or scale.dim() not in (2, 3):
        raise ValueError("scale must be float16 [E, N] or [E, N, K / group size]")
    E, N = scale.shape[:2]
    g = -1
    if scale.dim() == 3:
        g = K // scale.shape[2] if scale.shape[2] else 0
        if g not in (128, 256) or scale.shape[2] * g != K:
            raise ValueError(f"scale {tuple(scale.shape)} holds no groups of 128 or 256 of K={K}")
    if packed.dtype != torch.uint8 or packed.dim() < 1 or packed.shape[0] != E \
            or packed.numel() != E * tiled_bytes(N, K):
        raise ValueError(f"packed must be uint8 [{E}, ...] with {tiled_bytes(N, K)} bytes an expert")
    if routing.offsets.shape != (E + 1,):
        raise ValueError(f"routing.offsets must hold {E + 1} values")
    dev = _same_device(xq, xq, x_scale, packed, scale, routing.offsets, routing.order)
    if dtype not in _OUT:
        raise ValueError("dtype must be bfloat16, float16 or float32")
    out = _output(out, (R, N), dtype, dev, x_scale)
    _call("ternary_linear_experts", dev, xq.data_ptr(), x_scale.data_ptr(), n, packed.data_ptr(),
          scale.data_ptr(), E, N, K, g, routing.offsets.data_ptr(), routing.order.data_ptr(), R, k, by,
          out.data_ptr(), _OUT[out.dtype])
    return out


def combine(y: torch.Tensor, routing: Routing, add: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """out [T, N] = add + the sum of each token's rows of y [T * top_k, N] times
    routing.weights, in y's dtype (bf16, fp16 or fp32; ternary_combine).  ``add`` ([T, N],
    a shared expert's output or the residual) may be ``out`` itself."""
    dt = _OUT.get(y.dtype)
    if dt is None or y.dim() != 2:
        raise ValueError("y must be a 2-D bfloat16, float16 or float32 tensor")
    T, k = _check_routing(routing)
    R, N = y.shape
    if R != T * k:
        raise ValueError(f"y must have {T * k} rows")
    if add is not None and (add.dtype != y.dtype or add.shape != (T, N)):
        raise ValueError(f"add must match y's dtype and have shape [{T}, {N}]")
    dev = _same_device(y, y, routing.slots, routing.weights, add)
    out = _output(out, (T, N), y.dtype, dev, y)
    if out.dtype != y.dtype:
        raise ValueError("out must have y's dtype")
    _call("ternary_combine", dev, y.data_ptr(), dt, R, N, routing.slots.data_ptr(),
          routing.weights.data_ptr(), T, k, add.data_ptr() if add is not None else None, out.data_ptr())
    return out


# ---------------------------------------------------------------- sorted slots, the exchange's gradients, adapters

def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name: str, *sizes) -> int:
    """What library function `name` gives for these sizes."""
    need = getattr(lib(), name)(*sizes)
    if need < 0:
        raise TernaryError(need, name.removesuffix("_workspace"))
    return need


def _workspace(name: str, like: torch.Tensor, *sizes):
    """A new workspace of the size that library function `name` gives; None where it needs none."""
    need = _workspace_bytes(name, *sizes)
    return like.new_empty(need, dtype=torch.uint8) if need else None


def sort_slots(ids: torch.Tensor, experts: int, weights: torch.Tensor | None = None) -> Routing:
    """A Routing of given indices: ids int32 [T, top_k], each slot's expert (another router's choice), or [T] or [T, 1],
    each token's adapter; an id outside [0, experts) holds none (ternary_sort_slots).  ``weights`` (float32
    [T, top_k]; 1 if not given) and ``ids`` are passed on as they are."""
    if ids.dtype != torch.int32 or ids.dim() not in (1, 2):
        raise ValueError("ids must be an int32 tensor [T, top_k] or [T]")
    if ids.dim() == 1:
        ids = ids.unsqueeze(1)
    T, k = ids.shape
    if weights is not None and (weights.dtype != torch.float32 or weights.shape != (T, k)):
        raise ValueError(f"weights must be a float32 tensor [{T}, {k}]")
    dev = _same_device(ids, ids, weights)
    ones = weights is None
    # (held until the launches are enqueued, as route() does)
    ws = _workspace("ternary_sort_slots_workspace", ids, T, k, experts)
    if ones:
        weights = ids.new_empty((T, k), dtype=torch.float32)
    offsets, order, slots = ids.new_empty(experts + 1), ids.new_empty(T * k), torch.empty_like(ids)
    _call("ternary_sort_slots", dev, ids.data_ptr(), T, k, experts, weights.data_ptr() if ones else None,
          offsets.data_ptr(), order.data_ptr(), slots.data_ptr(), _ptr(ws))
    return Routing(ids, weights, offsets, order, slots)


def _rows_of(t: torch.Tensor, rows: int, name: str):
    """The dtype code and row length of `t`, a matrix of `rows` rows."""
    dt = _OUT.get(t.dtype)
    if dt is None or t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must be a bfloat16, float16 or float32 tensor of {rows} rows")
    return dt, t.shape[1]


def _match(t: torch.Tensor | None, shape: tuple, dtype: torch.dtype, name: str):
    if t is not None and (t.dtype != dtype or t.shape != shape):
        raise ValueError(f"{name} must be a {str(dtype)[6:]} tensor of shape {list(shape)}")


def dispatch(x: torch.Tensor, routing: Routing, weighted: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """out [T * top_k, N]: at each place of ``routing.order`` the token's row of x [T, N], with ``weighted`` times the
    slot's weight, in x's dtype (bf16, fp16 or fp32; ternary_dispatch): the rows that experts take with
    ``rows="sorted"``.  Rows of places that hold no slot are not written.  combine() is the way back."""
    T, k = _check_routing(routing)
    dt, N = _rows_of(x, T, "x")
    dev = _same_device(x, x, routing.slots, routing.weights)
    out = _output(out, (T * k, N), x.dtype, dev, x)
    if out.dtype != x.dtype:
        raise ValueError("out must have x's dtype")
    _call("ternary_dispatch", dev, x.data_ptr(), dt, T, N, routing.slots.data_ptr(),
          routing.weights.data_ptr() if weighted else None, k, T * k, out.data_ptr())
    return out


def dispatch_backward(grad: torch.Tensor, routing: Routing, x: torch.Tensor | None = None,
                      add: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """The gradient of dispatch(): grad [T * top_k, N] is that of its result, which gives dx [T, N], plus ``add`` (another
    gradient of x; may be ``out``, which receives dx).  With x, that of ``dispatch(x, routing, weighted=True)``: (dx,
    dweights), dweights float32 [T, top_k] (ternary_dispatch_backward)."""
    T, k = _check_routing(routing)
    dt, N = _rows_of(grad, T * k, "grad")
    _match(x, (T, N), grad.dtype, "x")
    _match(add, (T, N), grad.dtype, "add")
    dev = _same_device(grad, grad, routing.slots, routing.weights, x, add)
    out = _output(out, (T, N), grad.dtype, dev, grad)
    if out.dtype != grad.dtype:
        raise ValueError("out must have grad's dtype")
    dw = None if x is None else torch.empty_like(routing.weights)
    _call("ternary_dispatch_backward", dev, grad.data_ptr(), dt, T * k, N, routing.slots.data_ptr(),
          None if x is None else routing.weights.data_ptr(), T, k, _ptr(x), _ptr(add), out.data_ptr(), _ptr(dw))
    return out if x is None else (out, dw)


def combine_backward(grad: torch.Tensor, y: torch.Tensor, routing: Routing, out: torch.Tensor | None = None):
    """The gradient of ``combine(y, routing)`` from grad [T, N], that of its result: (dy [T * top_k, N], dweights float32
    [T, top_k]); that of its ``add`` is grad itself (ternary_combine_backward).  Rows of dy (``out``) at
    places that hold no slot are not written."""
    T, k = _check_routing(routing)
    dt, N = _rows_of(grad, T, "grad")
    _match(y, (T * k, N), grad.dtype, "y")
    dev = _same_device(grad, grad, y, routing.slots, routing.weights)
    out = _output(out, (T * k, N), grad.dtype, dev, grad)
    if out.dtype != grad.dtype:
        raise ValueError("out must have grad's dtype")
    dw = torch.empty_like(routing.weights)
    _call("ternary_combine_backward", dev, grad.data_ptr(), y.data_ptr(), dt, T * k, N, routing.slots.data_ptr(),
          routing.weights.data_ptr(), T, k, out.data_ptr(), dw.data_ptr())
    return out, dw


def _check_adapters(x, a, b, routing, scale):
    """Shapes of adapters' operands checked against each other -> dtype code, T, K, N, rank, E."""
    dtype, xs, ash, bsh = x.dtype, x.shape, a.shape, b.shape
    dt = _ACT.get(dtype)
    if dt is None or len(xs) != 2:
        raise ValueError("x must be a 2-D bfloat16 or float16 tensor")
    T, K = xs
    if len(ash) != 3 or len(bsh) != 3 or a.dtype is not dtype or b.dtype is not dtype or ash[2] != K \
            or bsh[0] != ash[0] or bsh[2] != ash[1]:
        raise ValueError(f"a [E, rank, {K}] and b [E, N, rank] must have x's dtype and share E and rank")
    E, rank, _ = ash
    if scale is not None and (scale.dtype != torch.float32 or scale.shape != (E,)):
        raise ValueError(f"scale must be a float32 tensor [{E}]")
    if _check_routing(routing) != (T, 1) or routing.offsets.shape != (E + 1,):
        raise ValueError(f"routing must be sort_slots() of {T} tokens' adapters, with {E + 1} offsets")
    return dt, T, K, bsh[1], rank, E


def linear_adapters(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, routing: Routing,
                    scale: torch.Tensor | None = None, add: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, hidden: torch.Tensor | None = None) -> torch.Tensor:
    """y [T, N] = add + scale[e] * (x @ a[e]^T) @ b[e]^T, e each token's adapter: low-rank adapters of many requests beside
    a shared projection, whose output ``add`` is (and may be ``out``).  x [T, K], a [E, rank, K] and b
    [E, N, rank] (rank up to 128; smaller ones filled up with zeros) share a dtype, bf16 or fp16; scale is float32
    [E] (1 if not given); ``routing`` is ``sort_slots(adapters, E)``, made once for all projections of a batch.  A
    token without an adapter gets ``add``, or 0.  ``hidden`` (float32 [T, rank]) receives x @ a[e]^T, for
    linear_adapters_backward() (ternary_linear_adapters)."""
    dt, T, K, N, rank, E = _check_adapters(x, a, b, routing, scale)
    _match(add, (T, N), x.dtype, "add")
    _match(hidden, (T, rank), torch.float32, "hidden")
    dev = _same_device(x, x, a, b, scale, add, hidden, routing.offsets, routing.order, routing.slots)
    out = _output(out, (T, N), x.dtype, dev, x)
    if out.dtype != x.dtype:
        raise ValueError("out must have x's dtype")
    ws = _workspace("ternary_linear_adapters_workspace", x, T, K, N, rank, E)
    _call("ternary_linear_adapters", dev, x.data_ptr(), dt, T, K, N, rank, a.data_ptr(), b.data_ptr(), E, _ptr(scale),
          routing.offsets.data_ptr(), routing.order.data_ptr(), routing.slots.data_ptr(), _ptr(add), out.data_ptr(),
          _ptr(hidden), _ptr(ws))
    return out


def linear_adapters_backward(grad: torch.Tensor, x: torch.Tensor, hidden: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                             routing: Routing, scale: torch.Tensor | None = None, add: torch.Tensor | None = None,
                             out: torch.Tensor | None = None):
    """The gradients of linear_adapters() from grad [T, N], that of its result: (dx [T, K], da, db), in x's dtype.
    ``hidden`` is what the forward call wrote; ``add`` ([T, K], another gradient of x, such as the
    projection's own; may be ``out``, which receives dx) is added to dx.  The gradient of the
    forward call's ``add`` is grad itself (ternary_linear_adapters_backward)."""
    dt, T, K, N, rank, E = _check_adapters(x, a, b, routing, scale)
    _match(grad, (T, N), x.dtype, "grad")
    _match(hidden, (T, rank), torch.float32, "hidden")
    _match(add, (T, K), x.dtype, "add")
    dev = _same_device(x, x, grad, hidden, a, b, scale, add, routing.offsets, routing.order, routing.slots)
    out = _output(out, (T, K), x.dtype, dev, x)
    if out.dtype != x.dtype:
        raise ValueError("out must have x's dtype")
    da, db = torch.empty_like(a), torch.empty_like(b)
    ws = _workspace("ternary_linear_adapters_backward_workspace", x, T, K, N, rank, E)
    _call("ternary_linear_adapters_backward", dev, grad.data_ptr(), x.data_ptr(), hidden.data_ptr(), dt, T, K, N, rank,
          a.data_ptr(), b.data_ptr(), E, _ptr(scale), routing.offsets.data_ptr(), routing.order.data_ptr(),
          routing.slots.data_ptr(), _ptr(add), out.data_ptr(), da.data_ptr(), db.data_ptr(), _ptr(ws))
    return out, da, db


# ---------------------------------------------------------------- probes

def probe_read(buf: torch.Tensor, sink: torch.Tensor, workgroups: int,
               nontemporal: bool = False) -> None:
    """Read all bytes of ``buf`` once (ternary_probe_read, or
    ternary_probe_read_nt with non-temporal loads); ``sink`` is a one-element
    int32 device tensor."""
    _dev(buf, "buf")
    _dev(sink, "sink")
    nbytes = buf.numel() * buf.element_size()
    name = "ternary_probe_read_nt" if nontemporal else "ternary_probe_read"
    _check(int(getattr(probe_lib(), name)(buf.data_ptr(), nbytes, workgroups, sink.data_ptr(),
                                          _stream(buf))), name)


def probe_copy(src: torch.Tensor, dst: torch.Tensor, workgroups: int) -> None:
    """Copy ``src`` into ``dst`` (same byte size) with ternary_probe_copy."""
    _dev(src, "src")
    _dev(dst, "dst")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst must hold the same number of bytes")
    _check(int(probe_lib().ternary_probe_copy(src.data_ptr(), dst.data_ptr(), nbytes,
                                              workgroups, _stream(src))),
           "ternary_probe_copy")


def probe_mfma(workgroups: int, iters: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Run the MFMA loop probe; returns its float32 [workgroups * 256] output.
    The launch performs workgroups * 4 * iters * 4 * 16384 flops."""
    n = workgroups * PROBE_THREADS
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device="cuda")
    elif out.dtype != torch.float32 or out.numel() < n:
        raise ValueError(f"out must be float32 with at least {n} elements")
    _dev(out, "out")
    _check(int(probe_lib().ternary_probe_mfma(workgroups, iters, out.data_ptr(), _stream(out))),
           "ternary_probe_mfma")
    return out


def probe_mfma_flops(workgroups: int, iters: int) -> int:
    return workgroups * 4 * iters * 4 * 16384
