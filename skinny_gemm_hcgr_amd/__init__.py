"""Python binding of the MI355X Hyper-Connection Gated Residual library.

The functions below carry the C ABI names of ``include/hcgr.h`` and only
marshal arguments (tensor pointers, sizes, the current HIP stream) to
``libhcgr.so``; every step of the op runs in the library's HIP kernels.
PyTorch provides device memory and streams. There is no fallback: if the
library is missing or cannot be loaded, every call raises.

``HCGR`` is a small convenience object over the same calls that allocates
outputs and the workspace with torch on the tensors' device.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhcgr.so")

HCGR_OK = 0
HCGR_ERR_INVALID_ARGUMENT = 1
HCGR_ERR_UNSUPPORTED = 2
HCGR_ERR_ALIASING = 3
HCGR_ERR_WORKSPACE_TOO_SMALL = 4
HCGR_ERR_HIP = 5
HCGR_WEIGHTS_SEPARATE = 0
HCGR_WEIGHTS_MERGED_FOLDED = 1
HCGR_PLAN_HEURISTIC = -1
HCGR_PLAN_SPLIT = 0
HCGR_PLAN_TILE = 3
HCGR_PLAN_FUSED = 4
HCGR_PLAN_PERSISTENT = 5
HCGR_SPLIT_VARIANTS = 13  # down-kernel variants of the decode plans (include/hcgr.h)
HCGR_WORKSPACE_COUNTER_BYTES = 131072
HCGR_BF16 = 0
HCGR_FP16 = 1
HCGR_FP32 = 2
HCGR_LINEAR_MAX_K = 131071
HCGR_LINEAR_MAX_N = 1048576
HCGR_LINEAR_MAX_LD = 4194304
HCGR_DEFAULT_WAIT_POLLS = 1 << 20
HCGR_MAX_WAIT_POLLS = 1 << 24
PLAN_FIELDS = ("tokens", "kind", "down_variant", "streams_per_wg", "segments", "up_variant", "ranges")


class HcgrError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}: {detail}")


class hcgr_config(ctypes.Structure):
    _fields_ = [("hc", ctypes.c_int32), ("hs", ctypes.c_int32), ("r", ctypes.c_int32),
                ("eps", ctypes.c_float), ("wnorm_len", ctypes.c_int32),
                ("weight_layout", ctypes.c_int32), ("n_pad", ctypes.c_int32)]


class hcgr_block_config(ctypes.Structure):
    _fields_ = [("hc", ctypes.c_int32), ("hs", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("res_scale", ctypes.c_float)]


class hcgr_linear_config(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("k", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class hcgr_plan_choice(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("kind", ctypes.c_int32), ("down_variant", ctypes.c_int32),
                ("streams_per_wg", ctypes.c_int32), ("segments", ctypes.c_int32), ("up_variant", ctypes.c_int32),
                ("ranges", ctypes.c_int32)]


def _choices_in(table):
    """A table (list of dicts with PLAN_FIELDS keys) as a ctypes array and its length."""
    table = list(table or [])
    arr = (hcgr_plan_choice * max(1, len(table)))()
    for i, e in enumerate(table):
        for f in PLAN_FIELDS:
            setattr(arr[i], f, int(e.get(f, 0)))
    return arr, len(table)


def _choice_out(c) -> dict:
    return {f: int(getattr(c, f)) for f in PLAN_FIELDS}


@dataclass(frozen=True)
class Config:
    hc: int = 4
    hs: int = 2560
    r: int = 320
    eps: float = 1e-6
    wnorm_len: int = 0          # 0 means hs
    weight_layout: int = HCGR_WEIGHTS_SEPARATE
    n_pad: int = 0

    def c(self) -> hcgr_config:
        return hcgr_config(self.hc, self.hs, self.r, self.eps, self.wnorm_len or self.hs,
                           self.weight_layout, self.n_pad)

    @property
    def k(self) -> int:
        return self.hc * self.hs

    @property
    def merged(self) -> bool:
        return self.weight_layout == HCGR_WEIGHTS_MERGED_FOLDED


@dataclass(frozen=True)
class BlockConfig:
    """Streams, width, type and constants of the norms around a block
    (``hcgr_block_config``)."""
    hc: int = 4
    hs: int = 2560
    dtype: int = HCGR_BF16
    eps: float = 1e-6
    res_scale: float = 1.0

    def c(self) -> hcgr_block_config:
        return hcgr_block_config(self.hc, self.hs, self.dtype, self.eps, self.res_scale)

    @property
    def k(self) -> int:
        return self.hc * self.hs


@dataclass(frozen=True)
class LinearConfig:
    """Sizes of an 8-bit linear layer and the type around it (``hcgr_linear_config``)."""
    n: int
    k: int
    dtype: int = HCGR_BF16

    def c(self) -> hcgr_linear_config:
        return hcgr_linear_config(self.n, self.k, self.dtype)


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libhcgr.so (built by ``skinny_gemm_hcgr_amd.build``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m skinny_gemm_hcgr_amd.build` "
                           "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(path)
    P, I64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    CFG = ctypes.POINTER(hcgr_config)
    lib.hcgr_create.argtypes = [CFG, ctypes.c_int, ctypes.POINTER(P)]
    lib.hcgr_destroy.argtypes = [P]
    lib.hcgr_destroy.restype = None
    lib.hcgr_workspace_size.argtypes = [P, I64, ctypes.POINTER(SZ)]
    lib.hcgr_workspace_size_for.argtypes = [CFG, I64, ctypes.POINTER(SZ)]
    lib.hcgr_forward.argtypes = [P, P, P, P, I64, P, P, P, P, I64, P, P, P, I64, P, P, SZ, P]
    lib.hcgr_forward_timed.argtypes = [P, P, P, P, I64, P, P, P, P, I64, P, P, P, I64, P, P, SZ, P,
                                       ctypes.POINTER(P)]
    lib.hcgr_forward_noalloc.argtypes = [P, P, P, P, I64, P, P, P, P, I64, P, P, P, I64, P, P]
    lib.hcgr_noalloc_scratch_bytes.argtypes = []
    lib.hcgr_noalloc_scratch_bytes.restype = SZ
    lib.hcgr_validate.argtypes = [CFG, P, P, P, I64, P, P, P, P, I64, P, P, P, I64, P, P, SZ]
    lib.hcgr_combine.argtypes = [P, P, P, P, I64, I64, P, P]
    lib.hcgr_mix.argtypes = [P, P, P, P, P, P, I64, P, P, I64, P, P, SZ, P]
    lib.hcgr_validate_combine.argtypes = [CFG, P, P, P, I64, I64, P]
    lib.hcgr_validate_mix.argtypes = [CFG, P, P, P, P, P, I64, P, P, I64, P, P, SZ]
    lib.hcgr_describe_plan.argtypes = [CFG, I64, ctypes.c_char_p, SZ]
    PC = ctypes.POINTER(hcgr_plan_choice)
    lib.hcgr_plan_candidates.argtypes = [CFG, I64, PC, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]
    lib.hcgr_plan_lookup.argtypes = [CFG, PC, ctypes.c_int32, I64, PC, ctypes.c_char_p, SZ]
    lib.hcgr_workspace_size_table.argtypes = [CFG, PC, ctypes.c_int32, I64, ctypes.POINTER(SZ)]
    lib.hcgr_set_plan_table.argtypes = [P, PC, ctypes.c_int32]
    lib.hcgr_set_wait_polls.argtypes = [P, ctypes.c_int32]
    BCFG, LCFG = ctypes.POINTER(hcgr_block_config), ctypes.POINTER(hcgr_linear_config)
    block = {"norm": [P, I64, P, I64, P, P, I64, P, P],
             "norm_bwd": [P, I64, P, P, P, I64, P, P, P, SZ],
             "residual": [P, P, I64, P, I64, P, P, I64, P, P, P, I64, P, P],
             "residual_bwd": [P, P, I64, P, I64, P, P, P, P, P, I64, P, P, P, I64, P, P, P, SZ]}
    linear = {"quantize": [P, I64, I64, P, I64, P],
              "forward": [P, I64, P, P, I64, P, P, I64, P, I64]}
    added = ["hcgr_block_create", "hcgr_block_workspace_size", "hcgr_block_workspace_size_for", "hcgr_linear_create"]
    lib.hcgr_block_create.argtypes = [BCFG, ctypes.c_int, ctypes.POINTER(P)]
    lib.hcgr_linear_create.argtypes = [LCFG, ctypes.c_int, ctypes.POINTER(P)]
    lib.hcgr_block_destroy.argtypes = lib.hcgr_linear_destroy.argtypes = [P]
    lib.hcgr_block_destroy.restype = lib.hcgr_linear_destroy.restype = None
    lib.hcgr_block_workspace_size.argtypes = [P, I64, ctypes.POINTER(SZ)]
    lib.hcgr_block_workspace_size_for.argtypes = [BCFG, I64, ctypes.POINTER(SZ)]
    for kind, cfg, calls in (("block", BCFG, block), ("linear", LCFG, linear)):
        for name, args in calls.items():
            getattr(lib, f"hcgr_{kind}_{name}").argtypes = [P, *args, P]
            getattr(lib, f"hcgr_validate_{kind}_{name}").argtypes = [cfg, *args]
            added += [f"hcgr_{kind}_{name}", f"hcgr_validate_{kind}_{name}"]
    lib.hcgr_status_string.argtypes = [ctypes.c_int]
    lib.hcgr_status_string.restype = ctypes.c_char_p
    lib.hcgr_last_error.argtypes = []
    lib.hcgr_last_error.restype = ctypes.c_char_p
    for name in ("hcgr_create", "hcgr_workspace_size", "hcgr_workspace_size_for", "hcgr_forward",
                 "hcgr_forward_timed", "hcgr_forward_noalloc", "hcgr_combine", "hcgr_mix", "hcgr_validate_combine",
                 "hcgr_validate_mix", "hcgr_validate", "hcgr_describe_plan", "hcgr_plan_candidates",
                 "hcgr_plan_lookup", "hcgr_workspace_size_table", "hcgr_set_plan_table", "hcgr_set_wait_polls",
                 *added):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().hcgr_status_string(int(status)).decode()


def last_error() -> str:
    return load_library().hcgr_last_error().decode()


def _check(status: int, where: str) -> int:
    if status != HCGR_OK:
        raise HcgrError(status, where, last_error())
    return status


def _p(t) -> int:
    """Device (or host) address of a tensor, an int address, or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# ------------------------------------------------------- C ABI, same names --
def hcgr_create(cfg: Config, device: int = 0) -> int:
    h = ctypes.c_void_p()
    c = cfg.c()
    _check(load_library().hcgr_create(ctypes.byref(c), int(device), ctypes.byref(h)), "hcgr_create")
    return h.value


def hcgr_destroy(handle: int) -> None:
    load_library().hcgr_destroy(handle)


def hcgr_workspace_size(handle: int, M: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().hcgr_workspace_size(handle, int(M), ctypes.byref(n)), "hcgr_workspace_size")
    return n.value


def hcgr_workspace_size_for(cfg: Config, M: int) -> int:
    n = ctypes.c_size_t()
    c = cfg.c()
    _check(load_library().hcgr_workspace_size_for(ctypes.byref(c), int(M), ctypes.byref(n)),
           "hcgr_workspace_size_for")
    return n.value


def hcgr_describe_plan(cfg: Config, M: int) -> str:
    buf = ctypes.create_string_buffer(1024)
    c = cfg.c()
    _check(load_library().hcgr_describe_plan(ctypes.byref(c), int(M), buf, len(buf)), "hcgr_describe_plan")
    return buf.value.decode()


def hcgr_plan_candidates(cfg: Config, M: int) -> list:
    """Every plan choice that can run cfg's shape at M tokens (dicts with PLAN_FIELDS)."""
    lib, c, n = load_library(), cfg.c(), ctypes.c_int32()
    _check(lib.hcgr_plan_candidates(ctypes.byref(c), int(M), None, 0, ctypes.byref(n)), "hcgr_plan_candidates")
    arr = (hcgr_plan_choice * max(1, n.value))()
    _check(lib.hcgr_plan_candidates(ctypes.byref(c), int(M), arr, n.value, ctypes.byref(n)), "hcgr_plan_candidates")
    return [_choice_out(arr[i]) for i in range(n.value)]


def hcgr_plan_lookup(cfg: Config, table, M: int):
    """(choice the table resolves M to, description of the resulting plan)."""
    c, (arr, n) = cfg.c(), _choices_in(table)
    out, buf = hcgr_plan_choice(), ctypes.create_string_buffer(1024)
    _check(load_library().hcgr_plan_lookup(ctypes.byref(c), arr, n, int(M), ctypes.byref(out), buf, len(buf)),
           "hcgr_plan_lookup")
    return _choice_out(out), buf.value.decode()


def hcgr_workspace_size_table(cfg: Config, table, M: int) -> int:
    c, (arr, n), b = cfg.c(), _choices_in(table), ctypes.c_size_t()
    _check(load_library().hcgr_workspace_size_table(ctypes.byref(c), arr, n, int(M), ctypes.byref(b)),
           "hcgr_workspace_size_table")
    return b.value


def hcgr_set_plan_table(handle: int, table) -> None:
    arr, n = _choices_in(table)
    _check(load_library().hcgr_set_plan_table(handle, arr, n), "hcgr_set_plan_table")


def hcgr_set_wait_polls(handle: int, polls: int) -> None:
    _check(load_library().hcgr_set_wait_polls(handle, int(polls)), "hcgr_set_wait_polls")


PLANS_DIR = os.path.join(_PKG, "plans")


def shipped_plan_table(cfg: Config):
    """Path of the tuned table shipped with the package for cfg (written by
    ``skinny_gemm_hcgr_amd.tune`` on an MI355X), or None."""
    name = f"hc{cfg.hc}_hs{cfg.hs}_r{cfg.r}" + ("_merged" if cfg.merged else "") + \
        ("_wnfull" if (cfg.wnorm_len or cfg.hs) != cfg.hs else "") + ".json"
    path = os.path.join(PLANS_DIR, name)
    return path if os.path.exists(path) else None


def load_plan_table(path: str, cfg: Config) -> list:
    """Entries of a tuned-plan JSON file (written by ``skinny_gemm_hcgr_amd.tune``);
    raises if the file was tuned for another configuration."""
    import json
    with open(path) as f:
        d = json.load(f)
    want = {"hc": cfg.hc, "hs": cfg.hs, "r": cfg.r, "wnorm_len": cfg.wnorm_len or cfg.hs,
            "weight_layout": cfg.weight_layout}
    got = {k: d.get("config", {}).get(k) for k in want}
    if got != want:
        raise ValueError(f"{path} was tuned for {got}, not {want}")
    return [{f: int(e[f]) for f in PLAN_FIELDS} for e in d["entries"]]


def _stream(stream, like):
    """Raw hipStream_t from an int, a torch stream, or None (torch's current
    stream on the device of the tensor ``like``)."""
    if stream is None:
        import torch
        dev = like.device if hasattr(like, "device") else None
        return torch.cuda.current_stream(dev).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def hcgr_forward(handle, R, y, inj, ld_inj, wnorm, wd, wi, wu, M, R2, rrms, inj_next, ld_inj_next, x,
                 workspace, workspace_bytes, stream=None, *, check: bool = True) -> int:
    """Tensors (or raw addresses) in, status out; ``stream`` is a raw hipStream_t
    (an int), a torch stream, or None for torch's current stream on ``R``'s device."""
    stream = _stream(stream, R)
    st = load_library().hcgr_forward(handle, _p(R), _p(y), _p(inj), int(ld_inj), _p(wnorm), _p(wd), _p(wi),
                                     _p(wu), int(M), _p(R2), _p(rrms), _p(inj_next), int(ld_inj_next), _p(x),
                                     _p(workspace), int(workspace_bytes), stream)
    if check:
        _check(st, "hcgr_forward")
    return st


def hcgr_forward_timed(handle, R, y, inj, ld_inj, wnorm, wd, wi, wu, M, R2, rrms, inj_next, ld_inj_next, x,
                       workspace, workspace_bytes, stream, events) -> int:
    """``hcgr_forward`` plus 6 caller-owned hipEvent_t handles (ints): events
    2i and 2i+1 take the start and end of stage i's kernel (down/inject,
    reduction, up/mix)."""
    if not isinstance(stream, int):
        stream = stream.cuda_stream
    if len(events) != 6:
        raise ValueError("hcgr_forward_timed takes 6 events")
    ev = (ctypes.c_void_p * 6)(*events)
    st = load_library().hcgr_forward_timed(handle, _p(R), _p(y), _p(inj), int(ld_inj), _p(wnorm), _p(wd), _p(wi),
                                           _p(wu), int(M), _p(R2), _p(rrms), _p(inj_next), int(ld_inj_next), _p(x),
                                           _p(workspace), int(workspace_bytes), stream, ev)
    return _check(st, "hcgr_forward_timed")


def hcgr_forward_noalloc(handle, R, y, inj, ld_inj, wnorm, wd, wi, wu, M, R2, rrms, inj_next, ld_inj_next, x,
                         stream=None, *, check: bool = True) -> int:
    """``hcgr_forward`` on the library's own per-GPU scratch instead of a caller
    workspace (stream as in ``hcgr_forward``)."""
    stream = _stream(stream, R)
    st = load_library().hcgr_forward_noalloc(handle, _p(R), _p(y), _p(inj), int(ld_inj), _p(wnorm), _p(wd), _p(wi),
                                             _p(wu), int(M), _p(R2), _p(rrms), _p(inj_next), int(ld_inj_next),
                                             _p(x), stream)
    if check:
        _check(st, "hcgr_forward_noalloc")
    return st


def hcgr_noalloc_scratch_bytes() -> int:
    return int(load_library().hcgr_noalloc_scratch_bytes())


def hcgr_combine(handle, R, y, inj, ld_inj, M, R2, stream=None, *, check: bool = True) -> int:
    """(COMBINE) alone: R2 = R + y*iw (stream as in ``hcgr_forward``)."""
    st = load_library().hcgr_combine(handle, _p(R), _p(y), _p(inj), int(ld_inj), int(M), _p(R2),
                                     _stream(stream, R))
    if check:
        _check(st, "hcgr_combine")
    return st


def hcgr_mix(handle, R, wnorm, wd, wi, wu, M, rrms, inj_next, ld_inj_next, x, workspace, workspace_bytes,
             stream=None, *, check: bool = True) -> int:
    """Every step but COMBINE on a residual R taken as R2 (stream as in ``hcgr_forward``)."""
    st = load_library().hcgr_mix(handle, _p(R), _p(wnorm), _p(wd), _p(wi), _p(wu), int(M), _p(rrms),
                                 _p(inj_next), int(ld_inj_next), _p(x), _p(workspace), int(workspace_bytes),
                                 _stream(stream, R))
    if check:
        _check(st, "hcgr_mix")
    return st


def hcgr_validate_combine(cfg: Config, R, y, inj, ld_inj, M, R2) -> int:
    """Host-only checks of ``hcgr_combine``; returns the status code (does not raise)."""
    c = cfg.c()
    return load_library().hcgr_validate_combine(ctypes.byref(c), _p(R), _p(y), _p(inj), int(ld_inj), int(M),
                                                _p(R2))


def hcgr_validate_mix(cfg: Config, R, wnorm, wd, wi, wu, M, rrms, inj_next, ld_inj_next, x, workspace,
                      workspace_bytes) -> int:
    """Host-only checks of ``hcgr_mix``; returns the status code (does not raise)."""
    c = cfg.c()
    return load_library().hcgr_validate_mix(ctypes.byref(c), _p(R), _p(wnorm), _p(wd), _p(wi), _p(wu), int(M),
                                            _p(rrms), _p(inj_next), int(ld_inj_next), _p(x), _p(workspace),
                                            int(workspace_bytes))


def hcgr_validate(cfg: Config, R, y, inj, ld_inj, wnorm, wd, wi, wu, M, R2, rrms, inj_next, ld_inj_next, x,
                  workspace, workspace_bytes) -> int:
    """Host-only argument checks; returns the status code (does not raise)."""
    c = cfg.c()
    return load_library().hcgr_validate(ctypes.byref(c), _p(R), _p(y), _p(inj), int(ld_inj), _p(wnorm), _p(wd),
                                        _p(wi), _p(wu), int(M), _p(R2), _p(rrms), _p(inj_next),
                                        int(ld_inj_next), _p(x), _p(workspace), int(workspace_bytes))


# ---------------------------------------- the block operators, same names --
def hcgr_block_create(cfg: BlockConfig, device: int = 0) -> int:
    h, c = ctypes.c_void_p(), cfg.c()
    _check(load_library().hcgr_block_create(ctypes.byref(c), int(device), ctypes.byref(h)), "hcgr_block_create")
    return h.value


def hcgr_block_destroy(handle: int) -> None:
    load_library().hcgr_block_destroy(handle)


def hcgr_block_workspace_size(handle: int, M: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().hcgr_block_workspace_size(handle, int(M), ctypes.byref(n)), "hcgr_block_workspace_size")
    return n.value


def hcgr_block_workspace_size_for(cfg: BlockConfig, M: int) -> int:
    n, c = ctypes.c_size_t(), cfg.c()
    _check(load_library().hcgr_block_workspace_size_for(ctypes.byref(c), int(M), ctypes.byref(n)),
           "hcgr_block_workspace_size_for")
    return n.value


def _call(name, handle, args, stream, like, check):
    st = getattr(load_library(), name)(handle, *args, _stream(stream, like))
    if check:
        _check(st, name)
    return st


def _validate(name, cfg, args):
    c = cfg.c()
    return getattr(load_library(), name)(ctypes.byref(c), *args)


def _norm_args(x, ld_x, w, M, xn, q, ld_q, q_scale, rrms):
    return _p(x), int(ld_x), _p(w), int(M), _p(xn), _p(q), int(ld_q), _p(q_scale), _p(rrms)


def _norm_bwd_args(x, ld_x, w, rrms, dxn, M, dx, dw, workspace, workspace_bytes):
    return (_p(x), int(ld_x), _p(w), _p(rrms), _p(dxn), int(M), _p(dx), _p(dw), _p(workspace), int(workspace_bytes))


def _residual_args(R, y, ld_y, inj, ld_inj, w_post, w_pre, M, R2, x, q, ld_q, q_scale, rrms):
    return (_p(R), _p(y), int(ld_y), _p(inj), int(ld_inj), _p(w_post), _p(w_pre), int(M), _p(R2), _p(x), _p(q),
            int(ld_q), _p(q_scale), _p(rrms))


def _residual_bwd_args(R, y, ld_y, inj, ld_inj, w_post, w_pre, rrms, dR2, dx, M, dR, dy, dinj, ld_dinj, dw_post,
                       dw_pre, workspace, workspace_bytes):
    return (_p(R), _p(y), int(ld_y), _p(inj), int(ld_inj), _p(w_post), _p(w_pre), _p(rrms), _p(dR2), _p(dx), int(M),
            _p(dR), _p(dy), _p(dinj), int(ld_dinj), _p(dw_post), _p(dw_pre), _p(workspace), int(workspace_bytes))


def _quantize_args(x, ld_x, M, q, ld_q, q_scale):
    return _p(x), int(ld_x), int(M), _p(q), int(ld_q), _p(q_scale)


def _linear_args(q, ld_q, q_scale, w, ld_w, w_scale, bias, M, out, ld_out):
    return (_p(q), int(ld_q), _p(q_scale), _p(w), int(ld_w), _p(w_scale), _p(bias), int(M), _p(out), int(ld_out))


def hcgr_block_norm(handle, x, *args, stream=None, check: bool = True) -> int:
    """(x, ld_x, w, M, xn, q, ld_q, q_scale, rrms); stream as in ``hcgr_forward``."""
    return _call("hcgr_block_norm", handle, _norm_args(x, *args), stream, x, check)


def hcgr_block_norm_bwd(handle, x, *args, stream=None, check: bool = True) -> int:
    """(x, ld_x, w, rrms, dxn, M, dx, dw, workspace, workspace_bytes)."""
    return _call("hcgr_block_norm_bwd", handle, _norm_bwd_args(x, *args), stream, x, check)


def hcgr_block_residual(handle, R, *args, stream=None, check: bool = True) -> int:
    """(R, y, ld_y, inj, ld_inj, w_post, w_pre, M, R2, x, q, ld_q, q_scale, rrms)."""
    return _call("hcgr_block_residual", handle, _residual_args(R, *args), stream, R, check)


def hcgr_block_residual_bwd(handle, R, *args, stream=None, check: bool = True) -> int:
    """(R, y, ld_y, inj, ld_inj, w_post, w_pre, rrms, dR2, dx, M, dR, dy, dinj,
    ld_dinj, dw_post, dw_pre, workspace, workspace_bytes)."""
    return _call("hcgr_block_residual_bwd", handle, _residual_bwd_args(R, *args), stream, R, check)


def hcgr_validate_block_norm(cfg: BlockConfig, *args) -> int:
    """Host-only checks of ``hcgr_block_norm``; returns the status code (does not raise)."""
    return _validate("hcgr_validate_block_norm", cfg, _norm_args(*args))


def hcgr_validate_block_norm_bwd(cfg: BlockConfig, *args) -> int:
    return _validate("hcgr_validate_block_norm_bwd", cfg, _norm_bwd_args(*args))


def hcgr_validate_block_residual(cfg: BlockConfig, *args) -> int:
    return _validate("hcgr_validate_block_residual", cfg, _residual_args(*args))


def hcgr_validate_block_residual_bwd(cfg: BlockConfig, *args) -> int:
    return _validate("hcgr_validate_block_residual_bwd", cfg, _residual_bwd_args(*args))


def hcgr_linear_create(cfg: LinearConfig, device: int = 0) -> int:
    h, c = ctypes.c_void_p(), cfg.c()
    _check(load_library().hcgr_linear_create(ctypes.byref(c), int(device), ctypes.byref(h)), "hcgr_linear_create")
    return h.value


def hcgr_linear_destroy(handle: int) -> None:
    load_library().hcgr_linear_destroy(handle)


def hcgr_linear_quantize(handle, x, *args, stream=None, check: bool = True) -> int:
    """(x, ld_x, M, q, ld_q, q_scale)."""
    return _call("hcgr_linear_quantize", handle, _quantize_args(x, *args), stream, x, check)


def hcgr_linear_forward(handle, q, *args, stream=None, check: bool = True) -> int:
    """(q, ld_q, q_scale, w, ld_w, w_scale, bias, M, out, ld_out)."""
    return _call("hcgr_linear_forward", handle, _linear_args(q, *args), stream, q, check)


def hcgr_validate_linear_quantize(cfg: LinearConfig, *args) -> int:
    return _validate("hcgr_validate_linear_quantize", cfg, _quantize_args(*args))


def hcgr_validate_linear_forward(cfg: LinearConfig, *args) -> int:
    return _validate("hcgr_validate_linear_forward", cfg, _linear_args(*args))


def new_workspace(nbytes: int, device: int = 0):
    """A zero-filled device workspace of at least nbytes (the counter bytes at
    its start must be zero before the first call that uses it)."""
    import torch
    return torch.zeros(max(int(nbytes), HCGR_WORKSPACE_COUNTER_BYTES), dtype=torch.uint8, device=f"cuda:{device}")


# ------------------------------------------------------------ convenience --
class HCGR:
    """Handle + torch-allocated outputs/workspace around ``hcgr_forward``."""

    def __init__(self, cfg: Config = Config(), device: int = 0, plan_table=None):
        """``plan_table``: a tuned table (list of entries, or the path of a JSON
        file written by ``skinny_gemm_hcgr_amd.tune``), "shipped" for the table
        shipped with the package for cfg (the heuristic if there is none), or
        None for the heuristic."""
        self.cfg = cfg
        self.device = device
        self.handle = hcgr_create(cfg, device)
        self._ws = None
        if plan_table == "shipped":
            plan_table = shipped_plan_table(cfg)
        if plan_table is not None:
            self.set_plan_table(plan_table)

    def set_plan_table(self, table):
        if isinstance(table, str):
            table = load_plan_table(table, self.cfg)
        hcgr_set_plan_table(self.handle, table)
        self.table = list(table)
        self._ws = None  # the workspace bound may change

    def set_wait_polls(self, polls: int):
        hcgr_set_wait_polls(self.handle, polls)

    def describe(self, M: int) -> str:
        return hcgr_plan_lookup(self.cfg, getattr(self, "table", []), M)[1]

    def close(self):
        if self.handle:
            hcgr_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace(self, M: int):
        """A workspace for M tokens, zero-filled when allocated (the library
        keeps its counter bytes zero afterwards)."""
        n = hcgr_workspace_size(self.handle, M)
        if self._ws is None or self._ws.numel() < n:
            self._ws = new_workspace(n, self.device)
        return self._ws

    def alloc_outputs(self, M: int, ld_inj_next: int | None = None):
        import torch
        c = self.cfg
        dev = f"cuda:{self.device}"
        ld = c.hc if ld_inj_next is None else ld_inj_next
        packed = torch.zeros((M, ld), dtype=torch.bfloat16, device=dev)
        return {"R2": torch.empty((M, c.k), dtype=torch.bfloat16, device=dev),
                "rrms": torch.empty((M, c.hc), dtype=torch.float32, device=dev),
                "inj_next_buf": packed, "inj_next": packed[:, :c.hc], "ld_inj_next": ld,
                "x": torch.empty((M, c.hs), dtype=torch.bfloat16, device=dev)}

    def combine(self, R, y, inj, *, ld_inj: int | None = None, R2=None, stream=None):
        import torch
        M = R.shape[0]
        if R2 is None:
            R2 = torch.empty((M, self.cfg.k), dtype=torch.bfloat16, device=R.device)
        ld = inj.stride(0) if ld_inj is None else ld_inj
        hcgr_combine(self.handle, R, y, inj, ld, M, R2, stream)
        return R2

    def mix(self, R, wnorm, wd, wi, wu, *, out: dict | None = None, workspace=None, stream=None) -> dict:
        M = R.shape[0]
        if out is None:
            out = self.alloc_outputs(M)
        ws = self.workspace(M) if workspace is None else workspace
        hcgr_mix(self.handle, R, wnorm, wd, wi, wu, M, out["rrms"], out["inj_next"], out["ld_inj_next"],
                 out["x"], ws, ws.numel(), stream)
        return out

    def forward(self, R, y, inj, wnorm, wd, wi, wu, *, ld_inj: int | None = None, out: dict | None = None,
                workspace=None, stream=None) -> dict:
        M = R.shape[0]
        if out is None:
            out = self.alloc_outputs(M)
        ws = self.workspace(M) if workspace is None else workspace
        ld = inj.stride(0) if ld_inj is None else ld_inj
        hcgr_forward(self.handle, R, y, inj, ld, wnorm, wd, wi, wu, M, out["R2"], out["rrms"],
                     out["inj_next"], out["ld_inj_next"], out["x"], ws, ws.numel(), stream)
        return out


def torch_dtype(dtype: int):
    """The torch type of an HCGR_BF16, HCGR_FP16 or HCGR_FP32 configuration."""
    import torch
    return {HCGR_BF16: torch.bfloat16, HCGR_FP16: torch.float16, HCGR_FP32: torch.float32}[dtype]


def _round16(n: int) -> int:
    return (n + 15) // 16 * 16


class _Op:
    """What ``Block`` and ``Int8Linear`` share: the handle, argument checks (a
    tensor of another type, shape or device raises ValueError before any
    launch) and outputs that may be used on another stream than torch's."""

    def __init__(self, cfg, device: int, create, destroy):
        import torch
        self.cfg, self.device = cfg, int(device)
        self._destroy = destroy
        self.handle = create(cfg, self.device)
        self.dtype = torch_dtype(cfg.dtype)
        self._torch = torch
        self._f32, self._i8 = torch.float32, torch.int8
        self._lib = load_library()
        # torch's current stream as a raw hipStream_t, without the stream object where torch offers that
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._current = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)

    def close(self):
        if getattr(self, "handle", None):
            self._destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _bad(self, name, t, want):
        got = f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}" if hasattr(t, "dtype") else repr(t)
        raise ValueError(f"{name}: expected {want} on cuda:{self.device}, got {got}")

    def _dense(self, name, t, dtype, shape):
        """Address of a contiguous tensor of this type and shape, None for None."""
        if t is None:
            return None
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self.device or not t.is_contiguous():
            self._bad(name, t, f"contiguous {dtype} {tuple(shape)}")
        return t.data_ptr()

    def _rows(self, name, t, dtype, m, cols):
        """Address and row pitch of a matrix whose rows are contiguous."""
        if t.dtype is not dtype or t.shape != (m, cols) or t.get_device() != self.device or \
                (cols > 1 and t.stride(1) != 1):
            self._bad(name, t, f"{dtype} {(m, cols)} with contiguous rows")
        return t.data_ptr(), t.stride(0) if m > 1 else cols

    def _rows8(self, name, t, m, cols):
        """The same for int8 rows, which are read in whole 16-byte pieces."""
        p, ld = self._rows(name, t, self._i8, m, cols)
        if m == 1:
            ld = _round16(cols)
        if m and cols % 16 and t.untyped_storage().nbytes() < t.storage_offset() + (m - 1) * ld + _round16(cols):
            raise ValueError(f"{name}: rows of {cols} int8 need a pitch of whole 16-byte pieces "
                             "(alloc_quantized makes such rows)")
        return p, ld

    def _raw(self, stream):
        if stream is None:
            return self._current(self.device)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _on(self, stream, alloc, *args, **kw):
        """alloc(...) for a call on `stream`: from that stream's memory, so that
        nothing still running elsewhere holds it, and kept until torch's
        current stream, which may read the results, is done with it."""
        cuda = self._torch.cuda
        if stream is None:
            return alloc(*args, **kw)
        s = cuda.ExternalStream(stream, device=self.device) if isinstance(stream, int) else stream
        now = cuda.current_stream(self.device)
        if s == now:
            return alloc(*args, **kw)
        with cuda.stream(s):
            made = alloc(*args, **kw)
        for t in made.values() if isinstance(made, dict) else made if isinstance(made, tuple) else (made,):
            t.record_stream(now)
        return made

    def _empty(self, shape, dtype):
        return self._torch.empty(shape, dtype=dtype, device=f"cuda:{self.device}")

    def _quantized(self, m, cols):
        """int8 [m, cols] at a pitch of whole 16-byte pieces, and its scales."""
        return self._empty((m, _round16(cols)), self._i8)[:, :cols], self._empty((m,), self._f32)


class Block(_Op):
    """The norms around a block and their gradients (``hcgr_block_*``), with
    outputs and workspaces allocated by torch. ``out`` takes a dict of an
    ``alloc_*`` method (or of an earlier call) and is returned."""

    def __init__(self, cfg: BlockConfig = BlockConfig(), device: int = 0):
        super().__init__(cfg, device, hcgr_block_create, hcgr_block_destroy)
        self._ws_bytes = {}  # workspace bytes by token count

    def alloc_norm(self, M: int, *, quantize: bool = False, keep: bool = False) -> dict:
        """``quantize``: q and q_scale in place of x; ``keep``: x as well."""
        f32, hs = self._f32, self.cfg.hs
        out = {"rrms": self._empty((M,), f32)}
        if quantize:
            out["q"], out["q_scale"] = self._quantized(M, hs)
        if keep or not quantize:
            out["x"] = self._empty((M, hs), self.dtype)
        return out

    def _weight_grad(self, M):
        """float32 [HS]. A call on no tokens writes nothing: their sum is zero."""
        dw = self._empty((self.cfg.hs,), self._f32)
        return dw if M else dw.zero_()

    def alloc_norm_bwd(self, M: int) -> dict:
        return {"dx": self._empty((M, self.cfg.hs), self.dtype), "dw": self._weight_grad(M)}

    def alloc_residual(self, M: int, *, norm: bool = True, quantize: bool = False, keep: bool = False) -> dict:
        """``norm``: the next norm is wanted (w_pre is given)."""
        out = self.alloc_norm(M, quantize=quantize, keep=keep) if norm else {}
        out["rrms"] = self._empty((M, 2), self._f32)
        out["R2"] = self._empty((M, self.cfg.k), self.dtype)
        return out

    def alloc_residual_bwd(self, M: int, *, gates: bool = True, post: bool = True, pre: bool = True) -> dict:
        c = self.cfg
        out = {"dR": self._empty((M, c.k), self.dtype), "dy": self._empty((M, c.hs), self.dtype)}
        if gates:
            out["dinj"] = self._empty((M, c.hc), self.dtype)
        if post:
            out["dw_post"] = self._weight_grad(M)
        if pre:
            out["dw_pre"] = self._weight_grad(M)
        return out

    def workspace(self, M: int):
        """A workspace for the backward entry points (no initialisation needed)."""
        n = self._ws_bytes.get(M)
        if n is None:
            if len(self._ws_bytes) >= 1024:
                self._ws_bytes.clear()
            n = self._ws_bytes[M] = hcgr_block_workspace_size(self.handle, M)
        return self._empty((n,), self._torch.uint8)

    def _norm_outputs(self, out, M, quantize):
        hs, f32 = self.cfg.hs, self._f32
        if quantize and out.get("q") is None:
            raise ValueError("quantize: out has no q (alloc_norm or alloc_residual with quantize=True makes it)")
        x = self._dense("x", out.get("x"), self.dtype, (M, hs))
        q, ld_q, qs = out.get("q"), 0, None
        if q is not None:
            q, ld_q = self._rows8("q", q, M, hs)
            qs = self._dense("q_scale", out["q_scale"], f32, (M,))
        return x, q, ld_q, qs

    def _ws(self, workspace, M, stream):
        if workspace is None:
            return self._on(stream, self.workspace, M)
        if workspace.dtype is not self._torch.uint8 or workspace.get_device() != self.device or \
                not workspace.is_contiguous():
            self._bad("workspace", workspace, "contiguous uint8")
        return workspace

    def norm(self, x, w, *, quantize: bool = False, out: dict | None = None, stream=None) -> dict:
        """x [M, HS] (rows may be strided) -> x or (q, q_scale), and rrms. With
        ``out`` what it holds of x and q is written; ``quantize`` then asks for q."""
        M, hs = x.shape[0], self.cfg.hs
        px, ld_x = self._rows("x", x, self.dtype, M, hs)
        if out is None:
            out = self._on(stream, self.alloc_norm, M, quantize=quantize)
        xn, q, ld_q, qs = self._norm_outputs(out, M, quantize)
        _check(self._lib.hcgr_block_norm(
            self.handle, px, ld_x, self._dense("w", w, self.dtype, (hs,)), M, xn, q, ld_q, qs,
            self._dense("rrms", out.get("rrms"), self._f32, (M,)), self._raw(stream)), "hcgr_block_norm")
        return out

    def norm_bwd(self, x, w, rrms, dxn, *, out: dict | None = None, workspace=None, stream=None) -> dict:
        """Gradients dx [M, HS] and dw [HS] (float32, summed over the tokens) of
        ``norm``. With no tokens, dw of a given ``out`` stays as it is."""
        M, hs, f32 = x.shape[0], self.cfg.hs, self._f32
        px, ld_x = self._rows("x", x, self.dtype, M, hs)
        if out is None:
            out = self._on(stream, self.alloc_norm_bwd, M)
        ws = self._ws(workspace, M, stream)
        _check(self._lib.hcgr_block_norm_bwd(
            self.handle, px, ld_x, self._dense("w", w, self.dtype, (hs,)), self._dense("rrms", rrms, f32, (M,)),
            self._dense("dxn", dxn, self.dtype, (M, hs)), M, self._dense("dx", out.get("dx"), self.dtype, (M, hs)),
            self._dense("dw", out.get("dw"), f32, (hs,)), ws.data_ptr(), ws.numel(), self._raw(stream)),
            "hcgr_block_norm_bwd")
        return out

    def residual(self, R, y, inj=None, w_post=None, w_pre=None, *, quantize: bool = False, out: dict | None = None,
                 stream=None) -> dict:
        """R [M, HC*HS], y [M, HS], inj [M, HC] (rows of y and inj may be strided)
        -> R2, rrms, and with w_pre the next norm as x or (q, q_scale); ``out``
        and ``quantize`` as in ``norm``."""
        c, dt = self.cfg, self.dtype
        if quantize and w_pre is None:
            raise ValueError("quantize: there is no next norm (w_pre is None)")
        M, hs, k = R.shape[0], c.hs, c.hc * c.hs
        py, ld_y = self._rows("y", y, dt, M, hs)
        pi, ld_i = self._rows("inj", inj, dt, M, c.hc) if inj is not None else (None, 0)
        if out is None:
            out = self._on(stream, self.alloc_residual, M, norm=w_pre is not None, quantize=quantize)
        x, q, ld_q, qs = self._norm_outputs(out, M, quantize)
        _check(self._lib.hcgr_block_residual(
            self.handle, self._dense("R", R, dt, (M, k)), py, ld_y, pi, ld_i,
            self._dense("w_post", w_post, dt, (hs,)), self._dense("w_pre", w_pre, dt, (hs,)), M,
            self._dense("R2", out["R2"], dt, (M, k)), x, q, ld_q, qs,
            self._dense("rrms", out.get("rrms"), self._f32, (M, 2)), self._raw(stream)),
            "hcgr_block_residual")
        return out

    def residual_bwd(self, R, y, inj, w_post, w_pre, rrms, dR2, dx, *, out: dict | None = None, workspace=None,
                     stream=None) -> dict:
        """Gradients dR, dy, dinj, dw_post and dw_pre (those whose input is
        given) of ``residual`` from dR2 [M, HC*HS] and dx [M, HS]."""
        c, dt, f32 = self.cfg, self.dtype, self._f32
        M, hs, k = R.shape[0], c.hs, c.hc * c.hs
        py, ld_y = self._rows("y", y, dt, M, hs)
        pi, ld_i = self._rows("inj", inj, dt, M, c.hc) if inj is not None else (None, 0)
        if out is None:
            out = self._on(stream, self.alloc_residual_bwd, M, gates=inj is not None, post=w_post is not None,
                           pre=w_pre is not None)
        di, ld_di = out.get("dinj"), 0
        if di is not None:
            di, ld_di = self._rows("dinj", di, dt, M, c.hc)
        ws = self._ws(workspace, M, stream)
        _check(self._lib.hcgr_block_residual_bwd(
            self.handle, self._dense("R", R, dt, (M, k)), py, ld_y, pi, ld_i,
            self._dense("w_post", w_post, dt, (hs,)), self._dense("w_pre", w_pre, dt, (hs,)),
            self._dense("rrms", rrms, f32, (M, 2)), self._dense("dR2", dR2, dt, (M, k)),
            self._dense("dx", dx, dt, (M, hs)), M, self._dense("dR", out["dR"], dt, (M, k)),
            self._dense("dy", out["dy"], dt, (M, hs)), di, ld_di, self._dense("dw_post", out.get("dw_post"), f32, (hs,)),
            self._dense("dw_pre", out.get("dw_pre"), f32, (hs,)), ws.data_ptr(), ws.numel(), self._raw(stream)),
            "hcgr_block_residual_bwd")
        return out


class Int8Linear(_Op):
    """An 8-bit linear layer [K] -> [N] (``hcgr_linear_*``). Weights are the
    caller's: int8 [N, K] with a float32 scale for each output channel, as
    ``quantize`` makes them from a float matrix."""

    def __init__(self, cfg: LinearConfig, device: int = 0):
        super().__init__(cfg, device, hcgr_linear_create, hcgr_linear_destroy)

    def alloc_quantized(self, M: int):
        """(q, q_scale) for M rows of K values, q at a pitch of whole 16-byte pieces."""
        return self._quantized(M, self.cfg.k)

    def alloc_output(self, M: int):
        return self._empty((M, self.cfg.n), self.dtype)

    def quantize(self, x, *, out=None, stream=None):
        """Rows [M, K] (tokens, or a weight's output channels) -> (q, q_scale)."""
        M, k = x.shape[0], self.cfg.k
        px, ld_x = self._rows("x", x, self.dtype, M, k)
        if out is None:
            out = self._on(stream, self.alloc_quantized, M)
        q, ld_q = self._rows8("q", out[0], M, k)
        _check(self._lib.hcgr_linear_quantize(
            self.handle, px, ld_x, M, q, ld_q, self._dense("q_scale", out[1], self._f32, (M,)),
            self._raw(stream)), "hcgr_linear_quantize")
        return out

    def forward(self, q, q_scale, w, w_scale, bias=None, *, out=None, stream=None):
        """out [M, N] from tokens q int8 [M, K] and weights w int8 [N, K]."""
        c, f32, M = self.cfg, self._f32, q.shape[0]
        pq, ld_q = self._rows8("q", q, M, c.k)
        pw, ld_w = self._rows8("w", w, c.n, c.k)
        if out is None:
            out = self._on(stream, self.alloc_output, M)
        po, ld_o = self._rows("out", out, self.dtype, M, c.n)
        _check(self._lib.hcgr_linear_forward(
            self.handle, pq, ld_q, self._dense("q_scale", q_scale, f32, (M,)), pw, ld_w,
            self._dense("w_scale", w_scale, f32, (c.n,)), self._dense("bias", bias, self.dtype, (c.n,)), M, po, ld_o,
            self._raw(stream)), "hcgr_linear_forward")
        return out
