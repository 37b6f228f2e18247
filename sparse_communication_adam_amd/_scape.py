"""ctypes binding of libscape (include/scape.h), same names as the C ABI.

Argument marshalling only: every step of the SCAPE path runs in the HIP
kernels of libscape.so.  Device arrays are torch tensors (PyTorch supplies
device memory and streams); host arrays are Python sequences.  If the
library is not built, every call raises - there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
# SCAPE_LIB selects another build of the library (the host-sanitizer build
# the CPU suite checks its host paths with).
LIB_PATH = os.environ.get("SCAPE_LIB") or os.path.join(HERE, "libscape.so")

SCAPE_OK = 0
SCAPE_ERR_INVALID_ARG = -1
SCAPE_ERR_SHAPE = -2
SCAPE_ERR_ALIGN = -3
SCAPE_ERR_OOM = -4
SCAPE_ERR_HIP = -5
SCAPE_ERR_STATE = -6
SCAPE_MAX_WORKERS = 32
PHASES = ("ef_compact", "reduce_update", "mask_select", "mask_index")

_ERR_NAMES = {-1: "INVALID_ARG", -2: "SHAPE", -3: "ALIGN", -4: "OOM", -5: "HIP", -6: "STATE"}

_lib = None


class ScapeError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"SCAPE_ERR_{_ERR_NAMES.get(code, code)}: {message}")
        self.code = code


class _Config(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("layer_numel", ctypes.POINTER(ctypes.c_int64)),
                ("workers", ctypes.c_int32), ("owner_shards", ctypes.c_int32), ("beta1", ctypes.c_float),
                ("beta2", ctypes.c_float), ("lr", ctypes.c_float), ("eps", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("keep_num", ctypes.c_uint32), ("keep_den", ctypes.c_uint32)]


class _Teacher(ctypes.Structure):
    _fields_ = [("val", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("idx", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("k", ctypes.c_int32)]


class _Mask(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("block_prefix", ctypes.c_void_p)]


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        f32 = ctypes.c_float
        cfgp, maskp, teachp = ctypes.POINTER(_Config), ctypes.POINTER(_Mask), ctypes.POINTER(_Teacher)
        sig = {
            "scape_version": [vp, vp],
            "scape_layout": [cfgp, vp, vp, vp, vp, vp],
            "scape_owner_map": [cfgp, i32, vp],
            "scape_init": [cfgp, ctypes.POINTER(vp)],
            "scape_destroy": [vp],
            "scape_workspace_bytes": [vp, vp],
            "scape_selection_flags": [vp, vp],
            "scape_set_select_path": [vp, i32],
            "scape_set_update_in_dense_pass": [vp, i32],
            "scape_set_offload_path": [vp, i32],
            "scape_step": [vp, vp, vp, vp, vp, vp, maskp, maskp, vp, vp, vp],
            "scape_step_offload": [vp, vp, vp, vp, vp, vp, maskp, maskp, vp, vp, vp],
            "scape_step_interleaved": [vp, vp, vp, vp, vp, maskp, maskp, vp, vp, vp],
            "scape_dense_step": [vp, vp, vp, vp, vp, vp],
            "scape_dense_step_interleaved": [vp, vp, vp, vp, vp, vp],
            "scape_mask_union_add": [vp, vp, vp, vp],
            "scape_mask_build": [vp, vp, i32, i32, maskp, vp],
            "scape_mask_index": [vp, maskp, vp],
            "scape_mask_index_static": [vp, i64, vp, i64, vp, vp],
            "scape_pack": [vp, i64, vp, vp],
            "scape_unpack": [vp, i64, vp, vp],
            "scape_reduce_sparse": [vp, i32, i64, vp, vp],
            "scape_profile_enable": [vp, i32],
            "scape_profile_read": [vp, vp, vp],
            "scape_copy_probe": [vp, vp, ctypes.c_uint64, vp],
            "scape_stream_probe": [vp, vp, i32, vp, vp, i32, ctypes.c_uint64, vp],
            "scape_topk_rows": [vp, i32, i64, i64, i64, i32, f32, vp, vp, vp, vp, i64, vp],
            "scape_topk_rows_workspace": [i32, i64, i64, i32, vp],
            "scape_distill_forward": [vp, i32, i64, i64, i64, teachp, f32, vp, vp, vp, vp, i64, vp, i64, vp],
            "scape_distill_workspace": [i32, i64, i64, i32, vp],
            "scape_distill_loss_workspace": [i32, i64, i64, i32, vp],
            "scape_distill_backward": [vp, i32, i64, i64, i64, teachp, f32, vp, vp, vp, vp, i64, vp],
            "scape_balance_forward": [vp, i32, i64, i32, i64, vp, i32, vp, i32, vp, i32, f32, vp, vp, vp, vp, vp, i64,
                                      vp],
            "scape_balance_workspace": [i64, i32, i32, vp],
            "scape_balance_loss": [vp, vp, vp, i32, i32, i32, f32, vp, vp],
            "scape_balance_backward": [vp, i32, i64, i32, i64, i32, vp, i32, vp, i32, f32, vp, vp, vp, vp, i64, vp],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.scape_last_error.argtypes = []
        L.scape_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def scape_last_error() -> str:
    return lib().scape_last_error().decode()


def _check(rc: int) -> None:
    if rc != SCAPE_OK:
        raise ScapeError(rc, scape_last_error())


# ----------------------------------------------------------------------------
# configuration and layout


@dataclass
class ScapeConfig:
    layer_numel: Sequence[int]
    workers: int
    keep_num: int
    keep_den: int
    owner_shards: int = 0
    beta1: float = 0.9
    beta2: float = 0.95
    lr: float = 1e-3
    eps: float = 1e-8
    weight_decay: float = 0.0

    def _c(self):
        arr = (ctypes.c_int64 * max(len(self.layer_numel), 1))(*[int(n) for n in self.layer_numel])
        c = _Config(len(self.layer_numel), arr, self.workers, self.owner_shards, self.beta1, self.beta2, self.lr,
                    self.eps, self.weight_decay, self.keep_num, self.keep_den)
        c._keep = arr  # keep the array alive with the struct
        return c


@dataclass
class Layout:
    n_pad: int
    k_total: int
    layer_offset: list
    layer_k: list
    layer_owner: list

    @property
    def n_words(self) -> int:
        return self.n_pad // 64


def scape_version():
    a, b = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().scape_version(ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def scape_layout(cfg: ScapeConfig) -> Layout:
    c = cfg._c()
    L = len(cfg.layer_numel)
    n_pad, k_total = ctypes.c_int64(), ctypes.c_int64()
    off = (ctypes.c_int64 * max(L, 1))()
    kk = (ctypes.c_int64 * max(L, 1))()
    own = (ctypes.c_int32 * max(L, 1))()
    _check(lib().scape_layout(ctypes.byref(c), ctypes.byref(n_pad), ctypes.byref(k_total), off, kk, own))
    return Layout(n_pad.value, k_total.value, list(off)[:L], list(kk)[:L], list(own)[:L])


def scape_owner_map(cfg: ScapeConfig, num_shards: int) -> list:
    c = cfg._c()
    L = len(cfg.layer_numel)
    own = (ctypes.c_int32 * max(L, 1))()
    _check(lib().scape_owner_map(ctypes.byref(c), num_shards, own))
    return list(own)[:L]


# ----------------------------------------------------------------------------
# device marshalling


def _stream(stream) -> int:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _shape(t, dtype, numel: Optional[int], name: str) -> None:
    """Check a tensor's type, dtype, layout and length."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} must have dtype {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")


def _dev(t, dtype, numel: Optional[int], name: str) -> int:
    """Device pointer of a torch tensor, after checking its type, dtype,
    layout, length and device (all before anything reaches the library)."""
    _shape(t, dtype, numel, name)
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    return t.data_ptr()


def _host(t, dtype, numel: Optional[int], name: str) -> int:
    """A pinned host tensor (the offloaded residuals)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cpu":
        raise ValueError(f"{name} must be in host memory (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_pinned():
        raise ValueError(f"{name} must be pinned host memory (pin_memory=True)")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def _ptr_array(ptrs) -> ctypes.Array:
    return (ctypes.c_void_p * max(len(ptrs), 1))(*ptrs)


class Mask:
    """A mask in the library layout, backed by three device tensors."""

    def __init__(self, bits, idx, block_prefix):
        self.bits, self.idx, self.block_prefix = bits, idx, block_prefix

    def _c(self, layout: "Layout", need_index: bool = True) -> _Mask:
        """The C struct, after checking each array against `layout`: bits
        needs n_pad/64 words, idx k_total entries and block_prefix
        n_pad/64 + 1 (idx and block_prefix only when the entry point uses
        them).  Every length is checked before any device check."""
        import torch
        nw = layout.n_words
        arrs = [(self.bits, (torch.int64,), nw, "mask.bits")]
        if need_index or self.idx is not None:
            arrs.append((self.idx, (torch.int32,), max(layout.k_total, 1), "mask.idx"))
        if need_index or self.block_prefix is not None:
            arrs.append((self.block_prefix, (torch.int32,), nw + 1, "mask.block_prefix"))
        for a in arrs:
            _shape(*a)
        ptrs = {name: _dev(*a[:3], name) for *a, name in arrs}
        return _Mask(ptrs["mask.bits"], ptrs.get("mask.idx"), ptrs.get("mask.block_prefix"))

    def clear(self):
        self.bits.zero_()
        self.idx.zero_()
        self.block_prefix.zero_()


def alloc_mask(layout: Layout, device="cuda") -> Mask:
    """An all-zero mask sized for `layout` (bits int64, idx/block_prefix int32)."""
    import torch
    return Mask(torch.zeros(layout.n_words, dtype=torch.int64, device=device),
                torch.zeros(max(layout.k_total, 1), dtype=torch.int32, device=device),
                torch.zeros(layout.n_words + 1, dtype=torch.int32, device=device))


# ----------------------------------------------------------------------------
# context and entry points


class Context:
    def __init__(self, cfg: ScapeConfig):
        self._h = None
        self.cfg = cfg
        self.layout = scape_layout(cfg)
        h = ctypes.c_void_p()
        c = cfg._c()
        _check(lib().scape_init(ctypes.byref(c), ctypes.byref(h)))
        self._h = h

    @property
    def handle(self):
        if self._h is None:
            raise ScapeError(SCAPE_ERR_STATE, "context destroyed")
        return self._h

    def destroy(self):
        if self._h is not None:
            _check(lib().scape_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def scape_init(cfg: ScapeConfig) -> Context:
    return Context(cfg)


def scape_destroy(ctx: Context) -> None:
    ctx.destroy()


def scape_workspace_bytes(ctx: Context) -> int:
    """Device memory the context's workspaces hold, in bytes."""
    b = ctypes.c_int64()
    _check(lib().scape_workspace_bytes(ctx.handle, ctypes.byref(b)))
    return b.value


SELECT_EXACT_HISTOGRAM = 1
SELECT_KEY_PASSES = 2


def scape_selection_flags(ctx: Context) -> int:
    """Fallbacks the last mask selection took (waits for the device): bit 0
    exact histogram, bit 1 passes over the keys (SELECT_* constants)."""
    f = ctypes.c_uint32()
    _check(lib().scape_selection_flags(ctx.handle, ctypes.byref(f)))
    return f.value


SELECT_PATH_AUTO = 0
SELECT_PATH_SAMPLED = 1
SELECT_PATH_COMPACT = 2


def scape_set_select_path(ctx: Context, path: int) -> None:
    """How the context selects masks from the next call on (SELECT_PATH_*):
    the sampled multi-pass path, the two-launch compact path, or AUTO (compact
    where every layer of the range has at most 2^22 elements)."""
    _check(lib().scape_set_select_path(ctx.handle, int(path)))


OFFLOAD_PATH_AUTO = 0
OFFLOAD_PATH_STAGED = 1


def scape_set_offload_path(ctx: Context, path: int) -> None:
    """From the next call on, move scape_step_offload's residuals by the
    dense pass itself over PCIe where they are pinned, mapped host memory
    (OFFLOAD_PATH_AUTO, the default), or always through the staging
    slots (OFFLOAD_PATH_STAGED)."""
    _check(lib().scape_set_offload_path(ctx.handle, int(path)))


def scape_set_update_in_dense_pass(ctx: Context, on: bool) -> None:
    """From the next call on, let the dense pass finish the reduction and the
    update at the mask's positions where the residuals are on the device (the
    default), or make the update a pass of its own (on = False)."""
    _check(lib().scape_set_update_in_dense_pass(ctx.handle, int(bool(on))))


def scape_step(ctx: Context, x, m, v, r: Sequence, g: Sequence, cur: Mask, next: Mask, sparse_bufs: Sequence,
               key_out=None, stream=None) -> None:
    import torch
    n, W, k = ctx.layout.n_pad, ctx.cfg.workers, ctx.layout.k_total
    if len(r) != W or len(g) != W or len(sparse_bufs) != W:
        raise ValueError(f"r, g and sparse_bufs need {W} entries each")
    xp = _dev(x, torch.float32, n, "x")
    mp = _dev(m, torch.float32, n, "m")
    vp = _dev(v, torch.float32, n, "v")
    rp = _ptr_array([_dev(t, torch.float32, n, f"r[{i}]") for i, t in enumerate(r)])
    gp = _ptr_array([_dev(t, (torch.int16, torch.bfloat16, torch.uint16), n, f"g[{i}]") for i, t in enumerate(g)])
    bp = _ptr_array([_dev(t, torch.float32, k, f"sparse_bufs[{i}]") for i, t in enumerate(sparse_bufs)])
    kp = _dev(key_out, torch.int32, n, "key_out") if key_out is not None else None
    c, nx = cur._c(ctx.layout), next._c(ctx.layout)
    _check(lib().scape_step(ctx.handle, xp, mp, vp, rp, gp, ctypes.byref(c), ctypes.byref(nx), bp, kp,
                            _stream(stream)))


def scape_step_interleaved(ctx: Context, xv, m, r_il, g_il, cur: Mask, next: Mask, sparse_bufs: Sequence,
                           key_out=None, stream=None) -> None:
    """scape_step in the interleaved layout: xv holds (x, v) pairs (2*n_pad
    fp32), r_il (fp32) and g_il (bf16 bits) n_pad*W elements each, word w of
    worker i at [(w*W + i)*64, (w*W + i)*64 + 64)."""
    import torch
    n, W, k = ctx.layout.n_pad, ctx.cfg.workers, ctx.layout.k_total
    if len(sparse_bufs) != W:
        raise ValueError(f"sparse_bufs needs {W} entries")
    xp = _dev(xv, torch.float32, 2 * n, "xv")
    mp = _dev(m, torch.float32, n, "m")
    rp = _dev(r_il, torch.float32, n * W, "r_il")
    gp = _dev(g_il, (torch.int16, torch.bfloat16, torch.uint16), n * W, "g_il")
    bp = _ptr_array([_dev(t, torch.float32, k, f"sparse_bufs[{i}]") for i, t in enumerate(sparse_bufs)])
    kp = _dev(key_out, torch.int32, n, "key_out") if key_out is not None else None
    c, nx = cur._c(ctx.layout), next._c(ctx.layout)
    _check(lib().scape_step_interleaved(ctx.handle, xp, mp, rp, gp, ctypes.byref(c), ctypes.byref(nx), bp, kp,
                                        _stream(stream)))


def scape_step_offload(ctx: Context, x, m, v, r_host: Sequence, g: Sequence, cur: Mask, next: Mask,
                       sparse_bufs: Sequence, key_out=None, stream=None) -> None:
    """scape_step with the residuals in pinned host tensors."""
    import torch
    n, W, k = ctx.layout.n_pad, ctx.cfg.workers, ctx.layout.k_total
    if len(r_host) != W or len(g) != W or len(sparse_bufs) != W:
        raise ValueError(f"r_host, g and sparse_bufs need {W} entries each")
    xp = _dev(x, torch.float32, n, "x")
    mp = _dev(m, torch.float32, n, "m")
    vp = _dev(v, torch.float32, n, "v")
    rp = _ptr_array([_host(t, torch.float32, n, f"r_host[{i}]") for i, t in enumerate(r_host)])
    gp = _ptr_array([_dev(t, (torch.int16, torch.bfloat16, torch.uint16), n, f"g[{i}]") for i, t in enumerate(g)])
    bp = _ptr_array([_dev(t, torch.float32, k, f"sparse_bufs[{i}]") for i, t in enumerate(sparse_bufs)])
    kp = _dev(key_out, torch.int32, n, "key_out") if key_out is not None else None
    c, nx = cur._c(ctx.layout), next._c(ctx.layout)
    _check(lib().scape_step_offload(ctx.handle, xp, mp, vp, rp, gp, ctypes.byref(c), ctypes.byref(nx), bp, kp,
                                    _stream(stream)))


def scape_dense_step(ctx: Context, x, m, v, g: Sequence, stream=None) -> None:
    import torch
    n, W = ctx.layout.n_pad, ctx.cfg.workers
    if len(g) != W:
        raise ValueError(f"g needs {W} entries")
    xp = _dev(x, torch.float32, n, "x")
    mp = _dev(m, torch.float32, n, "m")
    vp = _dev(v, torch.float32, n, "v")
    gp = _ptr_array([_dev(t, (torch.int16, torch.bfloat16, torch.uint16), n, f"g[{i}]") for i, t in enumerate(g)])
    _check(lib().scape_dense_step(ctx.handle, xp, mp, vp, gp, _stream(stream)))


def scape_dense_step_interleaved(ctx: Context, x, m, v, g_il, stream=None) -> None:
    """scape_dense_step with the gradients in the worker-interleaved layout."""
    import torch
    n, W = ctx.layout.n_pad, ctx.cfg.workers
    xp = _dev(x, torch.float32, n, "x")
    mp = _dev(m, torch.float32, n, "m")
    vp = _dev(v, torch.float32, n, "v")
    gp = _dev(g_il, (torch.int16, torch.bfloat16, torch.uint16), n * W, "g_il")
    _check(lib().scape_dense_step_interleaved(ctx.handle, xp, mp, vp, gp, _stream(stream)))


def interleaved_view(t, W: int):
    """Worker i's elements of a worker-interleaved array `t` (n_pad*W) as a
    strided (n_pad/64, 64) view; .reshape(-1) copies them out flat."""
    return t.view(-1, W, 64)


def scape_mask_build(ctx: Context, mtilde, out: Mask, num_shards: int = 0, shard: int = -1, stream=None) -> None:
    import torch
    mp = _dev(mtilde, torch.float32, ctx.layout.n_pad, "mtilde")
    o = out._c(ctx.layout, need_index=num_shards <= 0 or shard < 0)
    _check(lib().scape_mask_build(ctx.handle, mp, num_shards, shard, ctypes.byref(o), _stream(stream)))


def scape_mask_union_add(ctx: Context, mtilde, acc_bits, stream=None) -> None:
    import torch
    mp = _dev(mtilde, torch.float32, ctx.layout.n_pad, "mtilde")
    ap = _dev(acc_bits, torch.int64, ctx.layout.n_pad // 64, "acc_bits")
    _check(lib().scape_mask_union_add(ctx.handle, mp, ap, _stream(stream)))


def scape_mask_index(ctx: Context, mask: Mask, stream=None) -> None:
    c = mask._c(ctx.layout)
    _check(lib().scape_mask_index(ctx.handle, ctypes.byref(c), _stream(stream)))


def scape_mask_index_static(bits, idx, block_prefix, n_words: Optional[int] = None, k_cap: Optional[int] = None,
                            stream=None) -> None:
    """idx and block_prefix of the mask in `bits` without a context or any
    allocation (the library's static scratch)."""
    import torch
    n_words = bits.numel() if n_words is None else int(n_words)
    k_cap = (idx.numel() if idx is not None else 0) if k_cap is None else int(k_cap)
    bp = _dev(bits, torch.int64, n_words, "bits")
    ip = _dev(idx, torch.int32, k_cap, "idx") if idx is not None else None
    pp = _dev(block_prefix, torch.int32, n_words + 1, "block_prefix")
    _check(lib().scape_mask_index_static(bp, n_words, ip, k_cap, pp, _stream(stream)))


def scape_pack(pred, bits, n: Optional[int] = None, stream=None) -> None:
    import torch
    n = pred.numel() if n is None else n
    pp = _dev(pred, (torch.uint8, torch.bool), n, "pred")
    bp = _dev(bits, torch.int64, (n + 63) // 64, "bits")
    _check(lib().scape_pack(pp, n, bp, _stream(stream)))


def scape_unpack(bits, pred, n: Optional[int] = None, stream=None) -> None:
    import torch
    n = pred.numel() if n is None else n
    bp = _dev(bits, torch.int64, (n + 63) // 64, "bits")
    pp = _dev(pred, (torch.uint8, torch.bool), n, "pred")
    _check(lib().scape_unpack(bp, n, pp, _stream(stream)))


def scape_reduce_sparse(bufs: Sequence, out, k: Optional[int] = None, stream=None) -> None:
    import torch
    k = out.numel() if k is None else k
    ptrs = _ptr_array([_dev(b, torch.float32, k, f"bufs[{i}]") for i, b in enumerate(bufs)])
    op = _dev(out, torch.float32, k, "out")
    _check(lib().scape_reduce_sparse(ptrs, len(bufs), k, op, _stream(stream)))


def scape_copy_probe(src, dst, nbytes: Optional[int] = None, stream=None) -> None:
    """Copy nbytes (default: all of src) from src to dst, both device tensors
    (16-byte aligned, nbytes a multiple of 16), with the library's plain
    stream-copy kernel."""
    import torch
    nbytes = src.numel() * src.element_size() if nbytes is None else int(nbytes)
    for t, name in ((src, "src"), (dst, "dst")):
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous device tensor")
        if t.numel() * t.element_size() < nbytes:
            raise ValueError(f"{name} is smaller than {nbytes} bytes")
    _check(lib().scape_copy_probe(src.data_ptr(), dst.data_ptr(), nbytes, _stream(stream)))


def scape_stream_probe(srcs: Sequence, src_widths: Sequence[int], dsts: Sequence, dst_widths: Sequence[int],
                       n_words: int, stream=None) -> None:
    """A pass that reads every tensor of srcs and writes every tensor of dsts
    over n_words 64-element words, width bytes per element (2, 4, 8 or 16)
    each, with no other work (scape_stream_probe in include/scape.h)."""
    import torch
    for t, w in list(zip(srcs, src_widths)) + list(zip(dsts, dst_widths)):
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or not t.is_contiguous():
            raise ValueError("arrays must be contiguous device tensors")
        if t.numel() * t.element_size() < int(n_words) * 64 * int(w):
            raise ValueError(f"an array of {t.numel() * t.element_size()} bytes is smaller than "
                             f"{n_words} words of width {w}")
    sw = (ctypes.c_uint32 * max(len(srcs), 1))(*[int(w) for w in src_widths])
    dw = (ctypes.c_uint32 * max(len(dsts), 1))(*[int(w) for w in dst_widths])
    _check(lib().scape_stream_probe(_ptr_array([t.data_ptr() for t in srcs]), sw, len(srcs),
                                    _ptr_array([t.data_ptr() for t in dsts]), dw, len(dsts), int(n_words),
                                    _stream(stream)))


def scape_profile_enable(ctx: Context, enable: bool = True) -> None:
    _check(lib().scape_profile_enable(ctx.handle, 1 if enable else 0))


def scape_profile_read(ctx: Context):
    """(dict phase -> summed ms, steps recorded)."""
    ms = (ctypes.c_double * 4)()
    steps = ctypes.c_int64()
    _check(lib().scape_profile_read(ctx.handle, ms, ctypes.byref(steps)))
    return dict(zip(PHASES, list(ms))), steps.value


# ----------------------------------------------------------------------------
# losses: row top-k, distillation from a teacher's top logits, router balance.
# No context; outputs and workspaces are the caller's tensors.


# These calls are short (a router's loss takes a few microseconds on the GPU),
# so their argument checks are made with one cheap query each.

_TORCH = None
_FLOATS = None
_WROTE = None


def _torch():
    global _TORCH, _FLOATS, _WROTE
    if _TORCH is None:
        import torch
        _TORCH = torch
        _WROTE = torch.autograd.graph.increment_version
        _FLOATS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    return _TORCH


def _dtype_id(dtype) -> int:
    did = _FLOATS.get(dtype)
    if did is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16 (got {dtype})")
    return did


def _matrix(t, name: str, like=None):
    """(pointer, dtype id, rows, cols, ld) of a 2-D tensor whose rows are
    contiguous; `like`: the tensor whose dtype and shape it must have."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions (got {t.dim()})")
    if like is not None and (t.dtype is not like.dtype or t.shape != like.shape):
        raise ValueError(f"{name} must have the logits' dtype and shape ({like.dtype}, {tuple(like.shape)})")
    did = _dtype_id(t.dtype)
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows (stride {step} between columns)")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"{name}: rows of {cols} columns overlap (stride {ld})")
    return t.data_ptr(), did, rows, cols, ld


def _array(t, dtype, numel: int, name: str):
    """Pointer of a contiguous tensor of one dtype (None: no tensor)."""
    if t is None:
        return None
    if not isinstance(t, _TORCH.Tensor) or t.dtype is not dtype or t.numel() < numel or not t.is_contiguous():
        _shape(t, dtype, numel, name)  # says which
    return t.data_ptr()


def _needed(t, name: str):
    if t is None:
        raise TypeError(f"{name} must be a torch tensor")
    return t


def _launch_on(stream, **tensors) -> int:
    """The stream to launch on, after checking that every tensor is on the
    current GPU: a launch goes there, whatever device its pointers belong to."""
    here = None
    for name, t in tensors.items():
        if t is None:
            continue
        at = t.get_device()
        if at < 0:
            raise ValueError(f"{name} must be on the GPU (got {t.device})")
        if here is None:
            here = _TORCH.cuda.current_device()
        if at != here:
            raise ValueError(f"{name} is on {t.device} but cuda:{here} is the current device")
    if stream is None and here is not None:
        return _TORCH._C._cuda_getCurrentRawStream(here)  # current_stream() takes longer than a launch
    return _stream(stream)


def _workspace(t, need):
    """(pointer, bytes); the library compares the bytes with what it needs."""
    if t is None:
        if (n := need()):
            raise ValueError(f"this call needs a workspace of {n} bytes")
        return None, 0
    _shape(t, (_TORCH.uint8, _TORCH.int8), None, "workspace")
    return t.data_ptr(), t.numel()


def _wrote(*tensors) -> None:
    """Tells autograd that a call changed these tensors in place, so that a
    backward pass that needs what was there (a gradient over logits that tanh
    or log_softmax kept) is an error instead of a wrong result."""
    _WROTE([t for t in tensors if t is not None])


def scape_topk_rows_workspace_bytes(z, k: int) -> int:
    """Bytes of workspace scape_topk_rows needs for this tensor's shape."""
    _, did, rows, cols, _ = _matrix(z, "z")
    b = ctypes.c_int64()
    _check(lib().scape_topk_rows_workspace(did, rows, cols, int(k), ctypes.byref(b)))
    return b.value


def scape_topk_rows(z, k: int, val, idx, lse=None, scale: float = 1.0, workspace=None, stream=None) -> None:
    """The k largest entries of each row of z (2-D, rows contiguous) into val
    (z's dtype) and idx (int32), both rows*k elements, and the row's
    log-sum-exp of scale*z into lse (fp32) where given."""
    zp, did, rows, cols, ld = _matrix(z, "z")
    vp = _array(_needed(val, "val"), z.dtype, rows * k, "val")
    ip = _array(_needed(idx, "idx"), _TORCH.int32, rows * k, "idx")
    lp = _array(lse, _TORCH.float32, rows, "lse")
    wp, wb = _workspace(workspace, lambda: scape_topk_rows_workspace_bytes(z, k))
    st = _launch_on(stream, z=z, val=val, idx=idx, lse=lse, workspace=workspace)
    _check(lib().scape_topk_rows(zp, did, rows, cols, ld, k, scale, vp, ip, lp, wp, wb, st))
    _wrote(val, idx, lse)


def _teacher(t_val, t_idx, t_lse, rows: int) -> _Teacher:
    for t, name in ((t_val, "t_val"), (t_idx, "t_idx")):
        if not isinstance(t, _TORCH.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
    if t_val.dim() != 2 or t_val.shape != t_idx.shape or t_val.shape[0] != rows:
        raise ValueError(f"t_val and t_idx must both be [{rows}, k] (got {tuple(t_val.shape)}, {tuple(t_idx.shape)})")
    k = t_val.shape[1]
    did = _dtype_id(t_val.dtype)
    return _Teacher(_array(t_val, t_val.dtype, rows * k, "t_val"), did, _array(t_idx, _TORCH.int32, rows * k, "t_idx"),
                    _array(t_lse, _TORCH.float32, rows, "t_lse"), k)


def scape_distill_workspace_bytes(z, k: int, grad: Optional[bool] = None) -> int:
    """Bytes of workspace scape_distill_forward needs for this tensor's shape:
    with dz (grad=True), without (False), or enough for either."""
    _, did, rows, cols, _ = _matrix(z, "z")
    b = ctypes.c_int64()
    query = lib().scape_distill_loss_workspace if grad is not None and not grad else lib().scape_distill_workspace
    _check(query(did, rows, cols, int(k), ctypes.byref(b)))
    return b.value


def scape_distill_forward(z, t_val, t_idx, loss, stats, t_lse=None, scale: float = 1.0, weight=None, dz=None,
                          workspace=None, stream=None) -> None:
    """Distillation loss of the logits z [rows, cols] from a teacher's top
    logits t_val, t_idx [rows, k]: with t_lse the teacher's mass outside the
    entries is matched as one more class, without it the teacher is
    renormalised over them.  loss fp32 [rows], stats fp32 [rows, 2]; dz (z's
    dtype and shape, may be z) also takes the gradient of loss.sum().  For
    autograd: z.backward(dz) on the logits' graph; over z itself
    (z.backward(z.detach())) where the operation that made z does not need its
    output again, as a matrix product does not."""
    zp, did, rows, cols, ld = _matrix(z, "z")
    t = _teacher(t_val, t_idx, t_lse, rows)
    dp, ld_dz = None, 0
    if dz is not None:
        dp, _, _, _, ld_dz = _matrix(dz, "dz", like=z)
    f32 = _TORCH.float32
    wt = _array(weight, f32, rows, "weight")
    lp = _array(_needed(loss, "loss"), f32, rows, "loss")
    sp = _array(_needed(stats, "stats"), f32, 2 * rows, "stats")
    wp, wb = _workspace(workspace, lambda: scape_distill_workspace_bytes(z, t.k, grad=dz is not None))
    st = _launch_on(stream, z=z, t_val=t_val, t_idx=t_idx, t_lse=t_lse, weight=weight, loss=loss, stats=stats, dz=dz,
                    workspace=workspace)
    _check(lib().scape_distill_forward(zp, did, rows, cols, ld, t, scale, wt, lp, sp, dp, ld_dz, wp, wb, st))
    _wrote(loss, stats, dz)


def scape_distill_backward(z, t_val, t_idx, stats, dz, t_lse=None, scale: float = 1.0, weight=None, dloss=None,
                           stream=None) -> None:
    """dz = dloss * weight * dKL/dz per row, from the stats of a forward call
    on the same z, teacher and scale.  dz may be z."""
    zp, did, rows, cols, ld = _matrix(z, "z")
    t = _teacher(t_val, t_idx, t_lse, rows)
    dp, _, _, _, ld_dz = _matrix(dz, "dz", like=z)
    f32 = _TORCH.float32
    wt = _array(weight, f32, rows, "weight")
    sp = _array(_needed(stats, "stats"), f32, 2 * rows, "stats")
    gp = _array(dloss, f32, rows, "dloss")
    st = _launch_on(stream, z=z, t_val=t_val, t_idx=t_idx, t_lse=t_lse, weight=weight, stats=stats, dloss=dloss, dz=dz)
    _check(lib().scape_distill_backward(zp, did, rows, cols, ld, t, scale, wt, sp, gp, dp, ld_dz, st))
    _wrote(dz)


SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score: str) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)} (got {score!r})")
    return SCORES[score]


def _router(offsets, mask, tokens: int):
    """(offsets pointer, segments, mask pointer)"""
    segs = 1
    if offsets is not None:
        _array(offsets, _TORCH.int32, 2, "offsets")
        segs = offsets.numel() - 1
    mp = None
    if mask is not None:
        mp = _array(mask, _TORCH.bool if getattr(mask, "dtype", None) is _TORCH.bool else _TORCH.uint8, tokens, "mask")
    return (None if offsets is None else offsets.data_ptr()), segs, mp


def scape_balance_workspace_bytes(logits, segments: int = 1) -> int:
    """Bytes of workspace scape_balance_forward needs for this tensor's shape."""
    _, _, tokens, experts, _ = _matrix(logits, "logits")
    b = ctypes.c_int64()
    _check(lib().scape_balance_workspace(tokens, experts, int(segments), ctypes.byref(b)))
    return b.value


def scape_balance_forward(logits, idx, counts, psum, n_tok, loss=None, alpha: float = 1.0, offsets=None, mask=None,
                          score: str = "softmax", workspace=None, stream=None) -> None:
    """Per segment: the experts' counts (int32 [segments, experts]), the sums
    of their scores psum (fp32), the valid tokens n_tok (int32) and the
    balance loss (fp32) of router logits [tokens, experts] and choices idx
    (int32 [tokens, k]).  offsets: int32 [segments + 1], or one segment of all
    tokens; mask: uint8 or bool [tokens]."""
    zp, did, tokens, experts, ld = _matrix(logits, "logits")
    op, segs, mp = _router(offsets, mask, tokens)
    if not isinstance(idx, _TORCH.Tensor) or idx.dim() != 2 or idx.shape[0] != tokens:
        raise ValueError(f"idx must be a tensor of [{tokens}, k]")
    k = idx.shape[1]
    i32, f32 = _TORCH.int32, _TORCH.float32
    ip = _array(idx, i32, tokens * k, "idx")
    cp = _array(_needed(counts, "counts"), i32, segs * experts, "counts")
    pp = _array(_needed(psum, "psum"), f32, segs * experts, "psum")
    np_ = _array(_needed(n_tok, "n_tok"), i32, segs, "n_tok")
    lp = _array(loss, f32, segs, "loss")
    wp, wb = _workspace(workspace, lambda: scape_balance_workspace_bytes(logits, segs))
    st = _launch_on(stream, logits=logits, idx=idx, offsets=offsets, mask=mask, counts=counts, psum=psum, n_tok=n_tok,
                    loss=loss, workspace=workspace)
    _check(lib().scape_balance_forward(zp, did, tokens, experts, ld, ip, k, op, segs, mp, _score(score), alpha, cp, pp,
                                       np_, lp, wp, wb, st))
    _wrote(counts, psum, n_tok, loss)


def scape_balance_loss(counts, psum, n_tok, loss, k: int, alpha: float = 1.0, stream=None) -> None:
    """The loss of counts and psum [segments, experts] and n_tok [segments],
    for instance their sums over data-parallel workers."""
    if not isinstance(counts, _torch().Tensor) or counts.dim() != 2:
        raise ValueError("counts must be a tensor of [segments, experts]")
    segs, experts = counts.shape
    i32, f32 = _TORCH.int32, _TORCH.float32
    cp = _array(counts, i32, segs * experts, "counts")
    pp = _array(_needed(psum, "psum"), f32, segs * experts, "psum")
    np_ = _array(_needed(n_tok, "n_tok"), i32, segs, "n_tok")
    lp = _array(_needed(loss, "loss"), f32, segs, "loss")
    st = _launch_on(stream, counts=counts, psum=psum, n_tok=n_tok, loss=loss)
    _check(lib().scape_balance_loss(cp, pp, np_, segs, experts, k, alpha, lp, st))
    _wrote(loss)


def scape_balance_backward(logits, counts, n_tok, dloss, dlogits, k: int, alpha: float = 1.0, offsets=None, mask=None,
                           score: str = "softmax", stream=None) -> None:
    """dlogits (the logits' dtype and shape, may be the logits) from counts
    and n_tok (this worker's, or their sums over workers) and dloss
    [segments] (None: 1).  Rows outside every segment are left as they were."""
    zp, did, tokens, experts, ld = _matrix(logits, "logits")
    dp, _, _, _, ld_d = _matrix(dlogits, "dlogits", like=logits)
    op, segs, mp = _router(offsets, mask, tokens)
    i32, f32 = _TORCH.int32, _TORCH.float32
    cp = _array(_needed(counts, "counts"), i32, segs * experts, "counts")
    np_ = _array(_needed(n_tok, "n_tok"), i32, segs, "n_tok")
    gp = _array(dloss, f32, segs, "dloss")
    st = _launch_on(stream, logits=logits, counts=counts, n_tok=n_tok, dloss=dloss, dlogits=dlogits, offsets=offsets,
                    mask=mask)
    _check(lib().scape_balance_backward(zp, did, tokens, experts, ld, k, op, segs, mp, _score(score), alpha, cp, np_,
                                        gp, dp, ld_d, st))
    _wrote(dlogits)
