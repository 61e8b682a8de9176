"""Python binding of the engine's C ABI (include/zl.h), argument marshalling only.

Every entry point keeps its C name.  Tensors are torch tensors (device memory and
streams only); each call checks dtype, device, contiguity and sizes, then passes raw
pointers to libzl.so.  There is no fallback: if the library is missing the import of
this module's functions raises, and a non-OK status raises ZlError.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field
from typing import Dict, List, Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libzl.so")

ZL_OK, ZL_ERR_INVALID_ARG, ZL_ERR_ALIGN, ZL_ERR_CUDA, ZL_ERR_TIMEOUT, ZL_ERR_UNSUPPORTED, ZL_ERR_NO_MEMORY = range(7)
ZL_PLAN_HOST_ONLY = 1
ZL_PLAN_TEST_WITHHOLD_LOAD = 2
ZL_PLAN_FUSE_LOCAL_KMERGE = 8
ZL_PLAN_DETERMINISTIC_DQ = 16
ZL_PLAN_FORWARD_ONLY = 32
ZL_KV4_BAD_PAGE, ZL_KV4_BAD_LEN, ZL_KV4_BAD_STARTS, ZL_KV4_TIMEOUT = 1, 2, 4, 8


class ZlError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class zl_work_item(ctypes.Structure):
    _fields_ = [("seq_offset", ctypes.c_int64), ("seq_len", ctypes.c_int32),
                ("q_lo", ctypes.c_int32), ("q_hi", ctypes.c_int32),
                ("h_lo", ctypes.c_int32), ("h_hi", ctypes.c_int32),
                ("kv_lo", ctypes.c_int32), ("kv_hi", ctypes.c_int32),
                ("emit_lse", ctypes.c_int32),
                ("out_offset", ctypes.c_int64), ("lse_offset", ctypes.c_int64)]


class zl_qk_rope_desc(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("rot_dim", ctypes.c_int32), ("half_layout", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("axis_pairs", ctypes.c_int32 * 3), ("amplitude", ctypes.c_float),
                ("q_rows", ctypes.c_void_p), ("k_rows", ctypes.c_void_p)]


class zl_causal_seq(ctypes.Structure):
    _fields_ = [("q_offset", ctypes.c_int64), ("kv_offset", ctypes.c_int64),
                ("q_len", ctypes.c_int32), ("kv_len", ctypes.c_int32)]


class zl_kv4_cache(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                ("data", ctypes.c_void_p), ("pages", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class zl_bucket(ctypes.Structure):
    _fields_ = [("seq_len", ctypes.c_int64), ("count", ctypes.c_int32), ("time", ctypes.c_double),
                ("mem", ctypes.c_double)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libzl.so (built by coalesced_packed_attention_gb300.build) and declare
    the signatures.  Raises OSError when the library has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"{path} not found: build it with `python -m coalesced_packed_attention_gb300.build`")
    L = ctypes.CDLL(path)
    P, I32, I64, U32, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
    pI64, pI32 = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32)
    pD = ctypes.POINTER(ctypes.c_double)
    sig = {
        "zl_plan_worklist": (I32, [ctypes.POINTER(zl_work_item), I32, I32, I32, I64, U32, ctypes.POINTER(P)]),
        "zl_plan_worklist_groups": (I32, [ctypes.POINTER(zl_work_item), I32, I32, I32, I64, U32, pI32, pI32, I32,
                                          ctypes.POINTER(P)]),
        "zl_plan_destroy": (None, [P]),
        "zl_plan_arena_sizes": (I32, [P, pI64, pI64, pI64, pI64, pI64, pI64]),
        "zl_plan_item": (I32, [P, I32, ctypes.POINTER(zl_work_item), pI64, pI64, pI64, pI64, pI32]),
        "zl_plan_count": (I32, [P, I32, pI64]),
        "zl_plan_check_bounds": (I32, [P]),
        "zl_plan_tiles": (I32, [P, I32, pI32, I64]),
        "zl_plan_group": (I32, [P, I32, pI32, I32, pI32, pI64, pI64]),
        "zl_coalesced_attn_fwd": (I32, [P, P, P, P, P, P, P, F, P]),
        "zl_merge_partials": (I32, [P, P, P, P, P, P]),
        "zl_coalesced_attn_bwd": (I32, [P, P, P, P, P, P, P, P, P, P, P, F, P]),
        "zl_bwd_preprocess": (I32, [P, P, P, P, P]),
        "zl_bwd_main": (I32, [P, P, P, P, P, P, P, P, P, F, P]),
        "zl_bwd_finalize": (I32, [P, P, P, F, P]),
        "zl_get_device_status": (I32, [P, P, pI32]),
        "zl_status_string": (ctypes.c_char_p, [I32]),
        "zl_version": (I32, []),
        "zl_rope_frequencies": (I32, [pD, I32, ctypes.POINTER(ctypes.c_uint64)]),
        "zl_qk_rope_workspace": (I32, [ctypes.POINTER(zl_qk_rope_desc), pI64]),
        "zl_qk_rope_fwd": (I32, [ctypes.POINTER(zl_qk_rope_desc), P, I64, P, I64, P, P, P, P, P, I64, P, I64, P]),
        "zl_qk_rope_bwd": (I32, [ctypes.POINTER(zl_qk_rope_desc), P, I64, P, I64, P, P, P, P, P, I64, P, I64, P, I64,
                                 P, I64, P, P, P, P]),
        "zl_plan_causal": (I32, [ctypes.POINTER(zl_causal_seq), I32, I32, I32, I32, I64, I64, U32, ctypes.POINTER(P)]),
        "zl_causal_plan_destroy": (None, [P]),
        "zl_causal_plan_workspace": (I32, [P, pI64, pI64]),
        "zl_causal_plan_tiles": (I32, [P, I32, pI32, I64, pI64]),
        "zl_causal_attn_fwd": (I32, [P, P, I64, P, I64, P, I64, P, P, P, F, P]),
        "zl_causal_attn_bwd": (I32, [P, P, I64, P, I64, P, I64, P, P, P, P, I64, P, I64, P, I64, P, F, P]),
        "zl_causal_get_device_status": (I32, [P, P, pI32]),
        "zl_kv4_write": (I32, [ctypes.POINTER(zl_kv4_cache), P, I64, P, I64, I64, P, P, P, P]),
        "zl_kv4_read": (I32, [ctypes.POINTER(zl_kv4_cache), P, I64, P, I64, I64, P, P]),
        "zl_kv4_attn_workspace": (I32, [ctypes.POINTER(zl_kv4_cache), I32, I32, I32, pI64]),
        "zl_kv4_attn_fwd": (I32, [ctypes.POINTER(zl_kv4_cache), P, I64, I64, I32, P, I32, P, P, P, P, F, P, F, P]),
        "zl_kv4_evict_workspace": (I32, [ctypes.POINTER(zl_kv4_cache), pI64]),
        "zl_kv4_evict": (I32, [ctypes.POINTER(zl_kv4_cache), P, P, I32, I32, P, P, P, P]),
        "zl_catalog_cut": (I32, [ctypes.POINTER(zl_bucket), I32, pI32, ctypes.POINTER(ctypes.c_double)]),
        "zl_pack_fillers": (I32, [pD, pD, I32, I32, pD, pD, ctypes.c_double, ctypes.c_double, pI32, pD, pD, pI32, pD]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def status_string(status: int) -> str:
    return load_library().zl_status_string(status).decode()


def _check(status: int, what: str):
    if status != ZL_OK:
        raise ZlError(status, what)


@dataclass
class ItemPlacement:
    item: zl_work_item
    fin_out_offset: int
    fin_lse_offset: int
    dq_offset: int
    dkv_offset: int
    group: int


class Plan:
    """Owner of one zl_plan*.  Created by zl_plan_worklist()."""

    def __init__(self, handle: int, n_heads: int, head_dim: int, total_tokens: int, host_only: bool,
                 device: Optional[int] = None):
        self.handle = ctypes.c_void_p(handle)
        self.n_heads, self.head_dim, self.total_tokens, self.host_only = n_heads, head_dim, total_tokens, host_only
        self.device = device  # CUDA device index the plan was built on (None: host-only plan)
        L = load_library()
        v = [ctypes.c_int64() for _ in range(6)]
        _check(L.zl_plan_arena_sizes(self.handle, *[ctypes.byref(x) for x in v]), "zl_plan_arena_sizes")
        (self.o_elems, self.o_partial_elems, self.lse_elems, self.dq_elems, self.dkv_elems,
         self.workspace_bytes) = (x.value for x in v)
        self.n_fwd_tiles = self._count(0)
        self.n_bwd_tiles = self._count(1)
        self.n_groups = self._count(2)
        self.n_items = self._count(3)
        self.n_merge_groups = self._count(4)  # groups the merge launch combines (unfused)

    def _count(self, which: int) -> int:
        c = ctypes.c_int64()
        _check(load_library().zl_plan_count(self.handle, which, ctypes.byref(c)), "zl_plan_count")
        return c.value

    def item(self, i: int) -> ItemPlacement:
        it = zl_work_item()
        vals = [ctypes.c_int64() for _ in range(4)]
        g = ctypes.c_int32()
        _check(load_library().zl_plan_item(self.handle, i, ctypes.byref(it), *[ctypes.byref(x) for x in vals],
                                           ctypes.byref(g)), "zl_plan_item")
        return ItemPlacement(it, vals[0].value, vals[1].value, vals[2].value, vals[3].value, g.value)

    def check_bounds(self):
        """Host dry run: every access a launch would make stays inside the arenas."""
        _check(load_library().zl_plan_check_bounds(self.handle), "zl_plan_check_bounds")

    def tiles(self, which: int = 0):
        """Tile list in scheduler order as a list of (item, head, block, cost)."""
        n = self.n_fwd_tiles if which == 0 else self.n_bwd_tiles
        buf = (ctypes.c_int32 * (4 * max(n, 1)))()
        _check(load_library().zl_plan_tiles(self.handle, which, buf, n), "zl_plan_tiles")
        return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]

    def group(self, g: int):
        """(member item ids, final O offset, final LSE offset) of merge group g."""
        n = ctypes.c_int32()
        oo, lo = ctypes.c_int64(), ctypes.c_int64()
        cap = 64
        while True:
            buf = (ctypes.c_int32 * cap)()
            _check(load_library().zl_plan_group(self.handle, g, buf, cap, ctypes.byref(n), ctypes.byref(oo),
                                                ctypes.byref(lo)), "zl_plan_group")
            if n.value <= cap:
                return list(buf[:n.value]), oo.value, lo.value
            cap = n.value

    def destroy(self):
        if self.handle is not None and self.handle.value:
            load_library().zl_plan_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def _to_c_items(items: Sequence) -> ctypes.Array:
    arr = (zl_work_item * max(1, len(items)))()
    for i, it in enumerate(items):
        arr[i] = zl_work_item(it.seq_offset, it.seq_len, it.q_lo, it.q_hi, it.h_lo, it.h_hi, it.kv_lo, it.kv_hi,
                              it.emit_lse, getattr(it, "out_offset", -1), getattr(it, "lse_offset", -1))
    return arr


def _plan_device(flags: int):
    if flags & ZL_PLAN_HOST_ONLY:
        return None
    import torch
    return torch.cuda.current_device() if torch.cuda.is_available() else None  # else the library reports it


def zl_plan_worklist(items: Sequence, n_heads: int, head_dim: int, total_tokens: int, flags: int = 0) -> Plan:
    L = load_library()
    h = ctypes.c_void_p()
    device = _plan_device(flags)
    _check(L.zl_plan_worklist(_to_c_items(items), len(items), n_heads, head_dim, total_tokens, flags,
                              ctypes.byref(h)), "zl_plan_worklist")
    return Plan(h.value, n_heads, head_dim, total_tokens, bool(flags & ZL_PLAN_HOST_ONLY), device)


def zl_plan_worklist_groups(items: Sequence, n_heads: int, head_dim: int, total_tokens: int,
                            groups: Sequence[Sequence[int]], flags: int = 0) -> Plan:
    """zl_plan_worklist with caller-chosen merge groups: groups[g] lists the work-list
    indices of group g's emit_lse items in member order (passed as group_item_ids /
    group_ptr)."""
    L = load_library()
    h = ctypes.c_void_p()
    ids = [int(i) for g in groups for i in g]
    ptr = [0]
    for g in groups:
        ptr.append(ptr[-1] + len(g))
    c_ids = (ctypes.c_int32 * max(1, len(ids)))(*ids)
    c_ptr = (ctypes.c_int32 * len(ptr))(*ptr)
    device = _plan_device(flags)
    _check(L.zl_plan_worklist_groups(_to_c_items(items), len(items), n_heads, head_dim, total_tokens, flags, c_ids,
                                     c_ptr, len(groups), ctypes.byref(h)), "zl_plan_worklist_groups")
    return Plan(h.value, n_heads, head_dim, total_tokens, bool(flags & ZL_PLAN_HOST_ONLY), device)


# ---------------------------------------------------------------- launches
def _ptr(t, dtype, what, numel=None):
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{what}: expected a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{what}: needs at least {numel} elements, has {t.numel()}")
    return t.data_ptr()


def _on_plan_device(plan: Plan, *tensors):
    """Every tensor lives on the plan's device (the library checks the current device)."""
    for t in tensors:
        if t is not None and getattr(t, "device", None) is not None and t.device.type == "cuda" \
                and t.device.index != plan.device:
            raise ValueError(f"tensor on cuda:{t.device.index}, plan built on cuda:{plan.device}")


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _qkv(plan: Plan, q, k, v):
    import torch
    shape = (plan.total_tokens, plan.n_heads, plan.head_dim)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    return [_ptr(t, torch.bfloat16, n) for t, n in ((q, "q"), (k, "k"), (v, "v"))]


def zl_coalesced_attn_fwd(plan: Plan, q, k, v, o, o_partial, lse, scale: float, stream=None):
    import torch
    _on_plan_device(plan, q, k, v, o, o_partial, lse)
    pq, pk, pv = _qkv(plan, q, k, v)
    st = load_library().zl_coalesced_attn_fwd(
        plan.handle, pq, pk, pv,
        _ptr(o, torch.bfloat16, "o", plan.o_elems) if o is not None else None,
        _ptr(o_partial, torch.float32, "o_partial", plan.o_partial_elems) if o_partial is not None else None,
        _ptr(lse, torch.float32, "lse", plan.lse_elems), ctypes.c_float(scale), _stream(stream))
    _check(st, "zl_coalesced_attn_fwd")


def zl_merge_partials(plan: Plan, o_partial, lse_partial, o, lse_out, stream=None):
    import torch
    _on_plan_device(plan, o_partial, lse_partial, o, lse_out)
    st = load_library().zl_merge_partials(
        plan.handle, _ptr(o_partial, torch.float32, "o_partial", plan.o_partial_elems),
        _ptr(lse_partial, torch.float32, "lse_partial", plan.lse_elems),
        _ptr(o, torch.bfloat16, "o", plan.o_elems), _ptr(lse_out, torch.float32, "lse_out", plan.lse_elems),
        _stream(stream))
    _check(st, "zl_merge_partials")


def zl_coalesced_attn_bwd(plan: Plan, q, k, v, o, d_o, lse, dq, dk, dv, workspace, scale: float, stream=None):
    import torch
    _on_plan_device(plan, q, k, v, o, d_o, lse, dq, dk, dv, workspace)
    pq, pk, pv = _qkv(plan, q, k, v)
    st = load_library().zl_coalesced_attn_bwd(
        plan.handle, pq, pk, pv, _ptr(o, torch.bfloat16, "o", plan.o_elems),
        _ptr(d_o, torch.bfloat16, "d_o", plan.o_elems), _ptr(lse, torch.float32, "lse", plan.lse_elems),
        _ptr(dq, torch.float32, "dq", plan.dq_elems), _ptr(dk, torch.float32, "dk", plan.dkv_elems),
        _ptr(dv, torch.float32, "dv", plan.dkv_elems),
        _ptr(workspace, torch.uint8, "workspace", plan.workspace_bytes), ctypes.c_float(scale), _stream(stream))
    _check(st, "zl_coalesced_attn_bwd")


def zl_bwd_preprocess(plan: Plan, o, d_o, workspace, stream=None):
    import torch
    _on_plan_device(plan, o, d_o, workspace)
    _check(load_library().zl_bwd_preprocess(
        plan.handle, _ptr(o, torch.bfloat16, "o", plan.o_elems), _ptr(d_o, torch.bfloat16, "d_o", plan.o_elems),
        _ptr(workspace, torch.uint8, "workspace", plan.workspace_bytes), _stream(stream)), "zl_bwd_preprocess")


def zl_bwd_main(plan: Plan, q, k, v, d_o, lse, dk, dv, workspace, scale: float, stream=None):
    import torch
    _on_plan_device(plan, q, k, v, d_o, lse, dk, dv, workspace)
    pq, pk, pv = _qkv(plan, q, k, v)
    _check(load_library().zl_bwd_main(
        plan.handle, pq, pk, pv, _ptr(d_o, torch.bfloat16, "d_o", plan.o_elems),
        _ptr(lse, torch.float32, "lse", plan.lse_elems), _ptr(dk, torch.float32, "dk", plan.dkv_elems),
        _ptr(dv, torch.float32, "dv", plan.dkv_elems), _ptr(workspace, torch.uint8, "workspace", plan.workspace_bytes),
        ctypes.c_float(scale), _stream(stream)), "zl_bwd_main")


def zl_bwd_finalize(plan: Plan, dq, workspace, scale: float, stream=None):
    import torch
    _on_plan_device(plan, dq, workspace)
    _check(load_library().zl_bwd_finalize(
        plan.handle, _ptr(dq, torch.float32, "dq", plan.dq_elems),
        _ptr(workspace, torch.uint8, "workspace", plan.workspace_bytes), ctypes.c_float(scale), _stream(stream)),
        "zl_bwd_finalize")


def zl_get_device_status(plan: Plan, stream=None) -> int:
    s = ctypes.c_int32()
    _check(load_library().zl_get_device_status(plan.handle, _stream(stream), ctypes.byref(s)),
           "zl_get_device_status")
    return s.value


# ---------------------------------------------------------------- conveniences
def allocate(plan: Plan, device="cuda", backward: bool = False) -> Dict[str, "object"]:
    """Device arenas sized for the plan (fresh torch allocations, uninitialised)."""
    import torch
    out = {
        "o": torch.empty(max(plan.o_elems, 8), dtype=torch.bfloat16, device=device),
        "o_partial": torch.empty(max(plan.o_partial_elems, 8), dtype=torch.float32, device=device),
        "lse": torch.empty(max(plan.lse_elems, 4), dtype=torch.float32, device=device),
    }
    if backward:
        out["dq"] = torch.empty(max(plan.dq_elems, 4), dtype=torch.float32, device=device)
        out["dk"] = torch.empty(max(plan.dkv_elems, 4), dtype=torch.float32, device=device)
        out["dv"] = torch.empty(max(plan.dkv_elems, 4), dtype=torch.float32, device=device)
        out["workspace"] = torch.empty(max(plan.workspace_bytes, 16), dtype=torch.uint8, device=device)
    return out


def o_arena_from_tokens(plan: Plan, items: Sequence, x):
    """A [T, H, d] token tensor laid out like the `o` arena: each work item's final block
    (its own, or its merge group's) holds that item's query rows and heads of x.  This is
    the layout in which the backward reads the output gradient dO."""
    import torch
    d = plan.head_dim
    arena = torch.zeros(max(plan.o_elems, 8), dtype=x.dtype, device=x.device)
    for i, it in enumerate(items):
        pl = plan.item(i)
        n = (it.q_hi - it.q_lo) * (it.h_hi - it.h_lo) * d
        arena[pl.fin_out_offset: pl.fin_out_offset + n] = \
            x[it.seq_offset + it.q_lo: it.seq_offset + it.q_hi, it.h_lo:it.h_hi].reshape(-1)
    return arena


def forward(plan: Plan, q, k, v, scale: float, bufs: Optional[dict] = None, stream=None) -> dict:
    """Forward of every item, then the merge of every k-split group."""
    bufs = bufs if bufs is not None else allocate(plan, q.device)
    zl_coalesced_attn_fwd(plan, q, k, v, bufs["o"], bufs["o_partial"], bufs["lse"], scale, stream)
    if plan.n_merge_groups:
        zl_merge_partials(plan, bufs["o_partial"], bufs["lse"], bufs["o"], bufs["lse"], stream)
    return bufs


def backward(plan: Plan, q, k, v, d_o, scale: float, bufs: dict, stream=None) -> dict:
    zl_coalesced_attn_bwd(plan, q, k, v, bufs["o"], d_o, bufs["lse"], bufs["dq"], bufs["dk"], bufs["dv"],
                          bufs["workspace"], scale, stream)
    return bufs


def exported_symbols() -> List[str]:
    """Names of the entry points declared in include/zl.h."""
    return ["zl_plan_worklist", "zl_plan_worklist_groups", "zl_plan_destroy", "zl_plan_arena_sizes", "zl_plan_item", "zl_plan_check_bounds",
            "zl_plan_count",
            "zl_plan_tiles", "zl_plan_group", "zl_coalesced_attn_fwd", "zl_merge_partials",
            "zl_coalesced_attn_bwd", "zl_bwd_preprocess", "zl_bwd_main", "zl_bwd_finalize",
            "zl_get_device_status", "zl_status_string", "zl_version", "zl_catalog_cut", "zl_pack_fillers",
            "zl_rope_frequencies", "zl_qk_rope_workspace", "zl_qk_rope_fwd", "zl_qk_rope_bwd", "zl_plan_causal",
            "zl_causal_plan_destroy", "zl_causal_plan_workspace", "zl_causal_plan_tiles", "zl_causal_attn_fwd",
            "zl_causal_attn_bwd", "zl_causal_get_device_status", "zl_kv4_write", "zl_kv4_read", "zl_kv4_attn_workspace",
            "zl_kv4_attn_fwd", "zl_kv4_evict_workspace", "zl_kv4_evict"]


# ---------------------------------------------------------------- causal sequences
_torch_module = None


def _torch():
    """torch, imported by the first call that needs it (the launches below run every layer, and an import
    statement costs them half a microsecond each)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _heads(t, what, shape, dev):
    """(pointer, token stride) of a bf16 [tokens, heads, d] tensor on CUDA device `dev` whose heads are
    contiguous; the token stride is free, so views of a fused projection pass."""
    torch = _torch_module or _torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16:
        raise TypeError(f"{what}: expected a CUDA tensor of {torch.bfloat16}, got {getattr(t, 'dtype', type(t))}")
    if t.get_device() != dev:
        raise (ValueError if t.is_cuda else TypeError)(f"{what}: expected a tensor on cuda:{dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if n <= 1 or h == 0:
        s0 = h * d  # a lone token has no next one
        if n == 0 or h == 0:
            return None, s0
    if s2 != 1 or (s1 != d and h > 1):
        raise ValueError(f"{what}: the heads of a token must be contiguous, got strides {t.stride()}")
    if s0 < h * d:
        raise ValueError(f"{what}: token stride {s0} below heads * d = {h * d}")
    return t.data_ptr(), s0


def _dense(t, what, dtype, shape, dev):
    """Pointer of a contiguous tensor of exactly this type and shape on CUDA device `dev`."""
    if not isinstance(t, _torch().Tensor) or t.dtype is not dtype:
        raise TypeError(f"{what}: expected a CUDA tensor of {dtype}, got {getattr(t, 'dtype', type(t))}")
    if t.get_device() != dev:
        raise (ValueError if t.is_cuda else TypeError)(f"{what}: expected a tensor on cuda:{dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    return t.data_ptr()


def _scratch(t, what, nbytes, dev):
    """Pointer of a uint8 workspace of at least nbytes bytes on CUDA device `dev` (None where none is needed)."""
    torch = _torch()
    if t is None and nbytes == 0:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8 or t.get_device() != dev:
        raise TypeError(f"{what}: expected a torch.uint8 tensor on cuda:{dev}")
    if not t.is_contiguous() or t.numel() < nbytes:
        raise ValueError(f"{what}: needs {nbytes} contiguous bytes, has {t.numel()}")
    return t.data_ptr()


def _raw_stream(stream, dev):
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       original_len: int = 4096, slow: float = 1.0, fast: float = 32.0):
    """(radians per position of the rot_dim / 2 pairs, amplitude) of a rotary embedding,
    base^(-2i / rot_dim), optionally scaled for contexts `factor` times the original:
      "linear"  every frequency divided by the factor (positions pressed together);
      "ntk"     the base raised so that the slowest pair is divided by the factor, the
                fastest kept;
      "yarn"    the first pairs kept, the last divided by the factor, a ramp over the pair's index
                between: from the pair that turns `fast` times in original_len positions, rounded
                down, to the one that turns `slow` times, rounded up; amplitude 0.1 ln(factor) + 1.
                (As released checkpoints were trained.  A ramp over the number of turns, as the method is
                also written, gives other frequencies between, up to 3 times at factor 16;
                rotary_table takes those, or any.)"""
    import math
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim: expected an even number from 2 on, got {rot_dim}")
    if not (base > 0 and factor >= 1 and original_len > 0 and fast > slow):
        raise ValueError("expected base > 0, factor >= 1, original_len > 0 and fast > slow")
    if scaling == "ntk":
        base = base * factor ** (rot_dim / max(1, rot_dim - 2))
    freqs = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling in (None, "ntk"):
        return freqs, 1.0
    if scaling == "linear":
        return [f / factor for f in freqs], 1.0
    if scaling == "yarn":
        if not (base > 1 and fast > 0):
            raise ValueError("yarn: expected base > 1 and fast > 0")

        def pair_of(turns):  # original_len base^(-2i / rot_dim) / (2 pi) = turns
            if turns <= 0:  # no pair turns as seldom
                return rot_dim
            return rot_dim * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))

        first, last = max(0, math.floor(pair_of(fast))), min(rot_dim - 1, math.ceil(pair_of(slow)))
        out = []
        for i, f in enumerate(freqs):
            keep = 1.0 - min(1.0, max(0.0, (i - first) / max(last - first, 1e-3)))
            out.append(f * keep + f / factor * (1 - keep))
        return out, 0.1 * math.log(factor) + 1.0
    raise ValueError(f"scaling: expected None, 'linear', 'ntk' or 'yarn', got {scaling!r}")


@dataclass(frozen=True)
class RotaryTable:
    """Frequencies of a rotation on one device, and how the pairs are laid out.  Not to be changed once made (a call
    reuses the descriptor of the last call of the same sizes); dataclasses.replace makes another."""
    freq: "object"  # int64 tensor holding the 64-bit fractions of a turn per position
    rot_dim: int
    half: bool
    axis_pairs: Tuple[int, ...]
    amplitude: float
    device: int = field(init=False, default=-1, repr=False)           # CUDA device of freq
    ptr: Optional[int] = field(init=False, default=None, repr=False)  # and its address there
    last: list = field(init=False, default_factory=lambda: [(None, None)], repr=False, compare=False)

    def __post_init__(self):
        object.__setattr__(self, "axis_pairs", tuple(self.axis_pairs))
        if self.freq is None:
            if self.rot_dim != 0:
                raise ValueError(f"freq: needed where rot_dim is {self.rot_dim}")
        else:
            # kernels read rot_dim / 2 numbers from here
            torch = _torch()
            if not isinstance(self.freq, torch.Tensor) or self.freq.dtype not in (torch.int64, torch.uint64):
                raise TypeError(f"freq: expected a tensor of {torch.int64}, got {getattr(self.freq, 'dtype', type(self.freq))}")
            if not self.freq.is_contiguous() or 2 * self.freq.numel() < self.rot_dim:
                raise ValueError(f"freq: needs {self.rot_dim} / 2 contiguous numbers, got shape {tuple(self.freq.shape)}, "
                                 f"strides {self.freq.stride()}")
            object.__setattr__(self, "device", self.freq.get_device())
            object.__setattr__(self, "ptr", self.freq.data_ptr())


def rotary_table(inv_freq: Sequence[float], layout: str = "half", axis_pairs: Optional[Sequence[int]] = None,
                 amplitude: float = 1.0, device="cuda") -> RotaryTable:
    """Table for zl_qk_rope_fwd / bwd from radians per position, pair by pair.  layout: "half"
    (channels p and p + pairs) or "interleaved" (2p and 2p + 1).  axis_pairs: how many pairs each
    position axis turns, in order (default: one axis turns them all)."""
    import torch
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout: expected 'half' or 'interleaved', got {layout!r}")
    radians = [float(f) for f in inv_freq]
    n = len(radians)
    pairs = [int(a) for a in axis_pairs] if axis_pairs is not None else [n]
    if not 1 <= len(pairs) <= 3 or min(pairs) < 0 or sum(pairs) != n:
        raise ValueError(f"axis_pairs: expected one to three counts that add up to {n}, got {pairs}")
    out = (ctypes.c_uint64 * max(1, n))()
    _check(load_library().zl_rope_frequencies((ctypes.c_double * max(1, n))(*radians), n, out), "zl_rope_frequencies")
    freq = torch.tensor([ctypes.c_int64(x).value for x in out[:n]], dtype=torch.int64).to(device)
    return RotaryTable(freq, 2 * n, layout == "half", tuple(pairs), float(amplitude))


def zl_qk_rope_workspace_bytes(n_tokens: int, n_q_heads: int, n_kv_heads: int, head_dim: int) -> int:
    """Scratch bytes of a zl_qk_rope_bwd that returns weight gradients."""
    b = ctypes.c_int64()
    desc = zl_qk_rope_desc(n_tokens, n_q_heads, n_kv_heads, head_dim, 1, 0.0, 0, 0, 0, (ctypes.c_int32 * 3)(), 1.0)
    _check(load_library().zl_qk_rope_workspace(ctypes.byref(desc), ctypes.byref(b)), "zl_qk_rope_workspace")
    return b.value


_PLAIN = RotaryTable(None, 0, False, (), 1.0)  # no rotation


def _rope_args(q, k, positions, table, norm, eps, q_weight, k_weight):
    """(descriptor, device, query shape, key shape, pointers of positions, frequencies and weights)."""
    torch = _torch()
    lead = q if q is not None else k
    if not isinstance(lead, torch.Tensor):
        raise TypeError("q and k: at least one tensor is needed")
    if lead.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError(f"expected [tokens, heads, d], got {tuple(lead.shape)}")
    if not lead.is_cuda:
        raise TypeError(f"expected CUDA tensors, got one on {lead.device}")
    dev = torch._C._cuda_getDevice()
    n, hq, d = lead.shape
    hk = k.shape[1] if k is not None else 0
    if q is None:
        hq = 0
    if table is None:
        table = _PLAIN
    pos = freq = None
    if table.rot_dim > 0:
        axes = len(table.axis_pairs)
        pos = _dense(positions, "positions", torch.int32,
                     (n,) if axes == 1 and isinstance(positions, torch.Tensor) and positions.dim() == 1 else (n, axes), dev)
        freq = table.ptr
        if table.device != dev:
            raise ValueError(f"table on device {table.device}, current device is cuda:{dev}")
    key = (n, hq, hk, d, norm, eps)
    last = table.last[0]
    if last[0] != key:
        pairs = (table.axis_pairs + (0, 0, 0))[:3]
        last = (key, zl_qk_rope_desc(n, hq, hk, d, int(norm), eps, table.rot_dim, int(table.half), len(table.axis_pairs),
                                     (ctypes.c_int32 * 3)(*pairs), table.amplitude))
        table.last[0] = last
    qw = _dense(q_weight, "q_weight", torch.float32, (d,), dev) if q_weight is not None else None
    kw = _dense(k_weight, "k_weight", torch.float32, (d,), dev) if k_weight is not None else None
    return last[1], dev, (n, hq, d), (n, hk, d), pos, freq, qw, kw


def _maybe_heads(t, what, shape, dev):
    if t is None and shape[1] == 0:
        return None, 0
    return _heads(t, what, shape, dev)


def zl_qk_rope_fwd(q, k, q_out, k_out, positions, table: Optional[RotaryTable], norm: bool = False, q_weight=None,
                   k_weight=None, eps: float = 1e-6, stream=None):
    """Every head of q [tokens, Hq, d] and k [tokens, Hkv, d] (either may be None) normalised
    (norm=True) and rotated at its token's positions (int32 [tokens, axes]; table None: no
    rotation) into q_out, k_out, which may be q and k themselves.  Tensors live on the current device."""
    desc, dev, sq, sk, pos, freq, qw, kw = _rope_args(q, k, positions, table, norm, eps, q_weight, k_weight)
    pq, nq = _maybe_heads(q, "q", sq, dev)
    pk, nk = _maybe_heads(k, "k", sk, dev)
    oq, mq = _maybe_heads(q_out, "q_out", sq, dev)
    ok, mk = _maybe_heads(k_out, "k_out", sk, dev)
    st = load_library().zl_qk_rope_fwd(desc, pq, nq, pk, nk, qw, kw, pos, freq, oq, mq, ok, mk, _raw_stream(stream, dev))
    if st:
        _check(st, "zl_qk_rope_fwd")


_dw_bytes: Dict[int, int] = {}  # workspace of the weights' gradients by head dim


def zl_qk_rope_bwd(q, k, dq_out, dk_out, dq, dk, positions, table: Optional[RotaryTable], norm: bool = False,
                   q_weight=None, k_weight=None, dq_weight=None, dk_weight=None, workspace=None, eps: float = 1e-6,
                   stream=None, q_rows=None, k_rows=None):
    """Gradient of zl_qk_rope_fwd: dq, dk from dq_out, dk_out.  With norm=True q and k are the
    forward's inputs (else None will do) and dq_weight, dk_weight, where given, receive the
    weights' gradients (workspace: zl_qk_rope_workspace_bytes).  q_rows, k_rows (uint8 [tokens]): a token whose
    byte is 0 has gradient zero and adds nothing to the weights', whatever its rows hold."""
    torch = _torch()
    desc, dev, sq, sk, pos, freq, qw, kw = _rope_args(dq_out, dk_out, positions, table, norm, eps, q_weight, k_weight)
    if q_rows is not None or k_rows is not None:
        desc = zl_qk_rope_desc.from_buffer_copy(desc)  # the kept descriptor is of sizes alone
        for name, rows in (("q_rows", q_rows), ("k_rows", k_rows)):
            if rows is not None:
                setattr(desc, name, _dense(rows, name, torch.uint8, (sq[0],), dev))
    pq, nq = _maybe_heads(q, "q", sq, dev) if norm else (None, 0)
    pk, nk = _maybe_heads(k, "k", sk, dev) if norm else (None, 0)
    gq, lq = _maybe_heads(dq_out, "dq_out", sq, dev)
    gk, lk = _maybe_heads(dk_out, "dk_out", sk, dev)
    oq, mq = _maybe_heads(dq, "dq", sq, dev)
    ok, mk = _maybe_heads(dk, "dk", sk, dev)
    dqw = dkw = ws = None
    if dq_weight is not None or dk_weight is not None:
        d = sq[2]
        if d not in _dw_bytes:
            _dw_bytes[d] = zl_qk_rope_workspace_bytes(1, 1, 1, d)
        dqw = _dense(dq_weight, "dq_weight", torch.float32, (d,), dev) if dq_weight is not None else None
        dkw = _dense(dk_weight, "dk_weight", torch.float32, (d,), dev) if dk_weight is not None else None
        ws = _scratch(workspace, "workspace", _dw_bytes[d], dev)
    st = load_library().zl_qk_rope_bwd(desc, pq, nq, pk, nk, qw, kw, pos, freq, gq, lq, gk, lk, oq, mq, ok, mk, dqw, dkw,
                                       ws, _raw_stream(stream, dev))
    if st:
        _check(st, "zl_qk_rope_bwd")


class CausalPlan:
    """Owner of one zl_causal_plan*.  Created by zl_plan_causal()."""

    def __init__(self, handle: int, n_q_heads: int, n_kv_heads: int, head_dim: int, q_tokens: int, kv_tokens: int,
                 device: Optional[int]):
        self.handle = ctypes.c_void_p(handle)
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self.q_tokens, self.kv_tokens = q_tokens, kv_tokens
        self.device = device  # CUDA device index the plan was built on (None: host-only plan)
        self.q_shape, self.kv_shape = (q_tokens, n_q_heads, head_dim), (kv_tokens, n_kv_heads, head_dim)
        self.lse_shape = (q_tokens, n_q_heads)
        f, b = ctypes.c_int64(), ctypes.c_int64()
        _check(load_library().zl_causal_plan_workspace(self.handle, ctypes.byref(f), ctypes.byref(b)),
               "zl_causal_plan_workspace")
        self.fwd_workspace_bytes, self.bwd_workspace_bytes = f.value, b.value
        # uint8 [tokens], 1 where a row belongs to a sequence's queries (keys); None where every row does.  Tensors as any
        # other: a graph that captured qkv_attention_backward needs the plan object kept for them.
        self.q_rows = self.kv_rows = None
        self.kv_gaps = None  # int64, the rows whose kv_rows is 0

    def tiles(self, which: int = 0):
        """Schedule as (sequence, key head, block, first, end, part, thread block) tuples; which = 0
        forward (over key blocks), 1 backward (over query blocks)."""
        n = ctypes.c_int64()
        L = load_library()
        _check(L.zl_causal_plan_tiles(self.handle, which, None, 0, ctypes.byref(n)), "zl_causal_plan_tiles")
        buf = (ctypes.c_int32 * (7 * max(1, n.value)))()
        _check(L.zl_causal_plan_tiles(self.handle, which, buf, n.value, ctypes.byref(n)), "zl_causal_plan_tiles")
        return [tuple(buf[7 * i:7 * i + 7]) for i in range(n.value)]

    def destroy(self):
        if self.handle is not None and self.handle.value:
            load_library().zl_causal_plan_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def causal_seqs(lengths: Sequence[int]):
    """Sequences of self-attention packed one behind the other: (q_offset, q_len, kv_offset,
    kv_len) each, for zl_plan_causal."""
    out, at = [], 0
    for n in lengths:
        out.append((at, n, at, n))
        at += n
    return out


def _row_mask(ranges, tokens: int):
    """uint8 [tokens], 1 in the rows [offset, offset + len) of any range."""
    rows = bytearray(tokens)
    for at, n in ranges:
        rows[at:at + n] = b"\x01" * n
    return _torch().frombuffer(rows, dtype=_torch().uint8)


def zl_plan_causal(seqs: Sequence, n_q_heads: int, n_kv_heads: int, head_dim: int, q_tokens: int, kv_tokens: int,
                   flags: int = 0) -> CausalPlan:
    """Plan over seqs = [(q_offset, q_len, kv_offset, kv_len), ...] on the current device."""
    L = load_library()
    arr = (zl_causal_seq * max(1, len(seqs)))()
    for i, (qo, ql, ko, kl) in enumerate(seqs):
        for name, x, bits in (("q_offset", qo, 63), ("q_len", ql, 31), ("kv_offset", ko, 63), ("kv_len", kl, 31)):
            if not -(1 << bits) <= x < (1 << bits):
                raise ValueError(f"sequence {i}: {name} {x} does not fit {bits + 1} bits")
        arr[i] = zl_causal_seq(qo, ko, ql, kl)
    h = ctypes.c_void_p()
    device = _plan_device(flags)
    _check(L.zl_plan_causal(arr, len(seqs), n_q_heads, n_kv_heads, head_dim, q_tokens, kv_tokens, flags,
                            ctypes.byref(h)), "zl_plan_causal")
    plan = CausalPlan(h.value, n_q_heads, n_kv_heads, head_dim, q_tokens, kv_tokens, device)
    if device is not None and q_tokens == kv_tokens and not flags & ZL_PLAN_FORWARD_ONLY:
        # what qkv_attention_backward needs of a plan that leaves rows out (ranges that overlap have no backward)
        if sum(s[1] for s in seqs) < q_tokens:
            plan.q_rows = _row_mask([(s[0], s[1]) for s in seqs], q_tokens).to(f"cuda:{device}")
        if sum(s[3] for s in seqs) < kv_tokens:
            plan.kv_rows = _row_mask([(s[2], s[3]) for s in seqs], kv_tokens).to(f"cuda:{device}")
            plan.kv_gaps = (plan.kv_rows == 0).nonzero()[:, 0]
    return plan


def allocate_causal(plan: CausalPlan, device="cuda", backward: bool = False) -> Dict[str, "object"]:
    """Outputs, workspace and (backward) gradients of a causal plan, uninitialised."""
    import torch
    bf = dict(dtype=torch.bfloat16, device=device)
    ws = max(plan.fwd_workspace_bytes, plan.bwd_workspace_bytes if backward else 0)
    out = {"o": torch.empty(plan.q_tokens, plan.n_q_heads, plan.head_dim, **bf),
           "lse": torch.empty(plan.q_tokens, plan.n_q_heads, dtype=torch.float32, device=device),
           "workspace": torch.empty(max(16, ws), dtype=torch.uint8, device=device)}
    if backward:
        out["dq"] = torch.empty(plan.q_tokens, plan.n_q_heads, plan.head_dim, **bf)
        out["dk"] = torch.empty(plan.kv_tokens, plan.n_kv_heads, plan.head_dim, **bf)
        out["dv"] = torch.empty(plan.kv_tokens, plan.n_kv_heads, plan.head_dim, **bf)
    return out


def _plan_dev(plan: CausalPlan) -> int:
    return -2 if plan.device is None else plan.device  # no tensor is on a host-only plan's device


def zl_causal_attn_fwd(plan: CausalPlan, q, k, v, o, lse, workspace, scale: float, stream=None):
    """Causal attention of every sequence of the plan: q [q_tokens, Hq, d], k, v [kv_tokens, Hkv, d] (views of a
    fused projection will do) into o (contiguous) and lse [q_tokens, Hq]; workspace: plan.fwd_workspace_bytes."""
    torch = _torch()
    dev = _plan_dev(plan)
    pq, nq = _heads(q, "q", plan.q_shape, dev)
    pk, nk = _heads(k, "k", plan.kv_shape, dev)
    pv, nv = _heads(v, "v", plan.kv_shape, dev)
    st = load_library().zl_causal_attn_fwd(
        plan.handle, pq, nq, pk, nk, pv, nv, _dense(o, "o", torch.bfloat16, plan.q_shape, dev),
        _dense(lse, "lse", torch.float32, plan.lse_shape, dev),
        _scratch(workspace, "workspace", plan.fwd_workspace_bytes, dev), scale, _raw_stream(stream, dev))
    if st:
        _check(st, "zl_causal_attn_fwd")


def zl_causal_attn_bwd(plan: CausalPlan, q, k, v, o, d_o, lse, dq, dk, dv, workspace, scale: float, stream=None):
    """Gradients dq, dk, dv (bf16, token strides free) of zl_causal_attn_fwd from d_o (contiguous) and the o and lse
    that it left; workspace: plan.bwd_workspace_bytes."""
    torch = _torch()
    dev = _plan_dev(plan)
    pq, nq = _heads(q, "q", plan.q_shape, dev)
    pk, nk = _heads(k, "k", plan.kv_shape, dev)
    pv, nv = _heads(v, "v", plan.kv_shape, dev)
    gq, mq = _heads(dq, "dq", plan.q_shape, dev)
    gk, mk = _heads(dk, "dk", plan.kv_shape, dev)
    gv, mv = _heads(dv, "dv", plan.kv_shape, dev)
    st = load_library().zl_causal_attn_bwd(
        plan.handle, pq, nq, pk, nk, pv, nv, _dense(o, "o", torch.bfloat16, plan.q_shape, dev),
        _dense(d_o, "d_o", torch.bfloat16, plan.q_shape, dev), _dense(lse, "lse", torch.float32, plan.lse_shape, dev), gq, mq,
        gk, mk, gv, mv, _scratch(workspace, "workspace", plan.bwd_workspace_bytes, dev), scale, _raw_stream(stream, dev))
    if st:
        _check(st, "zl_causal_attn_bwd")


def zl_causal_get_device_status(plan: CausalPlan, stream=None) -> int:
    s = ctypes.c_int32()
    _check(load_library().zl_causal_get_device_status(plan.handle, _stream(stream), ctypes.byref(s)),
           "zl_causal_get_device_status")
    return s.value


def _qkv_views(plan: CausalPlan, qkv, what="qkv"):
    hq, hk = plan.n_q_heads, plan.n_kv_heads
    if plan.q_tokens != plan.kv_tokens:
        raise ValueError("a fused projection needs as many key rows as query rows")
    shape = (plan.q_tokens, hq + 2 * hk, plan.head_dim)
    if tuple(qkv.shape) != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(qkv.shape)}")
    return qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]


def allocate_qkv_attention(plan: CausalPlan, device="cuda", backward: bool = False) -> Dict[str, "object"]:
    """allocate_causal plus the normalised, rotated queries and keys, and the weights' gradients."""
    import torch
    sq, sk = plan.q_shape, plan.kv_shape
    out = allocate_causal(plan, device, backward)
    out["q"], out["k"] = (torch.empty(s, dtype=torch.bfloat16, device=device) for s in (sq, sk))
    if backward:
        out["dq_weight"], out["dk_weight"] = (torch.empty(plan.head_dim, dtype=torch.float32, device=device) for _ in range(2))
        out["rope_workspace"] = torch.empty(
            zl_qk_rope_workspace_bytes(plan.q_tokens, plan.n_q_heads, plan.n_kv_heads, plan.head_dim), dtype=torch.uint8,
            device=device)
    return out


def _sides(q_weight, k_weight):
    """(queries, keys, norm) of each launch of the rotation: both tensors in one, or, where one of them alone has a
    weight and with it a norm, one after the other."""
    if (q_weight is None) == (k_weight is None):
        return ((True, True, q_weight is not None),)
    return (True, False, q_weight is not None), (False, True, k_weight is not None)


def qkv_attention_forward(plan: CausalPlan, qkv, positions, table: Optional[RotaryTable], scale: float, bufs: dict,
                          q_weight=None, k_weight=None, eps: float = 1e-6, stream=None) -> dict:
    """Causal self-attention from a projection's output qkv [tokens, Hq + 2 Hkv, d]: queries and keys
    normalised where weights are given, rotated, attended; the values are read where they lie."""
    q, k, v = _qkv_views(plan, qkv)
    for of_q, of_k, norm in _sides(q_weight, k_weight):
        zl_qk_rope_fwd(q if of_q else None, k if of_k else None, bufs["q"] if of_q else None, bufs["k"] if of_k else None,
                       positions, table, norm, q_weight if of_q else None, k_weight if of_k else None, eps, stream)
    zl_causal_attn_fwd(plan, bufs["q"], bufs["k"], v, bufs["o"], bufs["lse"], bufs["workspace"], scale, stream)
    return bufs


def _zero_rows(t, rows, stream):
    """t[rows] = 0 on a stream given as the launches take it."""
    torch = _torch()
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_raw_stream(stream, t.get_device()), t.device)
    with torch.no_grad(), torch.cuda.stream(stream):  # None: the current one
        t.index_fill_(0, rows, 0.0)


def qkv_attention_backward(plan: CausalPlan, qkv, d_o, dqkv, positions, table: Optional[RotaryTable], scale: float,
                           bufs: dict, q_weight=None, k_weight=None, eps: float = 1e-6, stream=None) -> dict:
    """Gradient of qkv_attention_forward into dqkv (as qkv) and, with weights, bufs["dq_weight"] and
    bufs["dk_weight"].  Rows of no sequence get zeros and add nothing to the weights', whatever qkv and d_o hold
    there."""
    q, k, v = _qkv_views(plan, qkv)
    dq, dk, dv = _qkv_views(plan, dqkv, "dqkv")
    zl_causal_attn_bwd(plan, bufs["q"], bufs["k"], v, bufs["o"], d_o, bufs["lse"], bufs["dq"], bufs["dk"], dv,
                       bufs["workspace"], scale, stream)
    if plan.kv_gaps is not None:
        _zero_rows(dv, plan.kv_gaps, stream)
    for of_q, of_k, norm in _sides(q_weight, k_weight):
        zl_qk_rope_bwd(q if of_q else None, k if of_k else None, bufs["dq"] if of_q else None, bufs["dk"] if of_k else None,
                       dq if of_q else None, dk if of_k else None, positions, table, norm, q_weight if of_q else None,
                       k_weight if of_k else None, bufs["dq_weight"] if of_q and norm else None,
                       bufs["dk_weight"] if of_k and norm else None, bufs["rope_workspace"], eps, stream,
                       plan.q_rows if of_q else None, plan.kv_rows if of_k else None)
    return bufs


# ---------------------------------------------------------------- key-value cache in 4 bits
@dataclass(frozen=True)
class Kv4Cache:
    """A cache's tensors on one CUDA device.  Not to be changed once made (its calls reuse one descriptor), but for the
    tensors' contents: lens and pages are read by every call.
      data   uint8 [pages, key heads, page / 16, 18 d]: the rows' codes and scales (zl.h has the layout); zl_kv4_write fills it
      pages  int32 [sequences, pages of a sequence]: where slot s of a sequence lies, page s / page
      lens   int32 [sequences]: slots in use
    status: an int32 tensor of one number in which calls note what they had to leave out; see zl_kv4_get_device_status."""
    data: "object"
    pages: "object"
    lens: "object"
    status: "object" = None
    desc: zl_kv4_cache = field(init=False, repr=False, compare=False)
    no_rows: zl_kv4_cache = field(init=False, repr=False, compare=False)  # of no pages: calls on it note slots alone
    device: int = field(init=False, default=-1, repr=False)
    slots: int = field(init=False, default=0, repr=False)        # that the table has room for
    token_shape: tuple = field(init=False, default=(), repr=False)  # key heads, d
    slot_shape: tuple = field(init=False, default=(), repr=False)   # of weights and positions
    sizes: dict = field(init=False, default_factory=dict, repr=False, compare=False)  # workspaces by sizes

    def __post_init__(self):
        torch = _torch()
        if not isinstance(self.data, torch.Tensor) or self.data.dtype is not torch.uint8 or not self.data.is_cuda:
            raise TypeError(f"data: expected a CUDA tensor of {torch.uint8}, got {getattr(self.data, 'dtype', type(self.data))}")
        if self.data.dim() != 4 or self.data.shape[3] not in (18 * 64, 18 * 128):
            raise ValueError(f"data: expected [pages, key heads, page / 16, 18 d], d 64 or 128, got {tuple(self.data.shape)}")
        if not self.data.is_contiguous():
            raise ValueError("data: must be contiguous")
        dev = self.data.get_device()
        n_pages, heads, tiles, width = self.data.shape
        if not isinstance(self.pages, torch.Tensor) or self.pages.dim() != 2:
            raise TypeError("pages: expected a CUDA tensor [sequences, pages of a sequence]")
        n, most = self.pages.shape
        if self.status is None:
            object.__setattr__(self, "status", torch.zeros(1, dtype=torch.int32, device=self.data.device))
        pages, lens = _dense(self.pages, "pages", torch.int32, (n, most), dev), _dense(self.lens, "lens", torch.int32, (n,), dev)
        status = _dense(self.status, "status", torch.int32, (1,), dev)
        desc = zl_kv4_cache(n, heads, width // 18, 16 * tiles, most, n_pages, self.data.data_ptr(), pages, lens, status)
        _check(load_library().zl_kv4_evict_workspace(ctypes.byref(desc), ctypes.byref(ctypes.c_int64())), "Kv4Cache")
        no_rows = zl_kv4_cache(n, heads, width // 18, 16 * tiles, most, 0, None, pages, lens, None)
        for name, x in (("desc", desc), ("no_rows", no_rows), ("device", dev), ("slots", most * 16 * tiles),
                        ("token_shape", (heads, width // 18)), ("slot_shape", (n, heads, most * 16 * tiles))):
            object.__setattr__(self, name, x)


def allocate_kv4(n_seqs: int, max_pages: int, n_kv_heads: int, head_dim: int, page: int = 64, n_pages: Optional[int] = None,
                 device="cuda") -> Kv4Cache:
    """An empty cache; without n_pages, of n_seqs * max_pages pages that belong to the sequences in order (else the
    caller fills `pages`)."""
    import torch
    if page not in (16, 32, 64, 128, 256) or head_dim not in (64, 128):
        raise ValueError(f"expected a page of 16, 32, 64, 128 or 256 slots and d of 64 or 128, got {page} and {head_dim}")
    ids = torch.arange(n_seqs * max_pages, dtype=torch.int32, device=device).view(n_seqs, max_pages)
    if n_pages is not None:
        ids.fill_(-1)
    data = torch.zeros(n_seqs * max_pages if n_pages is None else n_pages, n_kv_heads, page // 16, 18 * head_dim,
                       dtype=torch.uint8, device=device)
    return Kv4Cache(data, ids, torch.zeros(n_seqs, dtype=torch.int32, device=device))


def _kv4_dev(cache: Kv4Cache) -> int:
    """The cache's device, which has to be the current one (launches go to it)."""
    dev = cache.device
    if _torch()._C._cuda_getDevice() != dev:
        raise ValueError(f"cache on cuda:{dev}, current device is another")
    return dev


def _kv4_starts(cache, starts, dev):
    return None if starts is None else _dense(starts, "starts", _torch().int32, (cache.slot_shape[0] + 1,), dev)


def zl_kv4_write(cache: Kv4Cache, k, v, starts=None, positions=None, slot_positions=None, stream=None):
    """New tokens' keys and values [tokens, Hkv, d] (views of a fused projection will do) into the last slots of their
    sequences: sequence b brings tokens starts[b] .. starts[b + 1] - 1 (int32 [sequences + 1]; None: token b) and cache.lens
    counts them already.  positions (int32 [tokens]) with slot_positions (int32 [sequences, Hkv, cache.slots]): the slots'
    positions, which zl_kv4_evict goes by."""
    torch = _torch()
    dev = _kv4_dev(cache)
    n = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
    shape = (n, *cache.token_shape)
    pk, nk = _heads(k, "k", shape, dev)
    pv, nv = _heads(v, "v", shape, dev)
    ps = ss = None
    if positions is not None or slot_positions is not None:
        ps = _dense(positions, "positions", torch.int32, (n,), dev)
        ss = _dense(slot_positions, "slot_positions", torch.int32, cache.slot_shape, dev)
    st = load_library().zl_kv4_write(cache.desc, pk, nk, pv, nv, n, _kv4_starts(cache, starts, dev), ps, ss,
                                     _raw_stream(stream, dev))
    if st:
        _check(st, "zl_kv4_write")


def zl_kv4_read(cache: Kv4Cache, k_out, v_out, row_starts, stream=None):
    """All that the cache holds as bf16 rows: slot s of sequence b becomes row row_starts[b] + s (int64 [sequences]) of
    k_out, v_out [rows, Hkv, d]; zl_causal_attn_fwd takes them as keys and values."""
    torch = _torch()
    dev = _kv4_dev(cache)
    n = k_out.shape[0] if isinstance(k_out, torch.Tensor) and k_out.dim() == 3 else 0
    shape = (n, *cache.token_shape)
    pk, nk = _heads(k_out, "k_out", shape, dev)
    pv, nv = _heads(v_out, "v_out", shape, dev)
    st = load_library().zl_kv4_read(cache.desc, pk, nk, pv, nv, n,
                                    _dense(row_starts, "row_starts", torch.int64, (cache.slot_shape[0],), dev),
                                    _raw_stream(stream, dev))
    if st:
        _check(st, "zl_kv4_read")


def zl_kv4_attn_workspace_bytes(cache: Kv4Cache, n_q_heads: int, max_new: int = 1, weights: bool = False) -> int:
    """Scratch bytes of zl_kv4_attn_fwd."""
    key = (n_q_heads, max_new, bool(weights))
    if key not in cache.sizes:
        b = ctypes.c_int64()
        _check(load_library().zl_kv4_attn_workspace(cache.desc, n_q_heads, max_new, int(key[2]), ctypes.byref(b)),
               "zl_kv4_attn_workspace")
        cache.sizes[key] = b.value
    return cache.sizes[key]


def zl_kv4_attn_fwd(cache: Kv4Cache, q, o, lse, workspace, scale: float, starts=None, max_new: int = 1, weights=None,
                    weights_out=None, decay: float = 1.0, stream=None):
    """Attention of the newest tokens q [tokens, Hq, d] over the cache, which holds their keys and values already, into o
    (contiguous) and lse [tokens, Hq].  starts as in zl_kv4_write; no sequence brings more than max_new tokens.
    weights_out (fp32 [sequences, Hkv, cache.slots]) becomes decay * weights plus what each slot received of the softmax,
    summed over the new tokens and the heads of its group; weights may be the same tensor, or None for zeros.
    workspace: zl_kv4_attn_workspace_bytes(cache, Hq, max_new, weights_out is not None)."""
    torch = _torch()
    dev = _kv4_dev(cache)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q: expected a CUDA tensor [tokens, Hq, d]")
    n, hq = q.shape[0], q.shape[1]
    shape = (n, hq, cache.token_shape[1])
    pq, nq = _heads(q, "q", shape, dev)
    if weights is not None and weights_out is None:
        raise ValueError("weights without weights_out")
    w = _dense(weights, "weights", torch.float32, cache.slot_shape, dev) if weights is not None else None
    wo = _dense(weights_out, "weights_out", torch.float32, cache.slot_shape, dev) if weights_out is not None else None
    st = load_library().zl_kv4_attn_fwd(
        cache.desc, pq, nq, n, hq, _kv4_starts(cache, starts, dev), max_new, _dense(o, "o", torch.bfloat16, shape, dev),
        _dense(lse, "lse", torch.float32, shape[:2], dev), w, wo, decay,
        _scratch(workspace, "workspace", zl_kv4_attn_workspace_bytes(cache, hq, max_new, wo is not None), dev), scale,
        _raw_stream(stream, dev))
    if st:
        _check(st, "zl_kv4_attn_fwd")


def zl_kv4_evict_workspace_bytes(cache: Kv4Cache) -> int:
    """Scratch bytes of zl_kv4_evict."""
    if "evict" not in cache.sizes:
        b = ctypes.c_int64()
        _check(load_library().zl_kv4_evict_workspace(cache.desc, ctypes.byref(b)), "zl_kv4_evict_workspace")
        cache.sizes["evict"] = b.value
    return cache.sizes["evict"]


def _kv4_check_budget(keep, recent):
    if not 1 <= keep < 1 << 31 or not 0 <= recent < 1 << 31:
        _check(ZL_ERR_INVALID_ARG, f"keep {keep}, recent {recent}")


def zl_kv4_evict(cache: Kv4Cache, weights, positions, keep: int, recent: int, workspace, weights_out=None, positions_out=None,
                 stream=None):
    """Every head of a sequence longer than `keep` keeps `keep` slots: those among the last `recent` positions first, then
    the largest weights (ties: the lower slot); survivors from behind move into the slots given up.  weights (fp32),
    positions (int32): [sequences, Hkv, cache.slots]; their new contents go to weights_out, positions_out (None: in
    place).  The new lengths are cache.lens.clamp(max=keep), which the caller sets."""
    torch = _torch()
    dev = _kv4_dev(cache)
    w = _dense(weights, "weights", torch.float32, cache.slot_shape, dev)
    ps = _dense(positions, "positions", torch.int32, cache.slot_shape, dev)
    _kv4_check_budget(keep, recent)
    wo = w if weights_out is None else _dense(weights_out, "weights_out", torch.float32, cache.slot_shape, dev)
    po = ps if positions_out is None else _dense(positions_out, "positions_out", torch.int32, cache.slot_shape, dev)
    st = load_library().zl_kv4_evict(cache.desc, w, ps, keep, recent, wo, po,
                                     _scratch(workspace, "workspace", zl_kv4_evict_workspace_bytes(cache), dev),
                                     _raw_stream(stream, dev))
    if st:
        _check(st, "zl_kv4_evict")


def zl_kv4_get_device_status(cache: Kv4Cache) -> int:
    """ZL_KV4_* bits of what calls on this cache had to leave out since the last query.  Waits for all of the device's streams;
    calls sent by other threads meanwhile may be told of now, in the next query, or not at all."""
    torch = _torch()
    torch.cuda.synchronize(cache.device)
    s = int(cache.status.item())
    if s:
        cache.status.zero_()
        torch.cuda.current_stream(cache.device).synchronize()  # calls on other streams come behind it
    return s


def allocate_kv4_attention(cache: Kv4Cache, n_tokens: int, n_q_heads: int, max_new: int = 1, evicts: bool = False,
                           state: Optional[Dict[str, "object"]] = None) -> Dict[str, "object"]:
    """Buffers of qkv_attention_cached for n_tokens new tokens, at most max_new of a sequence; evicts: with the slots'
    accumulated weights and positions, which belong to the cache's sequences and live as long as they do.  state: buffers
    that hold them already, for calls of other sizes on the same sequences (a prompt's, which without evicts need no room
    for its scores)."""
    import torch
    heads, d = cache.token_shape
    device = cache.data.device
    if state is not None:
        _dense(state["weights"], "state's weights", torch.float32, cache.slot_shape, cache.device)
        _dense(state["positions"], "state's positions", torch.int32, cache.slot_shape, cache.device)
    bf = dict(dtype=torch.bfloat16, device=device)
    ws = zl_kv4_attn_workspace_bytes(cache, n_q_heads, max_new, evicts)
    if evicts:
        ws = max(ws, zl_kv4_evict_workspace_bytes(cache))
    out = {"q": torch.empty(n_tokens, n_q_heads, d, **bf), "k": torch.empty(n_tokens, heads, d, **bf),
           "o": torch.empty(n_tokens, n_q_heads, d, **bf),
           "lse": torch.empty(n_tokens, n_q_heads, dtype=torch.float32, device=device),
           "workspace": torch.empty(max(16, ws), dtype=torch.uint8, device=device)}
    if evicts or state is not None:
        out["zeros"] = torch.zeros(n_tokens, dtype=torch.int32, device=device)
    if state is not None:
        out["weights"], out["positions"] = state["weights"], state["positions"]
    elif evicts:
        out["weights"] = torch.zeros(cache.slot_shape, dtype=torch.float32, device=device)
        out["positions"] = torch.zeros(cache.slot_shape, dtype=torch.int32, device=device)
    return out


def qkv_attention_cached(cache: Kv4Cache, qkv, positions, table: Optional[RotaryTable], scale: float, bufs: dict, q_weight=None,
                         k_weight=None, eps: float = 1e-6, starts=None, max_new: int = 1, keep: Optional[int] = None,
                         recent: int = 0, decay: float = 1.0, stream=None) -> dict:
    """A serving step from a projection's output qkv [tokens, Hq + 2 Hkv, d]: queries and keys normalised where weights are
    given and rotated, keys and values into the 4-bit cache, attention of the new tokens over it (bufs["o"],
    bufs["lse"]).  starts, max_new as in zl_kv4_attn_fwd; cache.lens counts the new tokens already.  With keep, sequences
    live on that many slots: the step's softmax weights are added to bufs["weights"] (decay * the sums so far), every
    head keeps its `keep` slots, and cache.lens becomes no more than that.  One captured graph serves every step.
    Without keep, buffers that hold weights and positions are brought up to date all the same: the new tokens' positions are
    noted and their slots' weights begin at 0, so that a prompt may enter this way and its steps go on with keep.  (With keep
    a prompt's rows are attended 16 at a time and every score is kept until the end; keep=cache.slots adds up weights and
    evicts nothing.)"""
    torch = _torch()
    heads, d = cache.token_shape
    if not isinstance(qkv, torch.Tensor) or qkv.dim() != 3 or qkv.shape[1] <= 2 * heads or qkv.shape[2] != d:
        raise ValueError(f"qkv: expected [tokens, Hq + {2 * heads}, {d}], got {tuple(getattr(qkv, 'shape', ()))}")
    w, at = bufs.get("weights"), bufs.get("positions")
    if keep is not None and w is None:
        raise ValueError("keep: needs buffers that were allocated with evicts=True")
    if w is not None and (not isinstance(positions, torch.Tensor) or positions.numel() != qkv.shape[0]):
        raise ValueError("buffers with weights: need one position a token")
    n, hq, dev = qkv.shape[0], qkv.shape[1] - 2 * heads, _kv4_dev(cache)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:]
    # all that one of the calls would refuse is refused here, before the first of them changes anything
    nbytes = zl_kv4_attn_workspace_bytes(cache, hq, max_new, keep is not None)
    if keep is not None:
        _kv4_check_budget(keep, recent)
        nbytes = max(nbytes, zl_kv4_evict_workspace_bytes(cache))
        if cache.slot_shape[0] > 65535:
            _check(ZL_ERR_UNSUPPORTED, "keep, more than 65535 sequences")
    (pq, nq), (pk, nk) = _heads(bufs["q"], "q", (n, hq, d), dev), _heads(bufs["k"], "k", (n, heads, d), dev)
    pv, nv = _heads(v, "qkv", (n, heads, d), dev)
    po, plse = _dense(bufs["o"], "o", torch.bfloat16, (n, hq, d), dev), _dense(bufs["lse"], "lse", torch.float32, (n, hq), dev)
    ws, ps = _scratch(bufs["workspace"], "workspace", nbytes, dev), _kv4_starts(cache, starts, dev)
    pw = pat = ppos = pzero = None
    if w is not None:
        pw = _dense(w, "weights", torch.float32, cache.slot_shape, dev)
        pat = _dense(at, "positions", torch.int32, cache.slot_shape, dev)
        ppos = _dense(positions.view(-1), "positions", torch.int32, (n,), dev)
        pzero = _dense(bufs["zeros"], "zeros", torch.int32, (n,), dev) if keep is None else None
    if n and (pq | pk | pv | po | ws | 2 * nq | 2 * nk | 2 * nv) % 16:
        _check(ZL_ERR_ALIGN, "qkv, q, k, o, workspace")
    scale32, decay32 = ctypes.c_float(scale).value, ctypes.c_float(decay).value
    if not 2.0 ** -126 <= scale32 < float("inf") or decay32 - decay32 != 0.0 or (starts is None and n != cache.slot_shape[0]):
        _check(ZL_ERR_INVALID_ARG, "scale, decay, tokens without starts")
    for of_q, of_k, norm in _sides(q_weight, k_weight):
        zl_qk_rope_fwd(q if of_q else None, k if of_k else None, bufs["q"] if of_q else None, bufs["k"] if of_k else None,
                       positions, table, norm, q_weight if of_q else None, k_weight if of_k else None, eps, stream)
    lib, raw, desc = load_library(), _raw_stream(stream, dev), cache.desc
    _check(lib.zl_kv4_write(desc, pk, nk, pv, nv, n, ps, ppos, pat, raw), "zl_kv4_write")
    if keep is None:
        if w is not None:  # the same tokens' slots of the weights: 0, which has the bits of the position 0
            _check(lib.zl_kv4_write(cache.no_rows, pk, nk, pv, nv, n, ps, pzero, pw, raw), "zl_kv4_write")
        _check(lib.zl_kv4_attn_fwd(desc, pq, nq, n, hq, ps, max_new, po, plse, None, None, 1.0, ws, scale, raw), "zl_kv4_attn_fwd")
        return bufs
    _check(lib.zl_kv4_attn_fwd(desc, pq, nq, n, hq, ps, max_new, po, plse, pw, pw, decay, ws, scale, raw), "zl_kv4_attn_fwd")
    _check(lib.zl_kv4_evict(desc, pw, pat, keep, recent, pw, pat, ws, raw), "zl_kv4_evict")
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(raw, cache.data.device)
    with torch.cuda.stream(stream):  # None: the current one
        cache.lens.clamp_(max=keep)
    return bufs


# ---------------------------------------------------------------- host placement slice
def catalog_cut(buckets):
    """zl_catalog_cut over [(seq_len, count, time, mem), ...] sorted by time: returns
    (k_star, dispersion); buckets[:k_star] are fillers, the rest anchors."""
    arr = (zl_bucket * len(buckets))(*[zl_bucket(int(L), int(n), float(t), float(m)) for (L, n, t, m) in buckets])
    k = ctypes.c_int32()
    disp = ctypes.c_double()
    _check(load_library().zl_catalog_cut(arr, len(buckets), ctypes.byref(k), ctypes.byref(disp)), "zl_catalog_cut")
    return k.value, disp.value


def pack_fillers(filler_time, filler_mem, n_ranks, rank_time=None, rank_mem=None, F=0.0, M_cap=1.0):
    """zl_pack_fillers: returns (assign, final_time, final_mem, n_overflow, makespan)."""
    D = ctypes.c_double
    n = len(filler_time)
    ft = (D * max(n, 1))(*map(float, filler_time))
    fm = (D * max(n, 1))(*map(float, filler_mem))
    rt = (D * n_ranks)(*map(float, rank_time)) if rank_time is not None else None
    rm = (D * n_ranks)(*map(float, rank_mem)) if rank_mem is not None else None
    assign = (ctypes.c_int32 * max(n, 1))()
    out_t, out_m = (D * n_ranks)(), (D * n_ranks)()
    over, mk = ctypes.c_int32(), D()
    _check(load_library().zl_pack_fillers(ft, fm, n, n_ranks, rt, rm, float(F), float(M_cap), assign, out_t, out_m,
                                          ctypes.byref(over), ctypes.byref(mk)), "zl_pack_fillers")
    return list(assign[:n]), list(out_t), list(out_m), over.value, mk.value

