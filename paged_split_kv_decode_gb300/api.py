"""Thin Python binding over the C ABI (include/psd.h).

The functions keep the C names and only marshal arguments: torch tensors become
device pointers, numpy int32 arrays become host pointers, the current torch stream
becomes the CUDA stream.  Every step of the decode path (planning included) runs in
``libpsd.so``; nothing here computes any part of it.
"""
from __future__ import annotations

import ctypes as C
import struct
from dataclasses import dataclass

import numpy as np
import torch

from . import _lib as L


def _ptr_i32(a: np.ndarray):
    return a.ctypes.data_as(L.P_i32)


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


# The current stream's raw handle without building a torch.cuda.Stream object (that
# costs about 3 us a call on a Grace host, the getter below about 0.4 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> C.c_void_p:
    if stream is None:
        if _raw_stream is not None:
            return C.c_void_p(_raw_stream(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return C.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))


def _new_fault(device, stream) -> torch.Tensor:
    """An int32 fault word that is 0 before what comes next on the call's stream."""
    if stream is None or torch.device(device).type != "cuda":
        return torch.zeros(1, dtype=torch.int32, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) \
            else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.zeros(1, dtype=torch.int32, device=device)


def _dev_ptr(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dev_or_pinned_ptr(t: torch.Tensor, name: str) -> int:
    """A CUDA tensor, or a pinned host tensor the kernels reach over the host link
    (the pointer is the same on both sides)."""
    if isinstance(t, torch.Tensor) and t.is_cuda:
        return _dev_ptr(t, name)
    if isinstance(t, torch.Tensor) and t.device.type == "cpu" and t.is_pinned():
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()
    return _dev_ptr(t, name)


def _out_ptr(t: torch.Tensor, name: str) -> int:
    """Decode outputs may be pinned host tensors: the merge kernel then stores them
    into host memory directly."""
    return _dev_or_pinned_ptr(t, name)


def kv_dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return L.PSD_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return L.PSD_FP8_E4M3
    raise ValueError(f"unsupported KV dtype {t.dtype}")


class Context:
    """A psd_ctx bound to one CUDA device."""

    def __init__(self, device=None):
        lib = L.load()
        dev = torch.cuda.current_device() if device is None else int(device)
        self._h = C.c_void_p()
        L.check(lib.psd_create(C.byref(self._h), dev))
        self.device = dev

    @property
    def handle(self):
        return self._h

    def set_partial_kernel(self, kind: str):
        """psd_set_partial_kernel: 'auto', 'cuda_core' or 'tensor_core'."""
        code = {"auto": L.PSD_KERNEL_AUTO, "cuda_core": L.PSD_KERNEL_CUDA_CORE,
                "tensor_core": L.PSD_KERNEL_TENSOR_CORE}[kind]
        L.check(L.load().psd_set_partial_kernel(self._h, code))

    def set_level0_kernel(self, kind: str):
        """psd_set_level0_kernel: 'auto', 'mma_sync' or 'tcgen05' for the stacked
        level-0 rows of a cascade."""
        code = {"auto": 0, "mma_sync": 1, "tcgen05": 2}[kind]
        L.check(L.load().psd_set_level0_kernel(self._h, code))

    def test_withhold_loads(self, from_tile: int, wait_limit_cycles: int = 0):
        """psd_test_withhold_loads: a testing aid that makes the partial kernels' waits
        for an item's tiles from `from_tile` on run out, and the streaming merge's waits
        for a CTA's input rows from that index on (from_tile < 0 switches it off)."""
        L.check(L.load().psd_test_withhold_loads(self._h, int(from_tile), int(wait_limit_cycles)))

    def set_timing(self, enable: bool = True):
        """psd_set_timing: CUDA events around every kernel the library launches."""
        L.check(L.load().psd_set_timing(self._h, int(bool(enable))))

    def kernel_times(self) -> dict:
        """psd_get_kernel_times of the most recent call, in milliseconds."""
        a, b, c = C.c_float(), C.c_float(), C.c_float()
        L.check(L.load().psd_get_kernel_times(self._h, C.byref(a), C.byref(b), C.byref(c)))
        return {"level0_ms": a.value, "partial_ms": b.value, "merge_ms": c.value}

    def autotune_tile(self, args: L.DecodeArgs, table: "HostTable", tiles, o: torch.Tensor, lse: torch.Tensor,
                      workspace: torch.Tensor, enable: int = 1, min_shared_pages: int = 16, min_members: int = 2,
                      reps: int = 5, stream=None):
        """psd_autotune_tile: times cascade_decode per candidate tile (cold L2) and
        records the fastest for this shape bucket.  Returns (best_tile, [mean ms])."""
        t = np.ascontiguousarray(tiles, dtype=np.int32)
        ms = (C.c_float * len(t))()
        best = C.c_int32()
        L.check(L.load().psd_autotune_tile(
            self._h, C.byref(args), C.byref(table.c), t.ctypes.data_as(L.P_i32), len(t), int(enable),
            int(min_shared_pages), int(min_members), int(reps), _dev_ptr(o, "o"), _dev_ptr(lse, "lse"),
            _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(), _stream(stream),
            C.byref(best), ms))
        return best.value, [float(x) for x in ms]

    def tuned_tile(self, args: L.DecodeArgs, table: "HostTable", default_tile: int, enable: int = 1,
                   min_shared_pages: int = 16, min_members: int = 2) -> int:
        """psd_tuned_tile: the tile recorded for this batch's shape bucket, else default_tile."""
        return int(L.load().psd_tuned_tile(self._h, C.byref(args), C.byref(table.c), int(enable),
                                           int(min_shared_pages), int(min_members), int(default_tile)))

    def counters(self) -> dict:
        c = L.Counters()
        L.check(L.load().psd_get_counters(self._h, C.byref(c)))
        return {k: getattr(c, k) for k, _ in L.Counters._fields_}

    def close(self):
        if self._h:
            L.load().psd_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HostTable:
    """A host CSR page table kept alive for the C ABI."""

    def __init__(self, page_indptr, page_indices, last_page_len, page_size: int):
        self.indptr = _i32(page_indptr)
        self.indices = _i32(page_indices)
        self.last = _i32(last_page_len)
        self.page_size = int(page_size)
        self.c = L.PageTable(_ptr_i32(self.indptr), _ptr_i32(self.indices), _ptr_i32(self.last),
                             int(self.indptr.shape[0] - 1), self.page_size)

    @property
    def batch(self):
        return int(self.indptr.shape[0] - 1)

    @property
    def nnz(self):
        return int(self.indptr[-1])


def split_plan(table: HostTable, tile_tokens: int):
    """psd_split_plan: flat work list -> (items [n, 4] int32, o_indptr [B+1])."""
    lib = L.load()
    cap = max(table.nnz, 1)
    items = (L.WorkItem * cap)()
    n = C.c_int32()
    o_indptr = np.zeros(table.batch + 1, dtype=np.int32)
    L.check(lib.psd_split_plan(C.byref(table.c), int(tile_tokens), items, cap, C.byref(n),
                               _ptr_i32(o_indptr)))
    arr = np.ctypeslib.as_array(C.cast(items, L.P_i32), shape=(cap * 4,)).reshape(cap, 4)
    return arr[: n.value].copy(), o_indptr


def detect_shared_prefix(table: HostTable, min_shared_pages: int = 16, min_members: int = 2):
    """detect_shared_prefix -> (members list, shared_pages, decline_reason)."""
    lib = L.load()
    members = np.zeros(max(table.batch, 1), dtype=np.int32)
    nm, sp, reason = C.c_int32(), C.c_int32(), C.c_int32()
    L.check(lib.detect_shared_prefix(C.byref(table.c), int(min_shared_pages), int(min_members),
                                     _ptr_i32(members), C.byref(nm), C.byref(sp), C.byref(reason)))
    return [int(x) for x in members[: nm.value]], int(sp.value), int(reason.value)


class Plan:
    """A psd_cascade_plan with caller-owned (numpy) arrays."""

    def __init__(self, table: HostTable):
        self.table = table
        bc, ic = C.c_int32(), C.c_int32()
        L.check(L.load().psd_plan_capacity(C.byref(table.c), C.byref(bc), C.byref(ic)))
        self.members_a = np.zeros(bc.value, dtype=np.int32)
        self.row_base_a = np.zeros(bc.value, dtype=np.int32)
        self.o_indptr_a = np.zeros(bc.value + 1, dtype=np.int32)
        self.l0 = (L.WorkItem * ic.value)()
        self.l1 = (L.WorkItem * ic.value)()
        self.c = L.CascadePlan()
        self.c.batch_capacity = bc.value
        self.c.item_capacity = ic.value
        self.c.members = _ptr_i32(self.members_a)
        self.c.member_row_base = _ptr_i32(self.row_base_a)
        self.c.l0_items = self.l0
        self.c.l1_items = self.l1
        self.c.o_indptr = _ptr_i32(self.o_indptr_a)

    def _items(self, arr, n):
        cap = self.c.item_capacity
        a = np.ctypeslib.as_array(C.cast(arr, L.P_i32), shape=(cap * 4,)).reshape(cap, 4)
        return a[:n].copy()

    @property
    def members(self):
        return [int(x) for x in self.members_a[: self.c.num_members]]

    @property
    def member_row_base(self):
        return [int(x) for x in self.row_base_a[: self.c.num_members]]

    @property
    def o_indptr(self):
        return [int(x) for x in self.o_indptr_a[: self.c.batch + 1]]

    @property
    def l0_items(self):
        return self._items(self.l0, self.c.l0_num_items)

    @property
    def l1_items(self):
        return self._items(self.l1, self.c.l1_num_items)

    @property
    def num_items(self):
        return self.c.l0_num_items + self.c.l1_num_items

    def __getattr__(self, name):
        if name in ("num_members", "shared_pages", "decline_reason", "num_rows", "tile_tokens",
                    "batch", "page_size", "l0_num_items", "l1_num_items"):
            return getattr(self.c, name)
        raise AttributeError(name)


class CachedPlan:
    """A plan owned by a PlanCache (a view of its psd_cascade_plan); valid until the
    next lookup on that cache.  Same read accessors as Plan."""

    def __init__(self, ptr, hit: bool):
        self.c = ptr.contents
        self.hit = hit

    def _i32(self, p, n):
        return [int(x) for x in np.ctypeslib.as_array(C.cast(p, L.P_i32), shape=(max(n, 1),))[:n]]

    @property
    def members(self):
        return self._i32(self.c.members, self.c.num_members)

    @property
    def member_row_base(self):
        return self._i32(self.c.member_row_base, self.c.num_members)

    @property
    def o_indptr(self):
        return self._i32(self.c.o_indptr, self.c.batch + 1)

    def _items(self, arr, n):
        if n == 0:
            return np.zeros((0, 4), dtype=np.int32)
        return np.ctypeslib.as_array(C.cast(arr, L.P_i32), shape=(n * 4,)).reshape(n, 4).copy()

    @property
    def l0_items(self):
        return self._items(self.c.l0_items, self.c.l0_num_items)

    @property
    def l1_items(self):
        return self._items(self.c.l1_items, self.c.l1_num_items)

    @property
    def num_items(self):
        return self.c.l0_num_items + self.c.l1_num_items

    def __getattr__(self, name):
        if name in ("num_members", "shared_pages", "decline_reason", "num_rows", "tile_tokens",
                    "batch", "page_size", "l0_num_items", "l1_num_items"):
            return getattr(self.c, name)
        raise AttributeError(name)


class PlanCache:
    """psd_plan_cache: plans memoised by page-table contents and KV lengths."""

    def __init__(self, capacity: int = 8):
        self._h = C.c_void_p()
        L.check(L.load().psd_plan_cache_create(C.byref(self._h), int(capacity)))

    def lookup(self, table: HostTable, tile_tokens: int, enable: int = 1, min_shared_pages: int = 16,
               min_members: int = 2, generation: int = -1) -> CachedPlan:
        """psd_plan_cache_lookup, or psd_plan_cache_lookup_gen when generation >= 0."""
        ptr = C.POINTER(L.CascadePlan)()
        hit = C.c_int32()
        L.check(L.load().psd_plan_cache_lookup_gen(self._h, int(generation), C.byref(table.c),
                                                   int(tile_tokens), int(enable), int(min_shared_pages),
                                                   int(min_members), C.byref(ptr), C.byref(hit)))
        return CachedPlan(ptr, bool(hit.value))

    def stats(self) -> dict:
        h, m, n = C.c_int64(), C.c_int64(), C.c_int32()
        L.check(L.load().psd_plan_cache_stats(self._h, C.byref(h), C.byref(m), C.byref(n)))
        return {"hits": h.value, "misses": m.value, "entries": n.value}

    def close(self):
        if self._h:
            L.load().psd_plan_cache_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def rope_append_kv(ctx: Context, q, k_nope, k_rope, v, cos_sin, positions, slot_mapping, k_pool, v_pool, *,
                   rot_dim: int, neox: bool, q_rope_col: int, page_size: int, k_scale: float = 1.0,
                   v_scale: float = 1.0, fault=None, stream=None):
    """rope_append_kv: rope q in place and write the new tokens' K/V rows into the pools.

    q [T, Hq, Dq] bf16, k_nope [T, Hkv, Dn] bf16 or None, k_rope [T, Hkv, Dr] bf16,
    v [T, Hkv, Dv] bf16 or None, cos_sin [max_position, rot_dim] f32, positions and
    slot_mapping [T] int32, pools bf16 (or uint8 fp8-e4m3 codes) [pages, page_size,
    Hkv, D].  Returns the int32 fault word tensor (the one given, or a new zero one)."""
    T = int(positions.numel())
    if fault is None:
        fault = _new_fault(k_pool.device, stream)
    for name, t in (("positions", positions), ("slot_mapping", slot_mapping)):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32")
    if cos_sin.dtype != torch.float32:
        raise TypeError("cos_sin must be float32")
    a = L.RopeAppendArgs()
    Hq = int(q.shape[1]) if q is not None else 0
    a.q = _dev_ptr(q, "q") if q is not None else None
    a.Hq, a.Dq, a.q_rope_col = Hq, (int(q.shape[2]) if q is not None else 0), int(q_rope_col)
    a.k_nope = _dev_ptr(k_nope, "k_nope") if k_nope is not None else None
    a.k_rope = _dev_ptr(k_rope, "k_rope")
    a.Hkv, a.Dk_nope, a.Dk_rope = int(k_rope.shape[1]), (int(k_nope.shape[2]) if k_nope is not None else 0), \
        int(k_rope.shape[2])
    a.v = _dev_ptr(v, "v") if v is not None else None
    a.Dv = int(v.shape[2]) if v is not None else 0
    a.rot_dim, a.neox = int(rot_dim), int(bool(neox))
    a.cos_sin = _dev_ptr(cos_sin, "cos_sin")
    a.max_position = int(cos_sin.shape[0])
    a.positions = _dev_ptr(positions, "positions")
    a.slot_mapping = _dev_ptr(slot_mapping, "slot_mapping")
    a.num_tokens = T
    a.k_pool = _dev_ptr(k_pool, "k_pool")
    a.v_pool = _dev_ptr(v_pool, "v_pool") if v_pool is not None else None
    a.num_pages, a.page_size = int(k_pool.shape[0]), int(page_size)
    a.kv_dtype = kv_dtype_code(k_pool)
    a.k_scale, a.v_scale = float(k_scale), float(v_scale)
    a.fault_dev = _dev_ptr(fault, "fault")
    L.check(L.load().rope_append_kv(ctx.handle, C.byref(a), _stream(stream)))
    return fault


class RopeFrequencies:
    """Rotary frequencies for append_tokens: inv_freq [rot_dim / 2] float64 and the factor on
    cos and sin.  `rope_frequencies` makes them; a caller's own go in as they are (copied)."""

    def __init__(self, inv_freq, magnitude: float = 1.0):
        self.inv_freq = inv_freq
        self.magnitude = float(magnitude)

    @property
    def inv_freq(self) -> np.ndarray:
        return self._f

    @inv_freq.setter
    def inv_freq(self, f):
        # the address is kept (numpy takes a microsecond for it) and changes with the array
        self._f = np.array(f, dtype=np.float64).reshape(-1)
        self._address = self._f.ctypes.data

    @property
    def rot_dim(self) -> int:
        return 2 * self._f.shape[0]

    @property
    def address(self) -> int:
        return self._address


def rope_frequencies(rot_dim: int, *, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original_max_position: int = 0, low: float = None, high: float = None) -> RopeFrequencies:
    """psd_rope_frequencies: scaling is 'plain', 'linear', 'ntk', 'yarn' or 'bands'.  low and
    high (turns within the original context) default to 1 and 32 for yarn, 1 and 4 for bands."""
    if scaling not in L.PSD_ROPE_KINDS:
        raise ValueError(f"scaling must be one of {sorted(L.PSD_ROPE_KINDS)}")
    a = L.RopeScaling(L.PSD_ROPE_KINDS[scaling], int(rot_dim), float(base), float(factor), int(original_max_position),
                      1.0 if low is None else float(low),
                      (4.0 if scaling == "bands" else 32.0) if high is None else float(high))
    f = np.zeros(max(int(rot_dim) // 2, 1), dtype=np.float64)
    m = C.c_double()
    L.check(L.load().psd_rope_frequencies(C.byref(a), f.ctypes.data_as(C.POINTER(C.c_double)), C.byref(m)))
    return RopeFrequencies(f, m.value)


def _ctx_stream(ctx: Context, stream):
    """The stream given, or the current one of the context's device (which need not be the
    current device)."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(ctx.device)
    return _stream(torch.cuda.current_stream(ctx.device) if stream is None else stream)


# The operators of a multi-token step run between other launches of a serving loop, so their
# host time counts: each fills its argument structure with one struct.pack (about 1 us on a
# Grace host; 35 ctypes field stores take 6) and asks a tensor for its device by get_device().
_APPEND = struct.Struct("@PPPqqqP9iPd5PqPPqiiffP")
_VERIFY = struct.Struct("@PPqqPPPiiiPPP")
_DECODE = struct.Struct("@PqPPPqq6i3fPi0P")
assert _APPEND.size == C.sizeof(L.AppendArgs) and _VERIFY.size == C.sizeof(L.VerifyArgs)
assert _DECODE.size == C.sizeof(L.MultiTokenArgs)


def _refuse(t, name: str, dtype, dev: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _flat(t: torch.Tensor, name: str, dtype, dev: int) -> int:
    """The address of a contiguous tensor on device `dev`."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, name, dtype, dev)
    return t.data_ptr()


def _shape(t: torch.Tensor, ndim: int, name: str):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    return shape


def _row_stride(t: torch.Tensor, shape, name: str, dtype, dev: int) -> int:
    """Elements between the rows of a tensor on device `dev` whose rows are contiguous but may
    lie apart (a view of a wider tensor)."""
    if t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, dtype, dev)
    stride, width = t.stride(), 1
    if len(stride) == 3 and stride[2] == 1 and stride[1] == shape[2] and shape[0] > 1:  # (the usual case, 0.4 us sooner)
        return stride[0]
    for d in range(len(shape) - 1, 0, -1):
        if stride[d] != width and shape[d] != 1:
            raise ValueError(f"{name}: the values of a row must be contiguous")
        width *= shape[d]
    return stride[0] if shape[0] > 1 else width


class BlockScales:
    """psd_block_scales: the scales of a cache of 8-bit blocks, uint8 k and v [num_pages,
    page_size // block, Hkv] on the device (byte e stands for 2^(e - 127), 255 for NaN); block is
    16, 32 or 64 tokens of a page.  The object keeps the tensors."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, block: int):
        self.shape = tuple(_shape(k, 3, "k scales"))
        if tuple(_shape(v, 3, "v scales")) != self.shape:
            raise ValueError("the scales of K and V must be alike, [num_pages, page_size // block, Hkv]")
        self.device = k.get_device()
        self.c = L.BlockScales(_flat(k, "k scales", torch.uint8, self.device),
                               _flat(v, "v scales", torch.uint8, self.device), int(block))
        self.k, self.v, self.block = k, v, int(block)

    def fit(self, pool_shape, dev: int):
        """Refuses pools [num_pages, page_size, Hkv, D] that these are not the scales of."""
        num_pages, page_size, Hkv = pool_shape[:3]
        if self.block < 1 or self.shape != (num_pages, page_size // self.block, Hkv):
            raise ValueError(f"scales must be [num_pages, page_size // block, Hkv] = "
                             f"{(num_pages, page_size // max(self.block, 1), Hkv)}, not {self.shape}")
        if self.device != dev:
            raise ValueError(f"the scales are on cuda:{self.device}, expected cuda:{dev}")


def append_tokens(ctx: Context, q, k, v, q_out, *, q_indptr, kv_len, page_indptr, page_indices, k_pool, v_pool,
                  rope: RopeFrequencies, neox: bool, rope_col: int = 0, positions=None, k_scale: float = 1.0,
                  v_scale: float = 1.0, scales: "BlockScales" = None, fault=None, stream=None):
    """append_tokens: rotate the new tokens' queries into q_out and append their rotated K and
    their V to the pools, at the places the device page table gives.

    q [T, Hq, D], k [T, Hkv, D], v [T, Hkv, Dv] bf16, possibly views with a token stride; q_out
    [T, Hq, D] bf16 (q and q_out None for a K/V-only append, v and v_pool None for a shared
    latent); q_indptr and page_indptr [B + 1], kv_len [B] (new tokens included), page_indices
    and positions ([T], optional) int32 on the device; pools bf16 or uint8 fp8-e4m3 codes
    [pages, page_size, Hkv, D].  scales: the pools are blocks with a scale each, which this call
    sets (append_tokens_scaled).  Returns the int32 fault word tensor (the one given, or a new
    zero one)."""
    dev, bf16, i32 = ctx.device, torch.bfloat16, torch.int32
    ks = _shape(k, 3, "k")
    T, Hkv, D = ks
    k_stride = _row_stride(k, ks, "k", bf16, dev)
    if (q is None) != (q_out is None) or (v is None) != (v_pool is None):
        raise ValueError("q goes with q_out, v with v_pool")
    q_ptr = out_ptr = q_stride = Hq = v_ptr = v_pool_ptr = v_stride = Dv = 0
    if q is not None:
        qs = _shape(q, 3, "q")
        Hq = qs[1]
        if qs[0] != T or qs[2] != D or _shape(q_out, 3, "q_out") != qs:
            raise ValueError("q and q_out must be bf16 [T, Hq, D] with k's T and D")
        q_ptr, q_stride = q.data_ptr(), _row_stride(q, qs, "q", bf16, dev)
        out_ptr = _flat(q_out, "q_out", bf16, dev)
    pool_shape = _shape(k_pool, 4, "k_pool")
    num_pages, page_size, pool_heads, pool_dim = pool_shape
    if pool_heads != Hkv or pool_dim != D:
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, D]")
    pool_type = k_pool.dtype
    if v is not None:
        vs = _shape(v, 3, "v")
        Dv = vs[2]
        if vs[0] != T or vs[1] != Hkv:
            raise ValueError("v must be [T, Hkv, Dv] with k's T and Hkv")
        if _shape(v_pool, 4, "v_pool") != pool_shape[:3] + (Dv,) or v_pool.dtype is not pool_type:
            raise ValueError("v_pool must be [num_pages, page_size, Hkv, Dv] of k_pool's type")
        v_ptr, v_stride = v.data_ptr(), _row_stride(v, vs, "v", bf16, dev)
        v_pool_ptr = _flat(v_pool, "v_pool", pool_type, dev)
    if fault is None:
        fault = _new_fault(k_pool.device, stream)
    tables = (_flat(q_indptr, "q_indptr", i32, dev), _flat(kv_len, "kv_len", i32, dev),
              0 if positions is None else _flat(positions, "positions", i32, dev),
              _flat(page_indptr, "page_indptr", i32, dev), _flat(page_indices, "page_indices", i32, dev))
    B = kv_len.numel()
    if q_indptr.numel() != B + 1 or page_indptr.numel() != B + 1:
        raise ValueError(f"q_indptr and page_indptr must hold {B + 1} values")
    if positions is not None and positions.numel() != T:
        raise ValueError(f"positions must hold {T} values")
    args = _APPEND.pack(
        q_ptr, k.data_ptr(), v_ptr, q_stride, k_stride, v_stride, out_ptr, T, B, Hq, Hkv, D, Dv, rope_col,
        rope.rot_dim, 1 if neox else 0, rope.address, rope.magnitude, *tables, page_indices.numel(),
        _flat(k_pool, "k_pool", pool_type, dev), v_pool_ptr, num_pages, page_size, kv_dtype_code(k_pool), k_scale,
        v_scale, _flat(fault, "fault", i32, dev))
    if scales is None:
        status = L.load().append_tokens(ctx._h, args, _ctx_stream(ctx, stream))
    else:
        scales.fit(pool_shape, dev)
        status = L.load().append_tokens_scaled(ctx._h, args, scales.c, _ctx_stream(ctx, stream))
    if status:
        L.check(status)
    return fault


class MultiTokenPlan:
    """A psd_multi_token_plan with caller-owned arrays."""

    def __init__(self, capacity: int):
        self.requests_a = (L.TokenRequest * max(int(capacity), 1))()
        self.c = L.MultiTokenPlan()
        self.c.batch_capacity = int(capacity)
        self.c.requests = self.requests_a

    @property
    def requests(self):
        return [(r.token0, r.num_new, r.page_off, r.kv_len) for r in self.requests_a[: self.c.batch]]

    def __getattr__(self, name):
        if name in ("batch", "page_size", "num_tokens", "max_new"):
            return getattr(self.c, name)
        raise AttributeError(name)


def plan_multi_token(table: HostTable, q_indptr, Hq: int = None, Hkv: int = None) -> MultiTokenPlan:
    """psd_plan_multi_token: the table after the append, and the new tokens' CSR (host).  Hq
    and Hkv, when given, are checked (Hq % Hkv == 0); the plan does not depend on them."""
    qi = _i32(q_indptr)
    if qi.shape != (table.batch + 1,):
        raise ValueError("q_indptr must hold batch + 1 values")
    if Hq is not None and Hkv is not None and (Hkv < 1 or Hq < 1 or Hq % Hkv):
        raise ValueError("need Hq % Hkv == 0")
    plan = MultiTokenPlan(table.batch)
    L.check(L.load().psd_plan_multi_token(C.byref(table.c), _ptr_i32(qi), C.byref(plan.c)))
    return plan


def multi_token_workspace(ctx: Context, plan: MultiTokenPlan, D: int, device) -> torch.Tensor:
    """A workspace for multi_token_decode: its size depends on the head dim alone, so one
    serves every plan."""
    n = int(L.load().psd_multi_token_workspace_bytes(ctx.handle, int(D)))
    return torch.empty(n, dtype=torch.uint8, device=device)


def multi_token_args(q, k_pool, v_pool, page_indices_dev, *, sm_scale: float, k_scale: float = 1.0,
                     v_scale: float = 1.0, tree_mask=None, scales: BlockScales = None) -> L.MultiTokenArgs:
    """psd_multi_token_args from device tensors: q [T, Hq, D] bf16 (possibly a view with a
    token stride), pools [pages, page_size, Hkv, D] bf16 or uint8 fp8-e4m3 codes, page_indices
    int32, tree_mask [T] int64 (64 bits a token) or None.  scales: the pools are blocks with a
    scale each (multi_token_decode then calls multi_token_decode_scaled).  The structure keeps
    the tensors."""
    shape = _shape(q, 3, "q")
    T, Hq, D = shape
    dev = q.get_device()
    stride = _row_stride(q, shape, "q", torch.bfloat16, dev)
    pool_shape, pool_type = _shape(k_pool, 4, "k_pool"), k_pool.dtype
    if _shape(v_pool, 4, "v_pool") != pool_shape or v_pool.dtype is not pool_type or pool_shape[3] != D:
        raise ValueError("k_pool and v_pool must be alike, [num_pages, page_size, Hkv, D]")
    if tree_mask is not None and (tree_mask.dtype is not torch.int64 or tree_mask.numel() != T):
        raise ValueError("tree_mask must be int64 [T]")
    fields = (q.data_ptr(), stride, _flat(k_pool, "k_pool", pool_type, dev), _flat(v_pool, "v_pool", pool_type, dev),
              _flat(page_indices_dev, "page_indices", torch.int32, dev), page_indices_dev.numel(), pool_shape[0], T, Hq,
              pool_shape[2], D, pool_shape[1], kv_dtype_code(k_pool), k_scale, v_scale, sm_scale,
              0 if tree_mask is None else _flat(tree_mask, "tree_mask", torch.int64, dev), 0)
    a = L.MultiTokenArgs.from_buffer_copy(_DECODE.pack(*fields))
    if scales is not None:
        scales.fit(pool_shape, dev)
    a.tensors, a.device, a.scales = (q, k_pool, v_pool, page_indices_dev, tree_mask), dev, scales
    return a


def multi_token_decode(ctx: Context, args: L.MultiTokenArgs, plan: MultiTokenPlan, o: torch.Tensor,
                       lse: torch.Tensor = None, workspace: torch.Tensor = None, stream=None):
    """multi_token_decode: o [T, Hq, D] bf16 or f32, lse [T, Hq] f32 (log2 units) or None;
    workspace from multi_token_workspace (a call without one is refused)."""
    dev, out_type, shape = ctx.device, o.dtype, (args.num_tokens, args.Hq, args.D)
    if args.device != dev:
        raise ValueError(f"the arguments are on cuda:{args.device}, the context on cuda:{dev}")
    args.out_f32 = out_type is torch.float32
    if not args.out_f32 and out_type is not torch.bfloat16:
        raise TypeError("o must be bf16 or f32")
    if o.shape != shape:
        raise ValueError("o must be [T, Hq, D]")
    if lse is not None and lse.shape != shape[:2]:
        raise ValueError("lse must be f32 [T, Hq]")
    rest = (plan.c, _flat(o, "o", out_type, dev), None if lse is None else _flat(lse, "lse", torch.float32, dev),
            _flat(workspace, "workspace", torch.uint8, dev), workspace.numel(), _ctx_stream(ctx, stream))
    if args.scales is None:
        status = L.load().multi_token_decode(ctx._h, args, *rest)
    else:
        status = L.load().multi_token_decode_scaled(ctx._h, args, args.scales.c, *rest)
    if status:
        L.check(status)


def verify_drafts(ctx: Context, target_probs, draft_probs, draft_tokens, draft_indptr, uniforms, num_accepted,
                  out_tokens, *, fault=None, stream=None):
    """verify_drafts: target_probs [D + B, vocab], draft_probs [D, vocab] or None (f32, rows
    possibly apart), draft_tokens [D], draft_indptr [B + 1] int32, uniforms [D + B] f32;
    num_accepted [B] and out_tokens [D + B] int32 outputs, all on the device.  Returns the
    int32 fault word tensor (the one given, or a new zero one)."""
    dev, i32, f32 = ctx.device, torch.int32, torch.float32
    shape = _shape(target_probs, 2, "target_probs")
    rows, V = shape
    t_stride = _row_stride(target_probs, shape, "target_probs", f32, dev)
    if fault is None:
        fault = _new_fault(target_probs.device, stream)
    ptrs = (_flat(draft_tokens, "draft_tokens", i32, dev), _flat(draft_indptr, "draft_indptr", i32, dev),
            _flat(uniforms, "uniforms", f32, dev))
    outs = (_flat(num_accepted, "num_accepted", i32, dev), _flat(out_tokens, "out_tokens", i32, dev),
            _flat(fault, "fault", i32, dev))
    D, B = draft_tokens.numel(), num_accepted.numel()
    if rows != D + B or uniforms.numel() != rows or out_tokens.numel() != rows or draft_indptr.numel() != B + 1:
        raise ValueError("target_probs, uniforms and out_tokens have num_drafts + batch rows, draft_indptr batch + 1")
    d_ptr = d_stride = 0
    if draft_probs is not None:
        d_shape = _shape(draft_probs, 2, "draft_probs")
        if d_shape[0] != D or d_shape[1] != V:
            raise ValueError("draft_probs must be [num_drafts, vocab]")
        d_stride = _row_stride(draft_probs, d_shape, "draft_probs", f32, dev)
        d_ptr = draft_probs.data_ptr()
    args = _VERIFY.pack(target_probs.data_ptr(), d_ptr, t_stride, d_stride, *ptrs, B, D, V, *outs)
    status = L.load().verify_drafts(ctx._h, args, _ctx_stream(ctx, stream))
    if status:
        L.check(status)
    return fault


# ------------------------------------------------------------------------------ beam search
_BEAM = struct.Struct("@PqiPP5iPPPP")
assert _BEAM.size == C.sizeof(L.BeamArgs)
_LOGITS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def beam_workspace(ctx: Context, rows: int, beams: int, k: int, device) -> torch.Tensor:
    """A workspace for beam_select calls of at most `rows` rows with these beams and k."""
    n = int(L.load().psd_beam_workspace_bytes(ctx.handle, int(rows), int(beams), int(k)))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def beam_select(ctx: Context, logits, scores, out_scores, out_rows, out_tokens, workspace, *, beams: int, finished=None,
                pad_token: int = 0, fault=None, stream=None):
    """beam_select: the k best continuations over each request's beams and the vocabulary.
    logits [rows, vocab] f32, bf16 or f16 (rows possibly apart), scores [rows] f32, finished
    [rows] uint8 or bool or None, request b's beams the rows [b * beams, (b + 1) * beams);
    out_scores f32, out_rows and out_tokens int32, all [rows / beams, k].  out_rows are numbers of
    rows, as fork_pages takes for its parents (-1: no continuation).  Returns the int32 fault word
    tensor (the one given, or a new zero one)."""
    dev, i32, f32 = ctx.device, torch.int32, torch.float32
    shape = _shape(logits, 2, "logits")
    rows, V = shape
    kind = _LOGITS.get(logits.dtype)
    if kind is None:
        raise TypeError("logits must be f32, bf16 or f16")
    stride = _row_stride(logits, shape, "logits", logits.dtype, dev)
    if beams < 1 or rows % beams:
        raise ValueError("logits must have a multiple of `beams` rows")
    out = _shape(out_tokens, 2, "out_tokens")
    if out[0] != rows // beams or _shape(out_scores, 2, "out_scores") != out or _shape(out_rows, 2, "out_rows") != out:
        raise ValueError("out_scores, out_rows and out_tokens must be [rows / beams, k]")
    if scores.numel() != rows or (finished is not None and finished.numel() != rows):
        raise ValueError("scores and finished must hold a value a row")
    if fault is None:
        fault = _new_fault(logits.device, stream)
    done = 0
    if finished is not None:
        done = _flat(finished, "finished", torch.bool if finished.dtype is torch.bool else torch.uint8, dev)
    args = _BEAM.pack(logits.data_ptr(), max(stride, V), kind, _flat(scores, "scores", f32, dev), done, rows, beams, V,
                      out[1], pad_token, _flat(out_scores, "out_scores", f32, dev), _flat(out_rows, "out_rows", i32, dev),
                      _flat(out_tokens, "out_tokens", i32, dev), _flat(fault, "fault", i32, dev))
    status = L.load().beam_select(ctx._h, args, _flat(workspace, "workspace", torch.uint8, dev), workspace.numel(),
                                  _ctx_stream(ctx, stream))
    if status:
        L.check(status)
    return fault


# ------------------------------------------------------------------------- pages of a cache
_FORK = struct.Struct("@PiiPPqPiiiPPqPPqPPiP")
_COMPACT = struct.Struct("@PqPqPPPPPiP")
assert _FORK.size == C.sizeof(L.ForkArgs) and _COMPACT.size == C.sizeof(L.CompactArgs)


class PagePools:
    """The arrays of a cache whose first axis is the page (K and V of each layer, their scales):
    contiguous tensors on one device, with equally many pages.  The object keeps them."""

    def __init__(self, tensors):
        tensors = list(tensors)
        if not tensors:
            raise ValueError("a cache has at least one array of pages")
        for t in tensors:
            if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous() or t.dim() < 1:
                raise ValueError("pools must be contiguous CUDA tensors")
            if t.shape[0] != tensors[0].shape[0] or t.get_device() != tensors[0].get_device():
                raise ValueError("pools must have equally many pages, on one device")
        self.num_pages, self.device = int(tensors[0].shape[0]), tensors[0].get_device()
        self.c = (L.PagePool * len(tensors))(
            *[L.PagePool(t.data_ptr(), t.numel() // max(self.num_pages, 1) * t.element_size()) for t in tensors])
        self.tensors, self.count, self.address = tensors, len(tensors), C.addressof(self.c)

    def fit(self, ref_count: torch.Tensor, dev: int):
        if self.device != dev:
            raise ValueError(f"the pools are on cuda:{self.device}, expected cuda:{dev}")
        if ref_count.numel() != self.num_pages:
            raise ValueError(f"ref_count must hold {self.num_pages} values")


def pages_workspace(pages: PagePools, num_new: int, device) -> torch.Tensor:
    """A workspace for fork_pages calls of at most num_new new requests (0: free_pages and
    compact_pages)."""
    n = int(L.load().psd_pages_workspace_bytes(pages.num_pages, int(num_new)))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def fork_pages(ctx: Context, pages: PagePools, parents, *, page_indptr, page_indices, kv_len, page_size: int, room: int,
               ref_count, new_indptr, new_indices, new_len, workspace, new_ref_count=None, keep_old: bool = False,
               fault=None, stream=None):
    """fork_pages: a new page table whose request i continues request parents[i] of the old one
    (-1: none) with space for `room` more tokens; pages are shared, and those that two would write
    to copied in all pools.  parents [N], page_indptr [B + 1], page_indices, kv_len [B], ref_count
    [num_pages] and the outputs new_indptr [N + 1], new_indices (capacity), new_len [N] are int32
    on the device; new_ref_count defaults to ref_count.  keep_old: the old requests live on.
    Returns the int32 fault word tensor (the one given, or a new zero one)."""
    dev, i32 = ctx.device, torch.int32
    pages.fit(ref_count, dev)
    if new_ref_count is None:
        new_ref_count = ref_count
    N, B = parents.numel(), kv_len.numel()
    if page_indptr.numel() != B + 1 or new_indptr.numel() != N + 1 or new_len.numel() != N or \
            new_ref_count.numel() != pages.num_pages:
        raise ValueError("page_indptr must hold batch + 1 values, new_indptr num_new + 1, new_len num_new, "
                         "new_ref_count num_pages")
    if fault is None:
        fault = _new_fault(ref_count.device, stream)
    args = _FORK.pack(
        _flat(parents, "parents", i32, dev), N, room, _flat(page_indptr, "page_indptr", i32, dev),
        _flat(page_indices, "page_indices", i32, dev), page_indices.numel(), _flat(kv_len, "kv_len", i32, dev), B,
        page_size, 1 if keep_old else 0, _flat(ref_count, "ref_count", i32, dev),
        _flat(new_ref_count, "new_ref_count", i32, dev), pages.num_pages, _flat(new_indptr, "new_indptr", i32, dev),
        _flat(new_indices, "new_indices", i32, dev), new_indices.numel(), _flat(new_len, "new_len", i32, dev),
        pages.address, pages.count, _flat(fault, "fault", i32, dev))
    status = L.load().fork_pages(ctx._h, args, _flat(workspace, "workspace", torch.uint8, dev), workspace.numel(),
                                 _ctx_stream(ctx, stream))
    if status:
        L.check(status)
    return fault


def free_pages(ctx: Context, page_indptr, page_indices, ref_count, workspace, *, fault=None, stream=None):
    """free_pages: lets go of every page of a table (page_indptr [B + 1], page_indices int32 on the
    device), counting ref_count down in place.  workspace: of pages_workspace.  Returns the fault
    word tensor."""
    dev, i32 = ctx.device, torch.int32
    if page_indptr.numel() < 1:
        raise ValueError("page_indptr must hold batch + 1 values")
    if fault is None:
        fault = _new_fault(ref_count.device, stream)
    status = L.load().free_pages(
        ctx._h, _flat(page_indptr, "page_indptr", i32, dev), _flat(page_indices, "page_indices", i32, dev),
        page_indices.numel(), page_indptr.numel() - 1, _flat(ref_count, "ref_count", i32, dev), ref_count.numel(),
        _flat(fault, "fault", i32, dev), _flat(workspace, "workspace", torch.uint8, dev), workspace.numel(),
        _ctx_stream(ctx, stream))
    if status:
        L.check(status)
    return fault


def compact_pages(ctx: Context, pages: PagePools, page_indices, ref_count, *, num_live, workspace, new_indices=None,
                  new_ref_count=None, page_map=None, fault=None, stream=None):
    """compact_pages: moves the live pages to the front of all pools, and the entries of
    page_indices (any number of tables, one behind the other) and ref_count with them, in place
    unless new_indices and new_ref_count are given.  num_live [1] int32 gets their number, page_map
    [num_pages] (optional) each old page's new id.  Returns the fault word tensor."""
    dev, i32 = ctx.device, torch.int32
    pages.fit(ref_count, dev)
    new_indices = page_indices if new_indices is None else new_indices
    new_ref_count = ref_count if new_ref_count is None else new_ref_count
    if new_indices.numel() != page_indices.numel() or new_ref_count.numel() != pages.num_pages or \
            (page_map is not None and page_map.numel() != pages.num_pages) or num_live.numel() != 1:
        raise ValueError("new_indices is as long as page_indices, new_ref_count and page_map hold num_pages values, "
                         "num_live one")
    if fault is None:
        fault = _new_fault(ref_count.device, stream)
    args = _COMPACT.pack(
        _flat(page_indices, "page_indices", i32, dev), page_indices.numel(), _flat(ref_count, "ref_count", i32, dev),
        pages.num_pages, _flat(new_indices, "new_indices", i32, dev), _flat(new_ref_count, "new_ref_count", i32, dev),
        _flat(num_live, "num_live", i32, dev), 0 if page_map is None else _flat(page_map, "page_map", i32, dev),
        pages.address, pages.count, _flat(fault, "fault", i32, dev))
    status = L.load().compact_pages(ctx._h, args, _flat(workspace, "workspace", torch.uint8, dev), workspace.numel(),
                                    _ctx_stream(ctx, stream))
    if status:
        L.check(status)
    return fault


def copy_pages(ctx: Context, pages: PagePools, src, dst, *, fault=None, stream=None):
    """copy_pages: page src[i] to page dst[i] in all pools (int32 on the device).  Returns the fault
    word tensor."""
    dev, i32 = ctx.device, torch.int32
    if pages.device != dev:
        raise ValueError(f"the pools are on cuda:{pages.device}, expected cuda:{dev}")
    if src.numel() != dst.numel():
        raise ValueError("src and dst must be equally long")
    if fault is None:
        fault = _new_fault(src.device, stream)
    status = L.load().copy_pages(ctx._h, pages.address, pages.count, pages.num_pages, _flat(src, "src", i32, dev),
                                 _flat(dst, "dst", i32, dev), src.numel(), _flat(fault, "fault", i32, dev),
                                 _ctx_stream(ctx, stream))
    if status:
        L.check(status)
    return fault


def build_cascade_plan(table: HostTable, members, shared_pages: int, tile_tokens: int) -> Plan:
    plan = Plan(table)
    m = _i32(list(members) if len(members) else [0])
    L.check(L.load().build_cascade_plan(C.byref(table.c), _ptr_i32(m), len(members),
                                        int(shared_pages), int(tile_tokens), C.byref(plan.c)))
    return plan


def plan_decode(table: HostTable, tile_tokens: int, enable: int = 1, min_shared_pages: int = 16,
                min_members: int = 2, plan: Plan = None) -> Plan:
    """psd_plan_decode: detection + cascade plan, or the flat plan with a reason."""
    plan = plan if plan is not None else Plan(table)
    L.check(L.load().psd_plan_decode(C.byref(table.c), int(tile_tokens), int(enable),
                                     int(min_shared_pages), int(min_members), C.byref(plan.c)))
    return plan


def cascade_env_enabled(fallback: int = 0) -> int:
    return int(L.load().psd_cascade_env_enabled(int(fallback)))


def workspace_bytes(batch: int, num_items: int, num_rows: int, Hq: int, Dv: int) -> int:
    return int(L.load().psd_workspace_bytes(int(batch), int(num_items), int(num_rows), int(Hq), int(Dv)))


def decode_args(q, k_pool, v_pool, page_indices_dev, *, num_pages: int, page_size: int,
                Hkv: int, Dv: int, sm_scale: float, k_scale: float = 1.0,
                v_scale: float = 1.0) -> L.DecodeArgs:
    """psd_decode_args from device tensors (v_pool is k_pool for a shared latent).
    q and page_indices may instead be pinned host tensors, read by the partial kernels
    over the host link (not by the MLA latent kernel, which takes device q)."""
    a = L.DecodeArgs()
    a.q = _dev_or_pinned_ptr(q, "q")
    a.k_pool = _dev_ptr(k_pool, "k_pool")
    a.v_pool = _dev_ptr(v_pool, "v_pool")
    if page_indices_dev.dtype != torch.int32:
        raise ValueError("page_indices must be int32")
    a.page_indices_dev = _dev_or_pinned_ptr(page_indices_dev, "page_indices")
    a.num_page_indices = int(page_indices_dev.numel())
    a.num_pages = int(num_pages)
    a.batch, a.Hq, a.Dqk = (int(x) for x in q.shape)
    a.Hkv = int(Hkv)
    a.Dv = int(Dv)
    a.page_size = int(page_size)
    a.kv_dtype = kv_dtype_code(k_pool)
    a.k_scale, a.v_scale, a.sm_scale = float(k_scale), float(v_scale), float(sm_scale)
    return a


def paged_decode_partial(ctx: Context, args: L.DecodeArgs, items: np.ndarray, v_out: torch.Tensor,
                         lse_out: torch.Tensor, workspace: torch.Tensor, stream=None):
    """paged_decode_partial over a host work list ([n, 4] int32 rows
    (q_index, page_off, n_tokens, out_row))."""
    it = _i32(items).reshape(-1, 4)
    n = it.shape[0]
    arr = (L.WorkItem * max(n, 1)).from_buffer_copy(it.tobytes() or bytes(16))
    L.check(L.load().paged_decode_partial(
        ctx.handle, C.byref(args), arr, n, _dev_ptr(v_out, "v_out"), _dev_ptr(lse_out, "lse_out"),
        int(v_out.shape[0]), _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def merge_states(ctx: Context, v_in: torch.Tensor, lse_in: torch.Tensor, o_indptr_dev: torch.Tensor,
                 v_out: torch.Tensor, lse_out: torch.Tensor = None, stream=None):
    """merge_states: v_in [N, H, D] f32, lse_in [N, H] f32, o_indptr [M+1] int32 (device)."""
    M = int(o_indptr_dev.numel()) - 1
    H, D = int(v_in.shape[1]), int(v_in.shape[2])
    L.check(L.load().merge_states(
        ctx.handle, _dev_ptr(v_in, "v_in"), _dev_ptr(lse_in, "lse_in"),
        _dev_ptr(o_indptr_dev, "o_indptr"), M, H, D, _dev_ptr(v_out, "v_out"),
        None if lse_out is None else _dev_ptr(lse_out, "lse_out"), _stream(stream)))


def cascade_decode(ctx: Context, args: L.DecodeArgs, plan: Plan, o: torch.Tensor,
                   lse: torch.Tensor = None, workspace: torch.Tensor = None, stream=None) -> dict:
    """cascade_decode (flat when the plan has no members); returns the path stats."""
    stats = L.CascadeStats()
    L.check(L.load().cascade_decode(
        ctx.handle, C.byref(args), C.byref(plan.c), _out_ptr(o, "o"),
        None if lse is None else _out_ptr(lse, "lse"), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), C.byref(stats), _stream(stream)))
    return {k: getattr(stats, k) for k, _ in L.CascadeStats._fields_}


def cascade_decode_no_alloc(ctx: Context, args: L.DecodeArgs, plan: Plan, o: torch.Tensor,
                            lse: torch.Tensor = None, fault_bits: torch.Tensor = None,
                            stream=None) -> dict:
    """cascade_decode_no_alloc: cascade_decode without a workspace, for callers that
    cannot allocate device memory (scratch lives in the library's fixed 16 MiB
    device array; see include/psd.h).  fault_bits: optional device int32[1]."""
    stats = L.CascadeStats()
    L.check(L.load().cascade_decode_no_alloc(
        ctx.handle, C.byref(args), C.byref(plan.c), _dev_ptr(o, "o"),
        None if lse is None else _dev_ptr(lse, "lse"),
        None if fault_bits is None else _dev_ptr(fault_bits, "fault_bits"),
        C.byref(stats), _stream(stream)))
    return {k: getattr(stats, k) for k, _ in L.CascadeStats._fields_}


def check_device_error(ctx: Context, workspace: torch.Tensor, stream=None) -> int:
    """psd_check_device_error: raises PsdError on a flagged device fault."""
    bits = C.c_int32()
    st = L.load().psd_check_device_error(ctx.handle, _dev_ptr(workspace, "workspace"), _ctx_stream(ctx, stream),
                                         C.byref(bits))
    if st != L.PSD_OK:
        err = L.PsdError(st, L.load().psd_last_error().decode(errors="replace"))
        err.fault_bits = int(bits.value)
        raise err
    return int(bits.value)


class NestedPlan:
    """A psd_nested_plan with caller-owned (numpy) arrays."""

    def __init__(self, table: HostTable, max_levels: int):
        self.table = table
        bc, ec, sc, ic = C.c_int32(), C.c_int32(), C.c_int32(), C.c_int32()
        L.check(L.load().psd_plan_nested_capacity(C.byref(table.c), int(max_levels), C.byref(bc), C.byref(ec),
                                                  C.byref(sc), C.byref(ic)))
        self.segments_a = (L.Segment * sc.value)()
        self.members_a = np.zeros(ec.value, dtype=np.int32)
        self.row_base_a = np.zeros(ec.value, dtype=np.int32)
        self.o_indptr_a = np.zeros(bc.value + 1, dtype=np.int32)
        self.l0 = (L.WorkItem * ic.value)()
        self.l1 = (L.WorkItem * ic.value)()
        self.c = L.NestedPlan()
        self.c.batch_capacity, self.c.entry_capacity = bc.value, ec.value
        self.c.segment_capacity, self.c.item_capacity = sc.value, ic.value
        self.c.segments = self.segments_a
        self.c.members = _ptr_i32(self.members_a)
        self.c.member_row_base = _ptr_i32(self.row_base_a)
        self.c.l0_items = self.l0
        self.c.l1_items = self.l1
        self.c.o_indptr = _ptr_i32(self.o_indptr_a)

    def _items(self, arr, n):
        cap = self.c.item_capacity
        a = np.ctypeslib.as_array(C.cast(arr, L.P_i32), shape=(cap * 4,)).reshape(cap, 4)
        return a[:n].copy()

    @property
    def segments(self):
        return [(s.first_member, s.num_members, s.start_page, s.shared_pages, s.first_item, s.num_items)
                for s in self.segments_a[: self.c.num_segments]]

    @property
    def members(self):
        return [int(x) for x in self.members_a[: self.c.num_entries]]

    @property
    def member_row_base(self):
        return [int(x) for x in self.row_base_a[: self.c.num_entries]]

    @property
    def o_indptr(self):
        return [int(x) for x in self.o_indptr_a[: self.c.batch + 1]]

    @property
    def l0_items(self):
        return self._items(self.l0, self.c.l0_num_items)

    @property
    def l1_items(self):
        return self._items(self.l1, self.c.l1_num_items)

    @property
    def num_items(self):
        return self.c.l0_num_items + self.c.l1_num_items

    def __getattr__(self, name):
        if name in ("num_segments", "num_entries", "decline_reason", "num_rows", "tile_tokens", "batch",
                    "page_size", "max_levels", "l0_num_items", "l1_num_items"):
            return getattr(self.c, name)
        raise AttributeError(name)


def plan_nested(table: HostTable, tile_tokens: int, enable: int = 1, min_shared_pages: int = 16,
                min_members: int = 2, max_levels: int = 2) -> NestedPlan:
    """psd_plan_nested: several disjoint and nested shared spans (see include/psd.h)."""
    plan = NestedPlan(table, max_levels)
    L.check(L.load().psd_plan_nested(C.byref(table.c), int(tile_tokens), int(enable), int(min_shared_pages),
                                     int(min_members), int(max_levels), C.byref(plan.c)))
    return plan


def nested_workspace_for(plan: NestedPlan, Hq: int, Dv: int, device) -> torch.Tensor:
    n = int(L.load().psd_nested_workspace_bytes(C.byref(plan.c), int(Hq), int(Dv)))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def cascade_decode_nested(ctx: Context, args: L.DecodeArgs, plan: NestedPlan, o: torch.Tensor,
                          lse: torch.Tensor = None, workspace: torch.Tensor = None, stream=None) -> dict:
    """cascade_decode_nested: one stacked level-0 launch per segment, level 1, one merge."""
    stats = L.CascadeStats()
    L.check(L.load().cascade_decode_nested(
        ctx.handle, C.byref(args), C.byref(plan.c), _dev_ptr(o, "o"),
        None if lse is None else _dev_ptr(lse, "lse"), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), C.byref(stats), _stream(stream)))
    return {k: getattr(stats, k) for k, _ in L.CascadeStats._fields_}


def workspace_for(plan: Plan, Hq: int, Dv: int, device) -> torch.Tensor:
    n = workspace_bytes(plan.batch, max(plan.num_items, 1), plan.num_rows, Hq, Dv)
    return torch.empty(n, dtype=torch.uint8, device=device)
