"""Batched, rank-specialized LoRA-delta apply on AMD Instinct MI355X.

Thin PyTorch binding over the C ABI (include/lora.h).  Torch provides device
memory and the current stream; every step of the apply runs in the HIP
kernels of librank_specialized.so.  The entry points keep the C names:

    store = lora_pack_retained(A_list, B_list, scales)        # pack
    seg   = lora_segment(ids, store.n)                        # group tokens
    h     = lora_shrink(store, x, seg)                        # h = A_a x (grouped rows)
    lora_expand(store, h, seg, y)                             # y += s_a B_a h
    lora_apply_batched(store, x, y, ids=ids)                  # all of the above

The 4-bit base layers and the router of a mixture of experts:

    base  = lora_w4_pack(q, scales, zeros, group=128)         # codes of one matrix, or of every expert
    y     = lora_w4_apply(base, x)                            # y = W x; then lora_apply_batched(store, x, y, ...)
    ids, w = lora_route(logits, k)                            # a token's experts and their weights
    y     = lora_w4_apply_experts(experts, x, ids, w)         # y[t] = sum_j w[t, j] W_{ids[t, j]} x

Workspaces (lora_workspace_bytes) are allocated here with torch when the
caller passes none.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

from . import _lib as L
from ._lib import LoraError, lora_store  # noqa: F401

__all__ = [
    "Store", "Segmentation", "LoraError", "lora_store_bytes", "lora_pack_retained",
    "lora_segment", "lora_plan_bytes", "lora_group", "lora_apply_planned", "lora_workspace_bytes", "lora_shrink", "lora_expand", "lora_apply_batched",
    "lora_apply_batched_phases", "lora_apply_batched_noalloc", "lora_apply_launches", "lora_apply_base_fused", "JDStore", "lora_jd_pack", "lora_jd_workspace_bytes",
    "lora_jd_apply", "lora_ranks_uniform", "lora_ranks_spectral", "RsvdFactors", "lora_rsvd_workspace_bytes",
    "lora_rsvd_factor", "lora_rsvd_write", "MultiStore", "lora_pack_multi", "lora_multi_workspace_bytes",
    "lora_apply_multi", "W4Store", "lora_w4_bytes", "lora_w4_pack", "lora_w4_workspace_bytes", "lora_w4_apply",
    "lora_w4_apply_experts", "lora_route", "load_library",
]

_DTYPES = {torch.bfloat16: L.LORA_DTYPE_BF16, torch.float32: L.LORA_DTYPE_F32}


def load_library():
    """Load librank_specialized.so (raises ImportError if it was not built)."""
    return L.lib()


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _p(t: Optional[torch.Tensor]):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _rows(t: torch.Tensor, name: str):
    if t.dim() != 2 or (t.shape[0] > 0 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return t.stride(0) if t.shape[0] > 0 else t.shape[1]


@dataclass
class Store:
    """A packed retained-rank store: the C struct plus the buffers it references."""

    c: lora_store
    A_pack: torch.Tensor
    B_pack: torch.Tensor
    meta: torch.Tensor
    ranks: List[int]
    dtype: torch.dtype

    @property
    def n(self) -> int:
        return self.c.n

    @property
    def d_in(self) -> int:
        return self.c.d_in

    @property
    def d_out(self) -> int:
        return self.c.d_out

    @property
    def r_max(self) -> int:
        return self.c.r_max

    @property
    def pad_to(self) -> int:
        return self.c.pad_to

    def ref(self):
        return C.byref(self.c)

    def clone(self) -> "Store":
        """An independent copy in fresh device memory (same layout)."""
        A, B, meta = self.A_pack.clone(), self.B_pack.clone(), self.meta.clone()
        c = lora_store.from_buffer_copy(self.c)
        n = self.c.n
        c.A_pack, c.B_pack = A.data_ptr(), B.data_ptr()
        c.row_off = meta.data_ptr()
        c.rank = meta.data_ptr() + (n + 1) * 4
        c.scale = meta.data_ptr() + (2 * n + 1) * 4
        return Store(c, A, B, meta, list(self.ranks), self.dtype)

    def device_meta(self):
        """(row_off, rank, scale) as device tensors (views of the meta buffer)."""
        n = self.n
        i32 = self.meta[: (3 * n + 1) * 4].view(torch.int32)
        return i32[: n + 1], i32[n + 1: 2 * n + 1], i32[2 * n + 1: 3 * n + 1].view(torch.float32)


def lora_store_bytes(n: int, d_in: int, d_out: int, dtype: torch.dtype, ranks: Sequence[int],
                     pad_to: int = 0):
    r = (C.c_int32 * max(n, 1))(*[int(v) for v in ranks])
    a, b, m = C.c_size_t(), C.c_size_t(), C.c_size_t()
    L.check("lora_store_bytes", L.lib().lora_store_bytes(n, d_in, d_out, _DTYPES[dtype], r, pad_to,
                                                         C.byref(a), C.byref(b), C.byref(m)))
    return a.value, b.value, m.value


def lora_pack_retained(A_list: Sequence[torch.Tensor], B_list: Sequence[torch.Tensor], scales,
                       pad_to: int = 0) -> Store:
    """Pack per-adapter factors (A_a [r_a, d_in], B_a [d_out, r_a], device tensors,
    row-major contiguous, one dtype) into a store.  pad_to > 0 builds the
    rank-padded comparison store."""
    n = len(A_list)
    if n == 0 or len(B_list) != n:
        raise ValueError("need one A and one B per adapter")
    dtype = A_list[0].dtype
    device = A_list[0].device
    d_in = A_list[0].shape[1]
    d_out = B_list[0].shape[0]
    ranks = [int(a.shape[0]) for a in A_list]
    for a, b, r in zip(A_list, B_list, ranks):
        if a.dtype != dtype or b.dtype != dtype or a.shape != (r, d_in) or b.shape != (d_out, r):
            raise ValueError("factor shapes/dtypes are inconsistent")
        if not (a.is_contiguous() and b.is_contiguous()):
            raise ValueError("factors must be contiguous")
    return _pack(n, d_in, d_out, dtype, ranks, scales, pad_to, device,
                 (C.c_void_p * n)(*[_p(a) for a in A_list]), (C.c_void_p * n)(*[_p(b) for b in B_list]))


def _pack(n, d_in, d_out, dtype, ranks, scales, pad_to, device, a_ptrs, b_ptrs) -> Store:
    """Allocate a store's buffers and call lora_pack_retained (a_ptrs and
    b_ptrs None: metadata only)."""
    a_bytes, b_bytes, m_bytes = lora_store_bytes(n, d_in, d_out, dtype, ranks, pad_to)
    A_pack = torch.empty(max(a_bytes, 16), dtype=torch.uint8, device=device)
    B_pack = torch.empty(max(b_bytes, 16), dtype=torch.uint8, device=device)
    meta = torch.empty(m_bytes, dtype=torch.uint8, device=device)
    r_arr = (C.c_int32 * n)(*ranks)
    s_arr = (C.c_float * n)(*[float(v) for v in scales])
    st = lora_store()
    L.check("lora_pack_retained", L.lib().lora_pack_retained(
        C.byref(st), n, d_in, d_out, _DTYPES[dtype], r_arr, s_arr, a_ptrs, b_ptrs,
        A_pack.data_ptr(), B_pack.data_ptr(), meta.data_ptr(), pad_to, _stream(meta)))
    return Store(st, A_pack, B_pack, meta, list(ranks), dtype)


@dataclass
class Segmentation:
    """Grouped order of T tokens over n adapters (as lora_segment writes it)."""

    T: int
    n: int
    seg_off: torch.Tensor  # int32 [n + 2]
    perm: torch.Tensor  # int32 [T]
    n_invalid: Optional[torch.Tensor] = None
    plan: Optional[torch.Tensor] = None  # uint8 [lora_plan_bytes(T, n)] (lora_group)


def lora_segment(ids: torch.Tensor, n: int, *, seg: Optional[Segmentation] = None) -> Segmentation:
    """Stable grouping of tokens by adapter id (ids: int32 device tensor [T])."""
    if ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 vector")
    T = ids.shape[0]
    dev = ids.device
    if seg is None:
        seg = Segmentation(T, n, torch.empty(n + 2, dtype=torch.int32, device=dev),
                           torch.empty(max(T, 1), dtype=torch.int32, device=dev)[:T],
                           torch.empty(1, dtype=torch.int32, device=dev))
    L.check("lora_segment", L.lib().lora_segment(
        _p(ids), T, n, seg.seg_off.data_ptr(), _p(seg.perm), seg.n_invalid.data_ptr(), _stream(seg.seg_off)))
    return seg


def lora_plan_bytes(T: int, n: int) -> int:
    return int(L.lib().lora_plan_bytes(T, n))


def lora_group(ids: torch.Tensor, n: int, *, seg: Optional[Segmentation] = None) -> Segmentation:
    """lora_segment plus the plan of the grouping (its sub-tiles), which
    lora_apply_planned reuses across stores."""
    if ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 vector")
    T = ids.shape[0]
    dev = ids.device
    nb = lora_plan_bytes(T, n)
    if seg is None or seg.plan is None:
        seg = Segmentation(T, n, torch.empty(n + 2, dtype=torch.int32, device=dev),
                           torch.empty(max(T, 1), dtype=torch.int32, device=dev)[:T],
                           torch.empty(1, dtype=torch.int32, device=dev),
                           torch.empty(max(nb, 16), dtype=torch.uint8, device=dev))
    L.check("lora_group", L.lib().lora_group(
        _p(ids), T, n, seg.seg_off.data_ptr(), _p(seg.perm), seg.plan.data_ptr(), seg.plan.numel(),
        seg.n_invalid.data_ptr(), _stream(seg.seg_off)))
    return seg


def lora_workspace_bytes(store: Store, T: int) -> int:
    return int(L.lib().lora_workspace_bytes(store.ref(), T))


def _ws(store: Store, T: int, ws: Optional[torch.Tensor], device) -> torch.Tensor:
    if ws is None:
        ws = torch.empty(max(lora_workspace_bytes(store, T), 16), dtype=torch.uint8, device=device)
    return ws


def lora_shrink(store: Store, x: torch.Tensor, seg: Segmentation, h: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h[i, :r_a] = A_a x[perm[i]] in float32 (grouped rows).  Columns >= r_a
    and rows of tokens without an adapter are left as they were in ``h``."""
    T = x.shape[0]
    if h is None:
        h = torch.zeros(T, max(store.r_max, 1), dtype=torch.float32, device=x.device)
    ws = _ws(store, T, ws, x.device)
    L.check("lora_shrink", L.lib().lora_shrink(
        store.ref(), _p(x), _rows(x, "x"), T, seg.seg_off.data_ptr(), _p(seg.perm), _p(h), _rows(h, "h"),
        ws.data_ptr(), ws.numel(), _stream(x)))
    return h


def lora_expand(store: Store, h: torch.Tensor, seg: Segmentation, y: torch.Tensor,
                ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[perm[i]] += s_a B_a h[i] in place."""
    T = y.shape[0]
    ws = _ws(store, T, ws, y.device)
    L.check("lora_expand", L.lib().lora_expand(
        store.ref(), _p(h), _rows(h, "h"), T, seg.seg_off.data_ptr(), _p(seg.perm), _p(y), _rows(y, "y"),
        ws.data_ptr(), ws.numel(), _stream(y)))
    return y


def lora_apply_batched(store: Store, x: torch.Tensor, y: torch.Tensor, *,
                       ids: Optional[torch.Tensor] = None, seg: Optional[Segmentation] = None,
                       ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] += s_a B_a (A_a x[t]) in place, for ids (grouped here) or a prior grouping."""
    T = x.shape[0]
    if (ids is None) == (seg is None):
        raise ValueError("pass exactly one of ids or seg")
    ws = _ws(store, T, ws, x.device)
    if seg is not None:
        so, pm = seg.seg_off.data_ptr(), _p(seg.perm)
    else:
        if ids.dtype != torch.int32 or not ids.is_contiguous():
            raise ValueError("ids must be a contiguous int32 vector")
        so = pm = None
    L.check("lora_apply_batched", L.lib().lora_apply_batched(
        store.ref(), _p(x), _rows(x, "x"), _p(y), _rows(y, "y"), T, _p(ids) if ids is not None else None,
        so, pm, ws.data_ptr(), ws.numel(), _stream(x)))
    return y


def lora_apply_batched_phases(store: Store, x: torch.Tensor, y: torch.Tensor, phases: int, *,
                              ids: Optional[torch.Tensor] = None, seg: Optional[Segmentation] = None,
                              ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One kernel of lora_apply_batched at a time (phases 1 = shrink, 2 =
    expand from the plan a phase-1 call left in ``ws``, 3 = the apply, a
    single fused kernel for decode-sized calls)."""
    T = x.shape[0]
    if (ids is None) == (seg is None):
        raise ValueError("pass exactly one of ids or seg")
    ws = _ws(store, T, ws, x.device)
    so = seg.seg_off.data_ptr() if seg is not None else None
    pm = _p(seg.perm) if seg is not None else None
    if ids is not None and (ids.dtype != torch.int32 or not ids.is_contiguous()):
        raise ValueError("ids must be a contiguous int32 vector")
    L.check("lora_apply_batched_phases", L.lib().lora_apply_batched_phases(
        store.ref(), _p(x), _rows(x, "x"), _p(y), _rows(y, "y"), T, _p(ids) if ids is not None else None,
        so, pm, ws.data_ptr(), ws.numel(), _stream(x), phases))
    return y


def lora_apply_batched_noalloc(store: Store, x: torch.Tensor, y: torch.Tensor, *,
                               ids: Optional[torch.Tensor] = None,
                               seg: Optional[Segmentation] = None) -> torch.Tensor:
    """lora_apply_batched without a workspace: the library's own per-device
    scratch array serves as one (nothing is allocated, here or in the
    library).  Calls that overlap on one device race on that array."""
    T = x.shape[0]
    if (ids is None) == (seg is None):
        raise ValueError("pass exactly one of ids or seg")
    if seg is not None:
        so, pm = seg.seg_off.data_ptr(), _p(seg.perm)
    else:
        if ids.dtype != torch.int32 or not ids.is_contiguous():
            raise ValueError("ids must be a contiguous int32 vector")
        so = pm = None
    L.check("lora_apply_batched_noalloc", L.lib().lora_apply_batched_noalloc(
        store.ref(), _p(x), _rows(x, "x"), _p(y), _rows(y, "y"), T, _p(ids) if ids is not None else None,
        so, pm, _stream(x)))
    return y


def lora_apply_base_fused(store: Store, W0: torch.Tensor, x: torch.Tensor, y: torch.Tensor, *,
                          ids: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x W0^T + s_a B_a (A_a x) per token (overwrites y): the base layer
    W0 [d_out, d_in] with the adapter branch added in its epilogue, y written
    once.  Without ids: the base product alone.  bf16 stores only."""
    T = x.shape[0]
    if W0.dim() != 2 or W0.shape[0] != store.d_out or W0.shape[1] < store.d_in:
        raise ValueError("W0 must be [d_out, >= d_in]")
    if ids is not None:
        if ids.dtype != torch.int32 or not ids.is_contiguous():
            raise ValueError("ids must be a contiguous int32 vector")
        ws = _ws(store, T, ws, x.device)
    L.check("lora_apply_base_fused", L.lib().lora_apply_base_fused(
        store.ref(), _p(W0), _rows(W0, "W0"), _p(x), _rows(x, "x"), _p(y), _rows(y, "y"), T,
        _p(ids) if ids is not None else None, ws.data_ptr() if ws is not None else None,
        ws.numel() if ws is not None else 0, _stream(x)))
    return y


def lora_apply_planned(store: Store, x: torch.Tensor, y: torch.Tensor, seg: Segmentation, *,
                       ws: Optional[torch.Tensor] = None, phases: int = 3) -> torch.Tensor:
    """y[t] += s_a B_a (A_a x[t]) in place on the plan of ``seg`` (from
    lora_group): the shrink and the expand only (phases 1 / 2: one of them)."""
    T = x.shape[0]
    if seg.plan is None:
        raise ValueError("seg has no plan (use lora_group)")
    ws = _ws(store, T, ws, x.device)
    L.check("lora_apply_planned_phases", L.lib().lora_apply_planned_phases(
        store.ref(), _p(x), _rows(x, "x"), _p(y), _rows(y, "y"), T, seg.plan.data_ptr(), seg.plan.numel(),
        ws.data_ptr(), ws.numel(), _stream(x), phases))
    return y


def lora_apply_launches(store: Store, T: int, with_ids=True) -> int:
    """Kernel launches an apply makes for this store and T: with_ids True / 1
    (ids), False / 0 (a caller's seg_off, perm), 2 (a plan).  1 = the fused
    decode kernel, 2 = shrink + expand, 3 = grouping + shrink + expand,
    4 = sort + plan + shrink + expand."""
    v = L.lib().lora_apply_launches(store.ref(), int(T), int(with_ids))
    if v < 0:
        L.check("lora_apply_launches", -v)
    return v


@dataclass
class JDStore:
    """A shared-basis store: the basis store over clusters (A = V_j^T, B = U_j,
    rank r, scale 1) plus per-adapter cluster, Sigma and scale buffers."""

    c: L.lora_jd_store
    basis: Store
    cluster_of: torch.Tensor
    sigma: torch.Tensor
    scale: torch.Tensor

    @property
    def n(self) -> int:
        return self.c.n_adapters

    @property
    def k(self) -> int:
        return self.basis.n

    @property
    def r(self) -> int:
        return self.c.r

    def ref(self):
        return C.byref(self.c)

    def clone(self) -> "JDStore":
        return _jd_store(self.basis.clone(), self.cluster_of.clone(), self.sigma.clone(), self.scale.clone(),
                         self.c.diag)


def _jd_store(basis: Store, cluster_of, sigma, scale, diag: int) -> JDStore:
    c = L.lora_jd_store()
    c.basis = basis.c
    c.n_adapters = int(cluster_of.numel())
    c.r = basis.r_max
    c.diag = int(diag)
    c.cluster_of, c.sigma, c.scale = cluster_of.data_ptr(), sigma.data_ptr(), scale.data_ptr()
    return JDStore(c, basis, cluster_of, sigma, scale)


def lora_jd_pack(U_list: Sequence[torch.Tensor], V_list: Sequence[torch.Tensor], cluster_of, sigma, scales) -> JDStore:
    """Shared-basis store from per-cluster U_j [d_out, r] and V_j [d_in, r]
    (device tensors of one dtype), cluster_of [n], Sigma [n, r, r] (full) or
    [n, r] (diagonal) and scales [n]."""
    k = len(U_list)
    if k == 0 or len(V_list) != k:
        raise ValueError("need one U and one V per cluster")
    device = U_list[0].device
    basis = lora_pack_retained([V.t().contiguous() for V in V_list], [U.contiguous() for U in U_list], [1.0] * k)
    r = basis.r_max
    sig = torch.as_tensor(sigma, dtype=torch.float32).to(device).contiguous()
    n = sig.shape[0]
    if sig.shape not in ((n, r, r), (n, r)):
        raise ValueError("sigma must be [n, r, r] or [n, r]")
    cl = torch.as_tensor(cluster_of, dtype=torch.int32).to(device).contiguous()
    sc = torch.as_tensor(scales, dtype=torch.float32).to(device).contiguous()
    if cl.shape != (n,) or sc.shape != (n,):
        raise ValueError("cluster_of and scales need one entry per adapter")
    return _jd_store(basis, cl, sig, sc, 1 if sig.dim() == 2 else 0)


def lora_jd_workspace_bytes(store: JDStore, T: int) -> int:
    return int(L.lib().lora_jd_workspace_bytes(store.ref(), int(T)))


def lora_jd_apply(store: JDStore, x: torch.Tensor, y: torch.Tensor, ids: torch.Tensor,
                  ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] += s_a U_c Sigma_a V_c^T x[t] in place (a = ids[t], c = its cluster)."""
    T = x.shape[0]
    if ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 vector")
    if ws is None:
        ws = torch.empty(max(lora_jd_workspace_bytes(store, T), 16), dtype=torch.uint8, device=x.device)
    L.check("lora_jd_apply", L.lib().lora_jd_apply(store.ref(), _p(x), _rows(x, "x"), _p(y), _rows(y, "y"), T,
                                                   _p(ids), ws.data_ptr(), ws.numel(), _stream(x)))
    return y


def lora_ranks_uniform(r_orig: Sequence[int], ratio: float, floor: int) -> List[int]:
    """Retained ranks by a uniform ratio of the original rank, with a floor."""
    m = len(r_orig)
    ro = (C.c_int32 * max(m, 1))(*[int(v) for v in r_orig])
    out = (C.c_int32 * max(m, 1))()
    L.check("lora_ranks_uniform", L.lib().lora_ranks_uniform(m, ro, float(ratio), int(floor), out))
    return list(out)[:m]


def lora_ranks_spectral(r_orig: Sequence[int], sigmas, floor: int, budget: int) -> List[int]:
    """Retained ranks by a spectral budget: floors first, then the largest
    remaining singular values over all units, `budget` ranks in total."""
    import numpy as np
    m = len(r_orig)
    ro = np.ascontiguousarray(np.asarray(r_orig, np.int32))
    flat = np.ascontiguousarray(np.concatenate([np.asarray(s, np.float32) for s in sigmas]) if m else
                                np.zeros(1, np.float32))
    off = np.zeros(m + 1, np.int64)
    off[1:] = np.cumsum(ro)
    out = np.zeros(max(m, 1), np.int32)
    L.check("lora_ranks_spectral", L.lib().lora_ranks_spectral(
        m, ro.ctypes.data, flat.ctypes.data, off.ctypes.data, int(floor), int(budget), out.ctypes.data))
    return [int(v) for v in out[:m]]


@dataclass
class RsvdFactors:
    """What lora_rsvd_factor leaves for lora_rsvd_write: the original factors
    (kept referenced), the singular values, the status flags and the
    workspace holding W_B, W_A."""

    A_all: torch.Tensor  # [n, r, d_in]
    B_all: torch.Tensor  # [n, d_out, r]
    sigma: torch.Tensor  # float32 [n, r], descending
    status: torch.Tensor  # int32 [n]
    ws: torch.Tensor

    @property
    def n(self) -> int:
        return self.A_all.shape[0]

    @property
    def r(self) -> int:
        return self.A_all.shape[1]


def lora_rsvd_workspace_bytes(n: int, d_in: int, d_out: int) -> int:
    return int(L.lib().lora_rsvd_workspace_bytes(n, d_in, d_out))


def lora_rsvd_factor(A_all: torch.Tensor, B_all: torch.Tensor, ws: Optional[torch.Tensor] = None,
                     phases: int = 15, out: Optional[RsvdFactors] = None) -> RsvdFactors:
    """Stage 1 of retained-factor construction for n adapters of one rank r:
    A_all [n, r, d_in], B_all [n, d_out, r] (contiguous, bf16 or float32).
    phases: a bit mask of its kernels (lora_rsvd_factor_phases; 15 = all);
    ``out`` reuses the sigma, status and workspace buffers of a previous call."""
    if A_all.dim() != 3 or B_all.dim() != 3:
        raise ValueError("A_all is [n, r, d_in] and B_all [n, d_out, r]")
    n, r, d_in = A_all.shape
    d_out = B_all.shape[1]
    if B_all.shape != (n, d_out, r) or A_all.dtype != B_all.dtype:
        raise ValueError("A_all and B_all are inconsistent")
    if not (A_all.is_contiguous() and B_all.is_contiguous()):
        raise ValueError("factors must be contiguous")
    if out is not None:
        sigma, status, ws = out.sigma, out.status, out.ws
    else:
        sigma = torch.empty(n, r, dtype=torch.float32, device=A_all.device)
        status = torch.empty(n, dtype=torch.int32, device=A_all.device)
    if ws is None:
        ws = torch.empty(max(lora_rsvd_workspace_bytes(n, d_in, d_out), 16), dtype=torch.uint8, device=A_all.device)
    L.check("lora_rsvd_factor", L.lib().lora_rsvd_factor_phases(
        n, d_in, d_out, _DTYPES[A_all.dtype], r, _p(A_all), _p(B_all), _p(sigma), _p(status), ws.data_ptr(),
        ws.numel(), _stream(A_all), int(phases)))
    return RsvdFactors(A_all, B_all, sigma, status, ws)


def lora_rsvd_write(f: RsvdFactors, ranks: Sequence[int], scales, pad_to: int = 0,
                    store: Optional[Store] = None) -> Store:
    """Stage 2: a store of the retained factors at `ranks` (one per adapter,
    e.g. from lora_ranks_uniform / lora_ranks_spectral over f.sigma).  With
    ``store`` (built by an earlier call for the same adapters), its buffers are
    rewritten in place and ranks / scales / pad_to are taken from it."""
    n, r, d_in = f.A_all.shape
    d_out = f.B_all.shape[1]
    if store is None:
        ranks = [int(v) for v in ranks]
        if len(ranks) != n:
            raise ValueError("one retained rank per adapter")
        store = _pack(n, d_in, d_out, f.A_all.dtype, ranks, scales, pad_to, f.A_all.device, None, None)
    L.check("lora_rsvd_write", L.lib().lora_rsvd_write(store.ref(), r, _p(f.A_all), _p(f.B_all), f.ws.data_ptr(),
                                                       f.ws.numel(), _stream(f.A_all)))
    return store


@dataclass
class MultiStore:
    """Slices of one input (q/k/v, gate/up) for the multi-slice apply: the
    slices' stores (kept referenced), the stacked A buffer, its metadata and
    hoff."""

    c: L.lora_multi_store
    slices: List[Store]
    A: torch.Tensor
    meta: torch.Tensor
    hoff: torch.Tensor

    @property
    def n(self) -> int:
        return self.c.stacked.n

    @property
    def n_slices(self) -> int:
        return self.c.n_slices

    def ref(self):
        return C.byref(self.c)


def lora_pack_multi(slices: Sequence[Store]) -> MultiStore:
    """Stack the A rows of stores of the same adapters (same n, d_in, dtype)."""
    k = len(slices)
    arr = (L.lora_store * max(k, 1))(*[st.c for st in slices])
    a, m, h = C.c_size_t(), C.c_size_t(), C.c_size_t()
    L.check("lora_multi_bytes", L.lib().lora_multi_bytes(k, arr, C.byref(a), C.byref(m), C.byref(h)))
    dev = slices[0].meta.device
    A = torch.empty(max(a.value, 16), dtype=torch.uint8, device=dev)
    meta = torch.empty(m.value, dtype=torch.uint8, device=dev)
    hoff = torch.empty(max(h.value // 4, 4), dtype=torch.int32, device=dev)
    c = L.lora_multi_store()
    L.check("lora_pack_multi", L.lib().lora_pack_multi(C.byref(c), k, arr, A.data_ptr(), meta.data_ptr(),
                                                       hoff.data_ptr(), _stream(meta)))
    return MultiStore(c, list(slices), A, meta, hoff)


def lora_multi_workspace_bytes(store: MultiStore, T: int) -> int:
    return int(L.lib().lora_multi_workspace_bytes(store.ref(), T))


def lora_apply_multi(store: MultiStore, x: torch.Tensor, ys: Sequence[torch.Tensor], ids=None,
                     seg: Optional[Segmentation] = None, ws: Optional[torch.Tensor] = None):
    """y_s += s B_s A_s x for every slice, x read once; ys may be column
    slices of one fused buffer (row stride taken from each view).  A ``seg``
    from lora_group carries a plan, which is then used as it is."""
    T = x.shape[0]
    k = store.n_slices
    if len(ys) != k:
        raise ValueError("one y per slice")
    if (ids is None) == (seg is None):
        raise ValueError("pass exactly one of ids or seg")
    yp = (C.c_void_p * k)(*[_p(y) for y in ys])
    ld = (C.c_int64 * k)(*[_rows(y, "y") for y in ys])
    if ids is not None and (ids.dtype != torch.int32 or not ids.is_contiguous()):
        raise ValueError("ids must be a contiguous int32 vector")
    if ws is None:
        ws = torch.empty(max(lora_multi_workspace_bytes(store, T), 16), dtype=torch.uint8, device=x.device)
    if seg is not None and seg.plan is not None:
        L.check("lora_apply_multi_planned", L.lib().lora_apply_multi_planned(
            store.ref(), _p(x), _rows(x, "x"), yp, ld, T, seg.plan.data_ptr(), seg.plan.numel(), ws.data_ptr(),
            ws.numel(), _stream(x)))
        return ys
    so = seg.seg_off if seg is not None else None
    pm = seg.perm if seg is not None else None
    L.check("lora_apply_multi", L.lib().lora_apply_multi(
        store.ref(), _p(x), _rows(x, "x"), yp, ld, T, _p(ids), _p(so), _p(pm), ws.data_ptr(), ws.numel(),
        _stream(x)))
    return ys


@dataclass
class W4Store:
    """4-bit matrices laid out by lora_w4_pack: the C struct plus its buffers."""

    c: L.lora_w4_store
    codes: torch.Tensor
    params: torch.Tensor

    def __post_init__(self):
        # Plain attributes: a decode step's call is short enough for the
        # struct's accessors to show.
        c = self.c
        self.n, self.d_in, self.d_out, self.group = c.n, c.d_in, c.d_out, c.group
        self.device_index = self.codes.get_device()
        if self.device_index < 0 or self.params.get_device() != self.device_index:
            raise ValueError("codes and params must be on one GPU")
        self._ref = C.byref(c)
        self._ws_bytes = {}

    def ref(self):
        return self._ref

    def clone(self) -> "W4Store":
        """An independent copy in fresh device memory (same layout)."""
        codes, params = self.codes.clone(), self.params.clone()
        c = L.lora_w4_store.from_buffer_copy(self.c)
        c.codes, c.params = codes.data_ptr(), params.data_ptr()
        return W4Store(c, codes, params)


# The handle of a device's current stream, without a Stream object around it
# where torch offers that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name: str, index: int, *args) -> None:
    """The library's `name` on the current stream of device `index`, which is
    made the current device for the call."""
    fn = getattr(L.lib(), name)
    if torch.cuda.current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        L.check(name, status)


def _same_device(index: int, **tensors) -> None:
    """Every tensor given is on GPU `index`."""
    if index < 0:
        raise ValueError("tensors must be on a GPU")
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")


_INT_MAX = 2**31 - 1  # what the C interface's sizes hold; ctypes would cut more off silently


def _int(v, name: str) -> int:
    v = int(v)
    if not -_INT_MAX <= v <= _INT_MAX:
        raise ValueError(f"{name} is out of range")
    return v


def _ld(t: torch.Tensor, name: str) -> int:
    """Row stride of a 2-D tensor with unit column stride; of at most one row,
    its length (its stride is then any number)."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    rows, cols = t.shape
    if rows > _INT_MAX or cols > _INT_MAX:
        raise ValueError(f"{name} has more rows or columns than an int counts")
    ld, step = t.stride()
    if rows > 0 and cols > 1 and step != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return ld if rows > 1 else cols


def _scratch(ws: torch.Tensor) -> int:
    """Bytes of a workspace tensor: all of them one run of memory, so that
    its size says how far a kernel may write (that of an expanded tensor or of
    a strided view does not)."""
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.numel() * ws.element_size()


def _dtype(t: torch.Tensor, name: str) -> int:
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be bfloat16 or float32")
    return dt


def lora_w4_bytes(n: int, d_in: int, d_out: int, group: int, scale_dtype: torch.dtype, has_zeros: bool):
    """Bytes of a w4 store's codes and params buffers."""
    a, b = C.c_size_t(), C.c_size_t()
    n, d_in, d_out, group = _int(n, "n"), _int(d_in, "d_in"), _int(d_out, "d_out"), _int(group, "group")
    L.check("lora_w4_bytes", L.lib().lora_w4_bytes(n, d_in, d_out, group, _DTYPES[scale_dtype], int(has_zeros),
                                                   C.byref(a), C.byref(b)))
    return a.value, b.value


def lora_w4_pack(q: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None, *,
                 group: int) -> W4Store:
    """Lay 4-bit matrices out: W[o, k] = scales[o, k // group] * (q[o, k] - zeros[o, k // group]).

    q: uint8 [n, d_out, d_in / 2] (or [d_out, d_in / 2] for one matrix), input
    2 i in the low four bits of byte i; scales (bfloat16 or float32) and zeros
    (uint8 0..15; None: 8) [n, d_out, ceil(d_in / group)]."""
    if q.dim() == 2:
        q, scales = q.unsqueeze(0), scales.unsqueeze(0)
        zeros = zeros.unsqueeze(0) if zeros is not None else None
    if q.dim() != 3 or q.dtype != torch.uint8:
        raise ValueError("q must be uint8 [n, d_out, d_in / 2]")
    n, d_out, half = q.shape
    d_in = 2 * half
    group = _int(group, "group")
    if group < 1:
        raise ValueError("group must be positive")
    shape = (n, d_out, -(-d_in // group))
    if scales.shape != shape:
        raise ValueError(f"scales must be {shape}")
    if zeros is not None and (zeros.shape != shape or zeros.dtype != torch.uint8):
        raise ValueError(f"zeros must be uint8 {shape}")
    sd = _dtype(scales, "scales")
    index = q.get_device()
    _same_device(index, scales=scales, zeros=zeros)
    q, scales = q.contiguous(), scales.contiguous()
    zeros = zeros.contiguous() if zeros is not None else None
    cb, pb = lora_w4_bytes(n, d_in, d_out, group, scales.dtype, zeros is not None)
    codes = torch.empty(cb, dtype=torch.uint8, device=q.device)
    params = torch.empty(pb, dtype=torch.uint8, device=q.device)
    c = L.lora_w4_store()
    _call("lora_w4_pack", index, C.byref(c), n, d_in, d_out, group, _p(q), _p(scales), sd, _p(zeros),
          codes.data_ptr(), params.data_ptr())
    return W4Store(c, codes, params)


def lora_w4_workspace_bytes(store: W4Store, dtype: torch.dtype, T: int, k: int = 0, weighted: bool = False) -> int:
    """Workspace of lora_w4_apply (k = 0) or lora_w4_apply_experts for T tokens."""
    return int(L.lib().lora_w4_workspace_bytes(store.ref(), _DTYPES[dtype], _int(T, "T"), _int(k, "k"), int(weighted)))


def _w4_run(name: str, store: W4Store, x: torch.Tensor, rows: int, y, T: int, k: int, ids, weights, ws, middle):
    """The part the two products share: y and the workspace, the checks, the call."""
    dt, ldx, index = _dtype(x, "x"), _ld(x, "x"), store.device_index
    if x.shape[1] != store.d_in:
        raise ValueError("x must have d_in columns")
    if x.get_device() != index:
        _same_device(index, x=x)
    if y is None:
        ldy = store.d_out
        y = torch.empty(rows, ldy, dtype=x.dtype, device=x.device)
    else:
        if y.shape != (rows, store.d_out) or y.dtype != x.dtype:
            raise ValueError(f"y must be [{rows}, {store.d_out}] of x's dtype")
        _same_device(index, y=y)
        ldy = _ld(y, "y")
    if ws is None:
        key = (dt, T, k, weights is not None)
        nb = store._ws_bytes.get(key)
        if nb is None:
            if len(store._ws_bytes) >= 1024:
                store._ws_bytes.clear()
            nb = store._ws_bytes[key] = lora_w4_workspace_bytes(store, x.dtype, T, k, weights is not None)
        if nb:
            ws = torch.empty(nb, dtype=torch.uint8, device=x.device)
        ws_ptr = ws.data_ptr() if nb else None
    else:
        _same_device(index, ws=ws)
        nb, ws_ptr = _scratch(ws), _p(ws)
    _call(name, index, store._ref, dt, _p(x), ldx, *middle[0], _p(y), ldy, T, *middle[1], ws_ptr, nb)
    return y


def lora_w4_apply(store: W4Store, x: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                  ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] = W x[t] (overwrites y; allocated when None): the 4-bit base layer
    of a store of one matrix, x [T, d_in] bfloat16 or float32."""
    T = x.shape[0]
    return _w4_run("lora_w4_apply", store, x, T, y, T, 0, None, None, ws, ((), ()))


def lora_w4_apply_experts(store: W4Store, x: torch.Tensor, ids: torch.Tensor, weights: Optional[torch.Tensor] = None,
                          y: Optional[torch.Tensor] = None, *, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The products with the experts that ids [T, k] (int32) name; an id
    outside [0, n) names none.

    x: [T, d_in] (every choice of a token reads its row) or [T k, d_in].
    Without weights y is [T k, d_out], a row per choice (zero without an
    expert); with weights (float32 [T, k]) y is [T, d_out], the weighted sum
    over a token's choices."""
    if ids.dim() != 2 or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 [T, k]")
    T, k = ids.shape
    if k > _INT_MAX:
        raise ValueError("ids has more columns than an int counts")
    x_rows = x.shape[0]
    if x_rows != T and x_rows != T * k:
        raise ValueError("x must be [T, d_in] or [T k, d_in]")
    if ids.get_device() != store.device_index:
        _same_device(store.device_index, ids=ids)
    if weights is not None:
        if weights.shape != ids.shape or weights.dtype != torch.float32 or not weights.is_contiguous():
            raise ValueError("weights must be a contiguous float32 [T, k]")
        _same_device(store.device_index, weights=weights)
    return _w4_run("lora_w4_apply_experts", store, x, T * k if weights is None else T, y, T, k, ids, weights, ws,
                   ((int(x_rows != T),), (k, _p(ids), _p(weights))))


_SCORES = {"softmax": L.LORA_ROUTE_SOFTMAX, "sigmoid": L.LORA_ROUTE_SIGMOID}


def lora_route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: Optional[torch.Tensor] = None,
               groups: int = 1, top_groups: int = 1, renormalize: bool = True, scale: float = 1.0,
               ids: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None):
    """The router: (ids int32 [T, k], weights float32 [T, k]) of each token's k
    experts, by descending score (softmax or sigmoid of logits [T, E], plus
    bias [E] for the choice alone), among the best top_groups of `groups`
    runs of experts.  Where fewer than k can be chosen: id -1, weight 0."""
    dt, ldl = _dtype(logits, "logits"), _ld(logits, "logits")
    T, E = logits.shape
    mode = _SCORES.get(score)
    if mode is None:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    k, index = _int(k, "k"), logits.get_device()
    if k < 1:
        raise ValueError("k must be positive")
    if bias is not None:
        if bias.shape != (E,) or bias.dtype != torch.float32 or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous float32 [E]")
        _same_device(index, bias=bias)
    if index < 0:
        _same_device(index)
    if ids is None:
        ids = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    elif ids.shape != (T, k) or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 [T, k]")
    else:
        _same_device(index, ids=ids)
    if weights is None:
        weights = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    elif weights.shape != (T, k) or weights.dtype != torch.float32 or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous float32 [T, k]")
    else:
        _same_device(index, weights=weights)
    _call("lora_route", index, _p(logits), ldl, dt, T, E, k, mode, bias.data_ptr() if bias is not None else None,
          _int(groups, "groups"), _int(top_groups, "top_groups"), int(renormalize), float(scale), _p(ids), _p(weights))
    return ids, weights
