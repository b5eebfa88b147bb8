"""Python binding of libbsa: Top-p block routing + block-sparse attention on B200.

Argument marshalling only: every step of the path runs in the CUDA kernels of
libbsa.so (csrc/).  PyTorch supplies device memory and streams.  If the
library is missing the import fails loudly; there is no CPU path.

The functions keep the C names (bsa_route, bsa_sparse_attn, ...) and take
torch tensors where the C call takes device pointers; `Plan` wraps
bsa_plan_create / bsa_plan_destroy.  `route`, `sparse_attn` and
`sparse_attn_fp8v` are thin conveniences that allocate the outputs and the
workspace with torch.

    import torch, block_sparse_attention_top_b200 as bsa
    # q, k, v: bf16 [B, N, H, d] on cuda, N = T * Hs * Ws latent tokens
    plan = bsa.Plan(B, H, T, Hs, Ws, d, 128)             # frame-major Hilbert order
    row_ptr, col_idx, L_h, nnz = bsa.route(plan, q, k, 0.9, 4)   # Top-p 0.9, floor 4
    o = bsa.sparse_attn(plan, q, k, v, row_ptr, col_idx)        # bf16 [B, N, H, d]
    o8 = bsa.sparse_attn_fp8v(plan, q, k, v, row_ptr, col_idx)  # e4m3 P.V product
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK

The operators of a block around its self-attention (cross attention to an
encoder's states, and the norms with modulation, gate and residual) take the
same plan; `dit_block` runs a whole block:

    c = bsa.cross_attn(plan, q, k_text, v_text, kv_len=lengths)       # k, v: bf16 [B, M, Hkv, d]
    h = bsa.norm_modulate(plan, x, scale=s1, shift=t1)                 # x: [B, N, C] bf16 or float32
    x, h = bsa.residual_norm(plan, x, y, gate=g1, scale=s2, shift=t2)  # x + g1 y, then its norm
    # gradients: cross_attn_backward, norm_modulate_backward, residual_norm_backward

None of the calls records an autograd graph: a model that trains through them calls the gradients in the backward of
a torch.autograd.Function of its own.  The operators above warn where an input requires a gradient that would be lost.
"""
from __future__ import annotations

import collections
import ctypes
import os
import warnings

import torch

from . import build as _build

LIB_PATH = _build.LIB
if _build.stale():
    # missing or older than its sources: build it now, or fail loudly (there is no CPU path)
    try:
        _build.build()
    except Exception as exc:  # noqa: BLE001
        raise ImportError(f"libbsa.so at {LIB_PATH} is missing or stale and could not be built: {exc}") from exc
_lib = ctypes.CDLL(LIB_PATH)

BSA_OK, BSA_EINVAL, BSA_EUNSUPPORTED, BSA_ECAPACITY, BSA_EWORKSPACE, BSA_ECUDA, BSA_EDEVICE = 0, -1, -2, -3, -4, -5, -6
BSA_ORDER_HILBERT2D_FRAME, BSA_ORDER_IDENTITY = 0, 1
BSA_BF16, BSA_F32 = 0, 1
BSA_OP_ROUTE, BSA_OP_ATTN, BSA_OP_MASK, BSA_OP_AUGMENT = 0, 1, 2, 3
BSA_SCHED_L2_HEADS, BSA_SCHED_HEAVIEST_FIRST, BSA_SCHED_IN_ORDER = 0, 1, 2
BSA_NORM_NONE, BSA_NORM_LAYER, BSA_NORM_RMS = 0, 1, 2

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_I64x9 = _I64 * 9


class NormArgs(ctypes.Structure):
    """bsa_norm_args."""
    _fields_ = [("C", _I), ("groups", _I), ("dtype", _I), ("norm", _I), ("post_norm", _I),
                ("eps", ctypes.c_float), ("res_scale", ctypes.c_float), ("gate", _P), ("scale", _P), ("shift", _P),
                ("weight", _P), ("bias", _P), ("post_weight", _P)]


_NA = ctypes.POINTER(NormArgs)

_SIGS = {
    "bsa_plan_create": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I, _I, _I, _I, _I]),
    "bsa_plan_destroy": (None, [_P]),
    "bsa_plan_info": (_I, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "bsa_plan_set_schedule": (_I, [_P, _I]),
    "bsa_plan_set_wait_limit": (_I, [_P, ctypes.c_uint64]),
    "bsa_schedule_balance": (_I, [_P, _P, _P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_I64),
                                  ctypes.POINTER(ctypes.c_double)]),
    "bsa_attn_intermediates": (_I, [_P, _P, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P)]),
    "bsa_token_order": (_I, [_I, _I, _I, _I, _P]),
    "bsa_workspace_size": (_SZ, [_P, _I]),
    "bsa_route": (_I, [_P, _P, _P, _I, ctypes.c_float, _I, _P, _P, _I64, _P, _P, _P, _SZ, _P]),
    "bsa_route_static": (_I, [_P, _P, _P, _I, ctypes.c_float, _I, _P, _P, _I64, _P, _P, _P]),
    "bsa_route_intermediates": (_I, [_P, _P, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P)]),
    "bsa_mask_window_anchor": (_I, [_P, _I, _I, _I, _P, _P, _I64, _P, _P, _SZ, _P]),
    "bsa_route_order": (_I, [_P, _P, ctypes.POINTER(_P)]),
    "bsa_augment": (_I, [_P, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _SZ, _P]),
    "bsa_sasa_budget": (_I, [_I, _P, ctypes.c_float, ctypes.c_float, ctypes.c_float, _P, _P, _P, _P, _P]),
    "bsa_rlb_plan": (_I, [_I, _I, _P, _P, _P, ctypes.POINTER(_I), _P, _P, _P]),
    "bsa_rank_loads": (_I, [_I, _I, _P, _P, _P, _P, _P]),
    "bsa_rlb_gain": (_I, [_I, _P, _P, ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                          _P, _P]),
    "bsa_mask_stripes": (_I, [_I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _I64, _P]),
    "bsa_mask_stripes_device": (_I, [_P, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "bsa_balance_policy": (_I, [ctypes.c_float, ctypes.c_float, ctypes.c_float]),
    "bsa_sparse_attn": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_attn_prepare": (_I, [_P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_attn_run": (_I, [_P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_attn_run_simt": (_I, [_P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_sparse_attn_fp8v": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_attn_prepare_fp8v": (_I, [_P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_attn_run_fp8v": (_I, [_P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_cross_attn": (_I, [_P, _P, _P, _P, _I64, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_cross_attn_bwd": (_I, [_P, _P, _P, _P, _I64, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_cross_attn_workspace_size": (_SZ, [_P, _I64, _I, _I]),
    "bsa_norm_modulate": (_I, [_P, _NA, _P, _P, _P]),
    "bsa_residual_norm": (_I, [_P, _NA, _P, _P, _P, _P, _P]),
    "bsa_norm_modulate_bwd": (_I, [_P, _NA, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_residual_norm_bwd": (_I, [_P, _NA, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "bsa_norm_bwd_workspace_size": (_SZ, [_P, _NA]),
    "bsa_last_device_error": (_I, [_P, _P]),
    "bsa_strerror": (ctypes.c_char_p, [_I]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


class BsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {bsa_strerror(status)} ({status})")
        self.status = status


def bsa_strerror(status: int) -> str:
    return _lib.bsa_strerror(status).decode()


def _check(status: int, where: str) -> None:
    if status != BSA_OK:
        raise BsaError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class Plan:
    """Owns a bsa_plan for one (B, H, T, Hs, Ws, head_dim, block, order) shape."""

    def __init__(self, B, H, T, Hs, Ws, head_dim, block, order=BSA_ORDER_HILBERT2D_FRAME):
        h = _P()
        _check(_lib.bsa_plan_create(ctypes.byref(h), B, H, T, Hs, Ws, head_dim, block, order), "bsa_plan_create")
        self.handle = h
        self.B, self.H, self.T, self.Hs, self.Ws, self.d, self.block, self.order = B, H, T, Hs, Ws, head_dim, block, order
        n, nb, rows = _I64(), _I64(), _I64()
        _check(_lib.bsa_plan_info(h, ctypes.byref(n), ctypes.byref(nb), ctypes.byref(rows)), "bsa_plan_info")
        self.N, self.nb, self.rows = n.value, nb.value, rows.value
        self.device = torch.device("cuda", torch.cuda.current_device())

    def set_schedule(self, schedule: int) -> None:
        _check(_lib.bsa_plan_set_schedule(self.handle, int(schedule)), "bsa_plan_set_schedule")

    def set_wait_limit(self, ns: int) -> None:
        _check(_lib.bsa_plan_set_wait_limit(self.handle, int(ns)), "bsa_plan_set_wait_limit")

    def workspace_size(self, op: int) -> int:
        return int(_lib.bsa_workspace_size(self.handle, op))

    def workspace(self, op: int, device="cuda") -> torch.Tensor:
        return torch.empty(self.workspace_size(op), dtype=torch.uint8, device=device)

    def close(self):
        if getattr(self, "handle", None):
            _lib.bsa_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def bsa_schedule_balance(plan, row_ptr, work):
    """Per-CTA load balance of a work list (host tensors or arrays): (rho, max blocks, mean blocks)."""
    rp = torch.as_tensor(row_ptr, dtype=torch.int32).cpu().contiguous()
    wk = torch.as_tensor(work, dtype=torch.int32).cpu().contiguous()
    if rp.numel() != plan.rows + 1 or wk.numel() != plan.rows:
        raise ValueError("row_ptr must hold rows + 1 entries and work rows entries")
    rho, mx, mean = ctypes.c_double(), _I64(), ctypes.c_double()
    _check(_lib.bsa_schedule_balance(plan.handle, rp.data_ptr(), wk.data_ptr(), ctypes.byref(rho), ctypes.byref(mx),
                                     ctypes.byref(mean)), "bsa_schedule_balance")
    return rho.value, mx.value, mean.value


def bsa_attn_intermediates(plan, workspace):
    """Device addresses of (work list, e4m3 V tiles, V scales) in a prepared attention workspace."""
    a, b, c = _P(), _P(), _P()
    _check(_lib.bsa_attn_intermediates(plan.handle, _ptr(workspace), ctypes.byref(a), ctypes.byref(b),
                                       ctypes.byref(c)), "bsa_attn_intermediates")
    return a.value, b.value, c.value


def bsa_token_order(T: int, Hs: int, Ws: int, order: int = BSA_ORDER_HILBERT2D_FRAME):
    """Host-only token permutation (int32 CPU tensor)."""
    out = torch.empty(T * Hs * Ws, dtype=torch.int32)
    _check(_lib.bsa_token_order(T, Hs, Ws, order, out.data_ptr()), "bsa_token_order")
    return out


def bsa_route(plan, q, k, dtype, p, k_floor, row_ptr, col_idx, col_cap, L_h, nnz, workspace, stream=None):
    return _lib.bsa_route(plan.handle, _ptr(q), _ptr(k), dtype, float(p), int(k_floor), _ptr(row_ptr),
                          _ptr(col_idx), int(col_cap), _ptr(L_h), _ptr(nnz), _ptr(workspace),
                          workspace.numel() if workspace is not None else 0, _stream(stream))


def bsa_route_static(plan, q, k, dtype, p, k_floor, row_ptr, col_idx, col_cap, L_h, nnz, stream=None):
    """bsa_route with the library's fixed device scratch instead of a caller workspace
    (for callers that cannot allocate when they route)."""
    return _lib.bsa_route_static(plan.handle, _ptr(q), _ptr(k), dtype, float(p), int(k_floor), _ptr(row_ptr),
                                 _ptr(col_idx), int(col_cap), _ptr(L_h), _ptr(nnz), _stream(stream))


def bsa_mask_window_anchor(plan, radius_frames, n_anchor, step, row_ptr, col_idx, col_cap, nnz, workspace,
                           stream=None):
    return _lib.bsa_mask_window_anchor(plan.handle, int(radius_frames), int(n_anchor), int(step), _ptr(row_ptr),
                                       _ptr(col_idx), int(col_cap), _ptr(nnz), _ptr(workspace),
                                       workspace.numel() if workspace is not None else 0, _stream(stream))


def bsa_route_order(plan, workspace):
    """Device address of the full importance order (uint16 [rows, nb]) in a route workspace."""
    out = _P()
    _check(_lib.bsa_route_order(plan.handle, _ptr(workspace), ctypes.byref(out)), "bsa_route_order")
    return out.value


def bsa_augment(plan, row_ptr, order, extra, row_ptr_out, col_idx_out, col_cap, L_h_out, nnz_out, workspace,
                stream=None):
    return _lib.bsa_augment(plan.handle, _ptr(row_ptr), _ptr(order), _ptr(extra), _ptr(row_ptr_out),
                            _ptr(col_idx_out), int(col_cap), _ptr(L_h_out), _ptr(nnz_out), _ptr(workspace),
                            workspace.numel() if workspace is not None else 0, _stream(stream))


def bsa_sasa_budget(L_r, n1=0.8, n2=0.07, S=0.0, heads_per_rank=None):
    """Host-only SASA budget (Eqs. 7-10).  Returns (B_r, L_aug, A, extra_per_head or None)."""
    R = len(L_r)
    L = torch.tensor(list(L_r), dtype=torch.float32)
    B = torch.empty(R, dtype=torch.float32)
    La = torch.empty(R, dtype=torch.float32)
    A = torch.empty(1, dtype=torch.float32)
    hp = ex = None
    if heads_per_rank is not None:
        hp = torch.tensor(list(heads_per_rank), dtype=torch.int32)
        ex = torch.empty(int(hp.sum()), dtype=torch.int32)
    _check(_lib.bsa_sasa_budget(R, L.data_ptr(), float(n1), float(n2), float(S), B.data_ptr(), La.data_ptr(),
                                A.data_ptr(), _ptr(hp), _ptr(ex)), "bsa_sasa_budget")
    return B, La, float(A[0]), ex


def bsa_rlb_plan(L_h, head_rank, R):
    """Host-only load-balancing plan: (moves [(src, dst, head)], L_r_new, rho_before, rho_after)."""
    Lh = torch.tensor(list(L_h), dtype=torch.float32)
    hr = torch.tensor(list(head_rank), dtype=torch.int32)
    moves = torch.empty(3 * R, dtype=torch.int32)
    n = _I()
    Ln = torch.empty(R, dtype=torch.float32)
    rb, ra = torch.empty(1), torch.empty(1)
    _check(_lib.bsa_rlb_plan(R, Lh.numel(), hr.data_ptr(), Lh.data_ptr(), moves.data_ptr(), ctypes.byref(n),
                             Ln.data_ptr(), rb.data_ptr(), ra.data_ptr()), "bsa_rlb_plan")
    mv = moves[:3 * n.value].view(-1, 3).tolist()
    return [tuple(m) for m in mv], Ln, float(rb[0]), float(ra[0])


def bsa_rank_loads(L_h, head_rank, R):
    """Host-only per-rank loads (Eq. 1), imbalance factor rho (Eq. 2) and head counts of a placement:
    returns (L_r float32 [R], rho, heads_per_rank int32 [R])."""
    Lh = torch.tensor([float(v) for v in L_h], dtype=torch.float32)
    hr = torch.tensor([int(v) for v in head_rank], dtype=torch.int32)
    if Lh.shape != hr.shape:
        raise ValueError("L_h and head_rank must have the same length")
    L_r = torch.empty(R, dtype=torch.float32)
    cnt = torch.empty(R, dtype=torch.int32)
    rho = ctypes.c_float()
    _check(_lib.bsa_rank_loads(int(R), Lh.numel(), hr.data_ptr(), Lh.data_ptr(), L_r.data_ptr(), ctypes.byref(rho),
                               cnt.data_ptr()), "bsa_rank_loads")
    return L_r, rho.value, cnt


def bsa_rlb_gain(L_r, L_r_new, c, P=0.0, C=0.0, A=0.0):
    """(K, G) of the review's gain model (Eqs. 3-4, 11) for rank loads before and after a plan."""
    a = torch.tensor([float(v) for v in L_r], dtype=torch.float32)
    b = torch.tensor([float(v) for v in L_r_new], dtype=torch.float32)
    if a.shape != b.shape:
        raise ValueError("L_r and L_r_new must have the same length")
    K, G = ctypes.c_double(), ctypes.c_double()
    _check(_lib.bsa_rlb_gain(a.numel(), a.data_ptr(), b.data_ptr(), float(c), float(P), float(C), float(A),
                             ctypes.byref(K), ctypes.byref(G)), "bsa_rlb_gain")
    return K.value, G.value


def bsa_mask_stripes(B, H, T, Hs, Ws, block, params, order=0):
    """Host stripe-mask CSR (row_ptr, col_idx) as int32 CPU tensors; params: H rows of
    (w_t, o_t, s_t, w_s, o_s, s_s)."""
    pr = torch.tensor([[int(v) for v in row] for row in params], dtype=torch.int32).reshape(-1)
    if pr.numel() != 6 * H:
        raise ValueError("params must hold 6 values per head")
    nb = -(-(T * Hs * Ws) // block)
    rows = B * H * nb
    row_ptr = torch.empty(rows + 1, dtype=torch.int32)
    nnz = ctypes.c_int64()
    cap = rows * nb                                   # every block kept: cannot overflow
    col_idx = torch.empty(max(cap, 1), dtype=torch.int32)
    _check(_lib.bsa_mask_stripes(B, H, T, Hs, Ws, block, order, pr.data_ptr(), row_ptr.data_ptr(),
                                 col_idx.data_ptr(), cap, ctypes.byref(nnz)), "bsa_mask_stripes")
    return row_ptr, col_idx[:nnz.value].clone()


def bsa_mask_stripes_device(plan, params, row_ptr, col_idx, col_cap, nnz, workspace, stream=None):
    """Device stripe-mask CSR into device row_ptr / col_idx / nnz; params: H rows of
    (w_t, o_t, s_t, w_s, o_s, s_s) (host)."""
    pr = torch.tensor([[int(v) for v in row] for row in params], dtype=torch.int32).reshape(-1)
    if pr.numel() != 6 * plan.H:
        raise ValueError("params must hold 6 values per head")
    return _lib.bsa_mask_stripes_device(plan.handle, pr.data_ptr(), _ptr(row_ptr), _ptr(col_idx), int(col_cap),
                                        _ptr(nnz), _ptr(workspace), workspace.numel() if workspace is not None else 0,
                                        _stream(stream))


def bsa_balance_policy(rho, k1=1.05, k2=1.10) -> int:
    return _lib.bsa_balance_policy(float(rho), float(k1), float(k2))


def migrate_heads(x, local_heads, moves, rank, group=None):
    """Carry out a plan's head moves with torch.distributed point-to-point sends.

    x: [B, N, H_local, d] tensor holding the heads listed in `local_heads`
    (global ids, same order); moves: [(src, dst, head)] from bsa_rlb_plan.
    Returns (x_new, local_heads_new): sent heads removed, received heads
    appended in move order.  Plumbing only: the data leaves and arrives as is.
    """
    import torch.distributed as dist
    keep = list(range(len(local_heads)))
    recv_bufs, recv_ids, reqs = [], [], []
    for src, dst, h in moves:
        if src == rank:
            i = local_heads.index(h)
            keep.remove(i)
            reqs.append(dist.isend(x[:, :, i].contiguous(), dst, group=group))
        elif dst == rank:
            buf = torch.empty_like(x[:, :, 0])
            reqs.append(dist.irecv(buf, src, group=group))
            recv_bufs.append(buf)
            recv_ids.append(h)
    for q in reqs:
        q.wait()
    parts = [x[:, :, i] for i in keep] + recv_bufs
    heads = [local_heads[i] for i in keep] + recv_ids
    return torch.stack(parts, dim=2) if parts else x[:, :, :0], heads


def balance_step(L_h_local, local_heads, tensors, rank, world, group=None, k1=1.05, k2=1.10, n1=0.8, n2=0.07):
    """One step of the pages' runtime balancing across ranks (FVAttn review, section 3 "Stage 2" and
    "Stage 3", section 3.3): all-gather the per-head workloads L_h (Eq. 1), take rho (Eq. 2) and the
    enabling policy; at policy 2 every rank computes the same pair-swap plan (Eqs. 5-6, bsa_rlb_plan)
    and the planned heads move with point-to-point sends; at policy >= 1 the slack-augmentation budget
    (Eqs. 7-10, bsa_sasa_budget) becomes a_h extra blocks for every query block of each local head.

    L_h_local: workloads of `local_heads` (global head ids, same order); tensors: [B, N, H_local, d]
    tensors holding those heads (all migrated alike).  Host plumbing over the library's host calls and
    torch.distributed; nothing here computes on the device.
    Returns dict(policy, rho_before, rho_after, moves, L_r, L_r_new, tensors, local_heads, extra).
    """
    import torch.distributed as dist
    mine = (list(local_heads), [float(v) for v in L_h_local])
    every = [None] * world
    dist.all_gather_object(every, mine, group=group)
    n_heads = sum(len(hs) for hs, _ in every)
    owner, L_h = [0] * n_heads, [0.0] * n_heads
    for r, (hs, ls) in enumerate(every):
        for h, l in zip(hs, ls):
            owner[h], L_h[h] = r, l
    L_r, rho, _ = bsa_rank_loads(L_h, owner, world)
    L_r = L_r.tolist()
    policy = bsa_balance_policy(rho, k1, k2)
    moves, L_r_new, rho_after = [], list(L_r), rho
    heads = list(local_heads)
    new_owner = list(owner)
    if policy == 2:
        moves, L_new, _, rho_after = bsa_rlb_plan(L_h, owner, world)
        L_r_new = L_new.tolist()
        for src, dst, h in moves:
            new_owner[h] = dst
        out = []
        for x in tensors:
            x_new, heads_new = migrate_heads(x, list(local_heads), moves, rank, group)
            out.append(x_new)
        tensors = out
        if tensors:
            heads = heads_new
        else:                                             # no payload: the head list still follows the plan
            heads = [h for h in local_heads if not any(m[2] == h and m[0] == rank for m in moves)]
            heads += [m[2] for m in moves if m[1] == rank]
    extra = [0] * len(heads)
    if policy >= 1:
        # heads each rank holds after the migration, in the order bsa_sasa_budget lists them
        _, _, counts = bsa_rank_loads(L_h, new_owner, world)
        counts = counts.tolist()
        if counts[rank] != len(heads):
            raise RuntimeError("head bookkeeping disagrees with the plan")
        _, _, _, ex = bsa_sasa_budget(L_r_new, n1, n2, heads_per_rank=counts)
        lo = sum(counts[:rank])
        extra = ex[lo:lo + counts[rank]].tolist()
    return dict(policy=policy, rho_before=rho, rho_after=rho_after, moves=moves, L_r=L_r, L_r_new=L_r_new,
                tensors=tensors, local_heads=heads, extra=extra)


def return_heads(out, heads, home_heads, moves, rank, group=None):
    """The reverse of migrate_heads: send every migrated head's output back to the rank it came from
    and return this rank's outputs in its original head order (FVAttn review, section 3 "Block-Sparse
    Attention Execution": the outputs of migrated heads go back and head order is restored).

    out: [B, N, H_now, d] outputs of the heads listed in `heads` (the order balance_step / migrate_heads
    returned); home_heads: this rank's heads before the migration, in their original order; moves: the
    plan's [(src, dst, head)].  Returns [B, N, len(home_heads), d].  Plumbing only."""
    import torch.distributed as dist
    home_of = {h: src for src, dst, h in moves}            # heads that moved: where they live
    reqs, kept, got = [], {}, {}
    for i, h in enumerate(heads):
        if h in home_of and home_of[h] != rank:            # computed here for another rank: send it home
            reqs.append(dist.isend(out[:, :, i].contiguous(), home_of[h], group=group))
        else:
            kept[h] = out[:, :, i]
    for src, dst, h in moves:
        if src == rank:                                    # ours, computed elsewhere: receive it
            buf = torch.empty_like(out[:, :, 0]) if out.shape[2] else torch.empty(
                out.shape[:2] + out.shape[3:], dtype=out.dtype, device=out.device)
            reqs.append(dist.irecv(buf, dst, group=group))
            got[h] = buf
    for q in reqs:
        q.wait()
    parts = []
    for h in home_heads:
        if h in kept:
            parts.append(kept[h])
        elif h in got:
            parts.append(got[h])
        else:
            raise RuntimeError(f"head {h} is neither kept nor received on rank {rank}")
    return torch.stack(parts, dim=2) if parts else out[:, :, :0]


def local_attention(q, k, v, T, Hs, Ws, block, p, k_floor, extra=None):
    """Route and attend over the heads a rank holds: bf16 [B, N, H_local, d] on its device; extra: SASA
    blocks per local head (bsa_augment), or None.  Returns (o, L_h) device tensors."""
    B, N, H, d = q.shape
    plan = Plan(B, H, T, Hs, Ws, d, block)
    ws = plan.workspace(BSA_OP_ROUTE, q.device)
    row_ptr, col_idx, L_h, _ = route(plan, q, k, p, k_floor, workspace=ws)
    if extra is not None and any(int(e) > 0 for e in extra):
        ex = torch.tensor([int(e) for e in extra], dtype=torch.int32, device=q.device)
        rp2 = torch.empty_like(row_ptr)
        ci2 = torch.empty(plan.rows * plan.nb, dtype=torch.int32, device=q.device)
        L2 = torch.empty_like(L_h)
        nnz2 = torch.empty(1, dtype=torch.int64, device=q.device)
        ws_aug = plan.workspace(BSA_OP_AUGMENT, q.device)
        _check(bsa_augment(plan, row_ptr, bsa_route_order(plan, ws), ex, rp2, ci2, ci2.numel(), L2, nnz2, ws_aug),
               "bsa_augment")
        row_ptr, col_idx, L_h = rp2, ci2, L2
    o = sparse_attn(plan, q, k, v, row_ptr, col_idx)
    _check(bsa_last_device_error(plan), "device error")
    return o, L_h


def balanced_attention(q, k, v, L_h_local, local_heads, rank, world, compute, group=None, **policy):
    """One balanced attention step over the ranks (FVAttn review, section 3): balance_step moves the
    planned heads' Q, K, V and decides the augmentation, `compute(q, k, v, heads, extra)` runs the
    rank-local route + attention over the heads the rank now holds (e.g. local_attention), and
    return_heads sends the migrated heads' outputs home in the original head order.
    Returns (o [B, N, H_local, d] in `local_heads` order, the balance_step record)."""
    st = balance_step(L_h_local, local_heads, [q, k, v], rank, world, group=group, **policy)
    q2, k2, v2 = st["tensors"]
    o2 = compute(q2, k2, v2, st["local_heads"], st["extra"])
    return return_heads(o2, st["local_heads"], list(local_heads), st["moves"], rank, group), st


def bsa_route_intermediates(plan, workspace):
    a, b, c = _P(), _P(), _P()
    _check(_lib.bsa_route_intermediates(plan.handle, _ptr(workspace), ctypes.byref(a), ctypes.byref(b),
                                        ctypes.byref(c)), "bsa_route_intermediates")
    return a.value, b.value, c.value


def bsa_sparse_attn(plan, q, k, v, row_ptr, col_idx, o, workspace, stream=None):
    return _lib.bsa_sparse_attn(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(row_ptr), _ptr(col_idx), _ptr(o),
                                _ptr(workspace), workspace.numel(), _stream(stream))


def bsa_attn_prepare(plan, q, k, v, row_ptr, workspace, stream=None):
    return _lib.bsa_attn_prepare(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(row_ptr), _ptr(workspace),
                                 workspace.numel(), _stream(stream))


def bsa_attn_run(plan, row_ptr, col_idx, o, workspace, stream=None):
    return _lib.bsa_attn_run(plan.handle, _ptr(row_ptr), _ptr(col_idx), _ptr(o), _ptr(workspace),
                             workspace.numel(), _stream(stream))


def bsa_attn_run_simt(plan, row_ptr, col_idx, o, workspace, stream=None):
    return _lib.bsa_attn_run_simt(plan.handle, _ptr(row_ptr), _ptr(col_idx), _ptr(o), _ptr(workspace),
                                  workspace.numel(), _stream(stream))


def bsa_sparse_attn_fp8v(plan, q, k, v, row_ptr, col_idx, o, workspace, stream=None):
    return _lib.bsa_sparse_attn_fp8v(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(row_ptr), _ptr(col_idx),
                                     _ptr(o), _ptr(workspace), workspace.numel(), _stream(stream))


def bsa_attn_prepare_fp8v(plan, q, k, v, row_ptr, workspace, stream=None):
    return _lib.bsa_attn_prepare_fp8v(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(row_ptr), _ptr(workspace),
                                      workspace.numel(), _stream(stream))


def bsa_attn_run_fp8v(plan, row_ptr, col_idx, o, workspace, stream=None):
    return _lib.bsa_attn_run_fp8v(plan.handle, _ptr(row_ptr), _ptr(col_idx), _ptr(o), _ptr(workspace),
                                  workspace.numel(), _stream(stream))


def bsa_last_device_error(plan, stream=None) -> int:
    return _lib.bsa_last_device_error(plan.handle, _stream(stream))


# ---- conveniences (allocate outputs with torch, raise on error) ----

def route(plan: Plan, q: torch.Tensor, k: torch.Tensor, p: float, k_floor: int, workspace=None,
          col_cap: int | None = None, stream=None):
    """Returns (row_ptr, col_idx[:col_cap], L_h, nnz) device tensors; nnz stays on device."""
    dev = q.device
    dtype = BSA_BF16 if q.dtype == torch.bfloat16 else BSA_F32
    if col_cap is None:
        col_cap = plan.rows * plan.nb
    row_ptr = torch.empty(plan.rows + 1, dtype=torch.int32, device=dev)
    col_idx = torch.empty(max(col_cap, 1), dtype=torch.int32, device=dev)
    L_h = torch.empty(plan.B * plan.H, dtype=torch.float32, device=dev)
    nnz = torch.empty(1, dtype=torch.int64, device=dev)
    if workspace is None:
        workspace = plan.workspace(BSA_OP_ROUTE, dev)
    _check(bsa_route(plan, q, k, dtype, p, k_floor, row_ptr, col_idx, col_cap, L_h, nnz, workspace, stream),
           "bsa_route")
    return row_ptr, col_idx, L_h, nnz


def sparse_attn(plan: Plan, q, k, v, row_ptr, col_idx, workspace=None, out=None, stream=None):
    """O = block-sparse attention of bf16 [B,N,H,d] inputs under the CSR mask."""
    if workspace is None:
        workspace = plan.workspace(BSA_OP_ATTN, q.device)
    o = torch.empty_like(q) if out is None else out
    _check(bsa_sparse_attn(plan, q, k, v, row_ptr, col_idx, o, workspace, stream), "bsa_sparse_attn")
    return o


def sparse_attn_fp8v(plan: Plan, q, k, v, row_ptr, col_idx, workspace=None, out=None, stream=None):
    """As sparse_attn, with the e4m3 P.V product (block 128 only)."""
    if workspace is None:
        workspace = plan.workspace(BSA_OP_ATTN, q.device)
    o = torch.empty_like(q) if out is None else out
    _check(bsa_sparse_attn_fp8v(plan, q, k, v, row_ptr, col_idx, o, workspace, stream), "bsa_sparse_attn_fp8v")
    return o


# ---- operators of a block around its self-attention ----
#
# These check types, shapes, layouts and devices (ValueError) before the call; the library checks the rest
# (BsaError).  Outputs and workspace come from `stream`'s pool (default: the current stream), so nothing
# that a launch still uses is handed out again.

class _On:
    """Makes `stream` (None: the current one) the current stream of the plan's device, and that device current;
    entered, it is the raw stream."""

    def __init__(self, plan, stream):
        self._dev = self._stream = None
        self._index = plan.device.index
        if stream is None and torch.cuda.current_device() == plan.device.index:
            return                                                    # nothing to change
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
            stream = torch.cuda.ExternalStream(raw, device=plan.device)
        if stream is not None and stream.device != plan.device:
            raise ValueError(f"stream is on {stream.device}, the plan on {plan.device}")
        self._dev, self._stream = torch.cuda.device(plan.device), torch.cuda.stream(stream)

    def __enter__(self):
        if self._dev is not None:
            self._dev.__enter__()
            self._stream.__enter__()
            return torch.cuda.current_stream().cuda_stream
        return torch._C._cuda_getCurrentRawStream(self._index)        # a tenth of current_stream()'s time

    def __exit__(self, *exc):
        if self._dev is not None:
            self._stream.__exit__(*exc)
            self._dev.__exit__(*exc)


def _need(plan, t, name, dtypes, shape, dense=True):
    if isinstance(t, torch.Tensor) and t.device == plan.device and t.dtype in dtypes and t.shape == shape and (
            not dense or t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor) or t.device != plan.device:
        raise ValueError(f"{name} must be a tensor on {plan.device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, not {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


_records = torch.is_grad_enabled


def _lost_gradient(name):
    """An input requires a gradient, and autograd will take the call's result for a constant."""
    warnings.warn(f"{name} records no autograd graph, and an input requires a gradient: call it in a "
                  f"torch.autograd.Function whose backward calls {name}_backward, or under torch.no_grad()", stacklevel=3)


def _learns(t):
    return t is not None and t.requires_grad


def _workspace(plan, need, workspace):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=plan.device) if need else None
    _need(plan, workspace, "workspace", (torch.uint8,), workspace.shape)
    return workspace


_BF16, _F32, _STREAM = (torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)


def _cross_inputs(plan, q, k, v, kv_len, key_mask):
    """Checks and the strides array of a cross attention's inputs: (M, Hkv, strides)."""
    _need(plan, q, "q", _BF16, (plan.B, plan.N, plan.H, plan.d), dense=False)
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be [B, M, Hkv, d]")
    M, Hkv = k.shape[1], k.shape[2]
    _need(plan, k, "k", _BF16, (plan.B, M, Hkv, plan.d), dense=False)
    _need(plan, v, "v", _BF16, (plan.B, M, Hkv, plan.d), dense=False)
    sq, sk, sv = q.stride(), k.stride(), v.stride()
    if sq[3] != 1 or sk[3] != 1 or sv[3] != 1:
        name = "q" if sq[3] != 1 else "k" if sk[3] != 1 else "v"
        raise ValueError(f"the channels of {name} must be contiguous")
    if kv_len is not None:
        _need(plan, kv_len, "kv_len", (torch.int32,), (plan.B,))
    if key_mask is not None:
        _need(plan, key_mask, "key_mask", (torch.bool, torch.uint8), (plan.B, M))
    return M, Hkv, _I64x9(*sq[:3], *sk[:3], *sv[:3])


def cross_attn(plan: Plan, q, k, v, kv_len=None, key_mask=None, return_lse=False, workspace=None, out=None,
               stream=None):
    """Cross attention of the plan's query tokens to an encoder's states (bsa_cross_attn).

    q: bf16 [B,N,H,d]; k, v: bf16 [B,M,Hkv,d], Hkv dividing H, e.g. views into one projection (channels
    contiguous, other strides multiples of 8 elements).  kv_len: int32 [B] on the device, key_mask: bool
    [B,M]; a state counts when both say so.  Returns o bf16 [B,N,H,d], or (o, lse float32 [B,H,N])."""
    M, Hkv, strides = _cross_inputs(plan, q, k, v, kv_len, key_mask)
    if _records() and (q.requires_grad or k.requires_grad or v.requires_grad):
        _lost_gradient("cross_attn")
    if out is not None:
        _need(plan, out, "out", _BF16, q.shape)
    with _On(plan, stream) as s:
        o = torch.empty_like(q, memory_format=torch.contiguous_format) if out is None else out
        lse = torch.empty(plan.B, plan.H, plan.N, dtype=torch.float32, device=plan.device) if return_lse else None
        ws = _workspace(plan, _lib.bsa_cross_attn_workspace_size(plan.handle, M, Hkv, 0), workspace)
        _check(_lib.bsa_cross_attn(plan.handle, _ptr(q), _ptr(k), _ptr(v), M, Hkv, strides, _ptr(kv_len),
                                   _ptr(key_mask), _ptr(o), _ptr(lse), _ptr(ws), ws.numel() if ws is not None else 0,
                                   s), "bsa_cross_attn")
    return (o, lse) if return_lse else o


def cross_attn_backward(plan: Plan, do, q, k, v, o, lse, kv_len=None, key_mask=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of cross_attn from do, its inputs and its outputs (bsa_cross_attn_bwd)."""
    M, Hkv, strides = _cross_inputs(plan, q, k, v, kv_len, key_mask)
    _need(plan, do, "do", _BF16, q.shape)
    _need(plan, o, "o", _BF16, q.shape)
    _need(plan, lse, "lse", _F32, (plan.B, plan.H, plan.N))
    with _On(plan, stream) as s:
        dq = torch.empty_like(q, memory_format=torch.contiguous_format)
        dk = torch.empty_like(k, memory_format=torch.contiguous_format)
        dv = torch.empty_like(v, memory_format=torch.contiguous_format)
        ws = _workspace(plan, _lib.bsa_cross_attn_workspace_size(plan.handle, M, Hkv, 1), workspace)
        _check(_lib.bsa_cross_attn_bwd(plan.handle, _ptr(q), _ptr(k), _ptr(v), M, Hkv, strides, _ptr(kv_len),
                                       _ptr(key_mask), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                                       _ptr(ws), ws.numel() if ws is not None else 0, s), "bsa_cross_attn_bwd")
    return dq, dk, dv


def _norm_inputs(plan, x, gate, scale, shift, weight, bias, post_weight, norm, post_norm, res_scale, eps):
    """Checks of a norm operator's stream and parameters, as a filled NormArgs."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be [B, N, C]")
    C = x.shape[2]
    _need(plan, x, "x", _STREAM, (plan.B, plan.N, C))
    first = gate if gate is not None else scale if scale is not None else shift
    groups = 1
    if first is not None:
        if not isinstance(first, torch.Tensor) or first.dim() != 3:
            raise ValueError("gate, scale and shift must be [B, groups, C]")
        groups = first.shape[1]
        shape = (plan.B, groups, C)
        if gate is not None:
            _need(plan, gate, "gate", _F32, shape)
        if scale is not None:
            _need(plan, scale, "scale", _F32, shape)
        if shift is not None:
            _need(plan, shift, "shift", _F32, shape)
    if weight is not None:
        _need(plan, weight, "weight", _F32, (C,))
    if bias is not None:
        _need(plan, bias, "bias", _F32, (C,))
    if post_weight is not None:
        _need(plan, post_weight, "post_weight", _F32, (C,))
    return NormArgs(C, groups, BSA_BF16 if x.dtype == torch.bfloat16 else BSA_F32, norm, post_norm, eps, res_scale,
                    _ptr(gate), _ptr(scale), _ptr(shift), _ptr(weight), _ptr(bias), _ptr(post_weight))


def norm_modulate(plan: Plan, x, scale=None, shift=None, weight=None, bias=None, norm=BSA_NORM_LAYER, eps=1e-6,
                  out=None, stream=None):
    """h = (norm(x) * weight + bias) * (1 + scale) + shift in bf16 (bsa_norm_modulate).  x: bf16 or float32
    [B,N,C]; scale, shift: float32 [B,groups,C], token n in group n // (N / groups); weight, bias: float32 [C]."""
    a = _norm_inputs(plan, x, None, scale, shift, weight, bias, None, norm, BSA_NORM_NONE, 1.0, eps)
    if _records() and (x.requires_grad or _learns(scale) or _learns(shift) or _learns(weight) or _learns(bias)):
        _lost_gradient("norm_modulate")
    if out is not None:
        _need(plan, out, "out", _BF16, x.shape)
    with _On(plan, stream) as s:
        h = torch.empty_like(x, dtype=torch.bfloat16) if out is None else out
        _check(_lib.bsa_norm_modulate(plan.handle, ctypes.byref(a), _ptr(x), _ptr(h), s), "bsa_norm_modulate")
    return h


def residual_norm(plan: Plan, x, y, gate=None, scale=None, shift=None, weight=None, bias=None, post_weight=None,
                  norm=BSA_NORM_LAYER, post_norm=BSA_NORM_NONE, res_scale=1.0, eps=1e-6, x_out=None, h_out=None,
                  stream=None):
    """A block's boundary (bsa_residual_norm): x_out = res_scale x + gate (post_norm(y) post_weight) in x's type and
    h = (norm(x_out) weight + bias)(1 + scale) + shift in bf16.  y: bf16 [B,N,C]; parameters as for
    norm_modulate.  norm=BSA_NORM_NONE: no h.  x_out may be x, h_out may be y.  Returns (x_out, h or None)."""
    a = _norm_inputs(plan, x, gate, scale, shift, weight, bias, post_weight, norm, post_norm, res_scale, eps)
    _need(plan, y, "y", _BF16, x.shape)
    if _records() and (x.requires_grad or y.requires_grad or any(
            map(_learns, (gate, scale, shift, weight, bias, post_weight)))):
        _lost_gradient("residual_norm")
    if x_out is not None:
        _need(plan, x_out, "x_out", (x.dtype,), x.shape)
    if h_out is not None:
        _need(plan, h_out, "h_out", _BF16, x.shape)
    with _On(plan, stream) as s:
        xo = torch.empty_like(x) if x_out is None else x_out
        h = None
        if norm != BSA_NORM_NONE:
            h = torch.empty_like(y) if h_out is None else h_out
        _check(_lib.bsa_residual_norm(plan.handle, ctypes.byref(a), _ptr(x), _ptr(y), _ptr(xo), _ptr(h), s),
               "bsa_residual_norm")
    return xo, h


NormGrads = collections.namedtuple("NormGrads", "dx dy dgate dscale dshift dweight dbias dpost_weight")


def _like(t):
    return None if t is None else torch.empty_like(t)


def norm_modulate_backward(plan: Plan, dh, x, scale=None, shift=None, weight=None, bias=None, norm=BSA_NORM_LAYER,
                           eps=1e-6, workspace=None, stream=None):
    """Gradients of norm_modulate from dh (bf16) as NormGrads: dx in x's type, one float32 tensor for each
    parameter given, None for the rest (bsa_norm_modulate_bwd)."""
    a = _norm_inputs(plan, x, None, scale, shift, weight, bias, None, norm, BSA_NORM_NONE, 1.0, eps)
    _need(plan, dh, "dh", _BF16, x.shape)
    with _On(plan, stream) as s:
        dx, ds, dt, dw, db = (_like(t) for t in (x, scale, shift, weight, bias))
        ws = _workspace(plan, _lib.bsa_norm_bwd_workspace_size(plan.handle, ctypes.byref(a)), workspace)
        _check(_lib.bsa_norm_modulate_bwd(plan.handle, ctypes.byref(a), _ptr(dh), _ptr(x), _ptr(dx), _ptr(ds),
                                          _ptr(dt), _ptr(dw), _ptr(db), _ptr(ws), ws.numel() if ws is not None else 0,
                                          s), "bsa_norm_modulate_bwd")
    return NormGrads(dx, None, None, ds, dt, dw, db, None)


def residual_norm_backward(plan: Plan, dh, dx_out, x_out, y, gate=None, scale=None, shift=None, weight=None,
                           bias=None, post_weight=None, norm=BSA_NORM_LAYER, post_norm=BSA_NORM_NONE, res_scale=1.0,
                           eps=1e-6, workspace=None, stream=None):
    """Gradients of residual_norm (bsa_residual_norm_bwd) from those of its outputs: dh (bf16; None exactly when
    norm is BSA_NORM_NONE) and dx_out (x's type, or None for zero).  x_out: the forward pass's output, y its
    input.  Returns NormGrads: dx, dy, and one float32 tensor for each parameter given."""
    a = _norm_inputs(plan, x_out, gate, scale, shift, weight, bias, post_weight, norm, post_norm, res_scale, eps)
    _need(plan, y, "y", _BF16, x_out.shape)
    if dh is not None:
        _need(plan, dh, "dh", _BF16, x_out.shape)
    if dx_out is not None:
        _need(plan, dx_out, "dx_out", (x_out.dtype,), x_out.shape)
    with _On(plan, stream) as s:
        dx, dy, dg, ds, dt, dw, db, dp = (_like(t) for t in (x_out, y, gate, scale, shift, weight, bias, post_weight))
        ws = _workspace(plan, _lib.bsa_norm_bwd_workspace_size(plan.handle, ctypes.byref(a)), workspace)
        _check(_lib.bsa_residual_norm_bwd(plan.handle, ctypes.byref(a), _ptr(dh), _ptr(dx_out), _ptr(x_out), _ptr(y),
                                          _ptr(dx), _ptr(dy), _ptr(dg), _ptr(ds), _ptr(dt), _ptr(dw), _ptr(db),
                                          _ptr(dp), _ptr(ws), ws.numel() if ws is not None else 0, s),
               "bsa_residual_norm_bwd")
    return NormGrads(dx, dy, dg, ds, dt, dw, db, dp)


def dit_block(plan: Plan, x, mod, qkv, attn_out, cross_q, cross_out, ffn, k_ctx, v_ctx, p, k_floor, kv_len=None,
              key_mask=None, cross_weight=None, cross_bias=None, norm=BSA_NORM_LAYER, eps=1e-6):
    """One video transformer block: routed block-sparse self-attention, cross attention to an encoder's states
    and the feed-forward half, each between its norms.

    x: [B,N,C] bf16 or float32; mod: six float32 [B,groups,C] tensors (shift, scale, gate of the self-attention
    half, then of the feed-forward half).  The host model's projections are callables: qkv(h) -> three [B,N,H,d],
    attn_out(o) -> y, cross_q(h) -> [B,N,H,d], cross_out(o) -> y, ffn(h) -> y, with h and y bf16 [B,N,C].  What qkv
    returns may be views of one fused projection (the self-attention reads dense tensors: others are copied).
    k_ctx, v_ctx: bf16 [B,M,Hkv,d] projections of the encoder's states; kv_len, key_mask: as for cross_attn;
    cross_weight, cross_bias: affine of the norm before the cross attention.  p, k_floor: as for route.
    Returns the block's output in x's type."""
    with _On(plan, None):                                 # route and sparse_attn launch on the current device
        t1, s1, g1, t2, s2, g2 = mod
        h = norm_modulate(plan, x, scale=s1, shift=t1, norm=norm, eps=eps)
        q, k, v = qkv(h)
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            _need(plan, t, name, _BF16, (plan.B, plan.N, plan.H, plan.d), dense=False)
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        row_ptr, col_idx, _, _ = route(plan, q, k, p, k_floor)
        y = attn_out(sparse_attn(plan, q, k, v, row_ptr, col_idx))
        x, h = residual_norm(plan, x, y, gate=g1, weight=cross_weight, bias=cross_bias, norm=norm, eps=eps)
        y = cross_out(cross_attn(plan, cross_q(h), k_ctx, v_ctx, kv_len=kv_len, key_mask=key_mask))
        x, h = residual_norm(plan, x, y, scale=s2, shift=t2, norm=norm, eps=eps)
        return residual_norm(plan, x, ffn(h), gate=g2, norm=BSA_NORM_NONE, eps=eps)[0]
