"""Calls of the block operators at the edges of what their documentation allows, on the GPU."""
import ctypes

import pytest
import torch

from oracle import block as ob
from test_gpu_block import (ALL, check_boundary, check_boundary_grad, check_cross, check_cross_grad, f64, norm_case,
                            residual_both)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_top_b200 import build
    build.build()
    import block_sparse_attention_top_b200 as m
    return m


def rand(shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def plan_of(bsa, B, N, H, d):
    return bsa.Plan(B, H, 1, 1, N, d, 64, bsa.BSA_ORDER_IDENTITY)


# ------------------------------------------------------------------------ the norms

@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [8, 129, 520, 1219, 5120, 8200])
@pytest.mark.parametrize("N,groups", [(6, 6), (1, 1), (6, 2), (6, 1)])
def test_gradients_of_parameters_that_make_no_h_are_zero(bsa, N, groups, C, stream):
    """norm NONE: the boundary makes no h, so scale, shift, weight and bias have no part in it.  Every gradient that is
    asked for is written all the same: zeros."""
    B = 2
    plan = plan_of(bsa, B, N, 1, 64)
    x, y, dxo = rand((B, N, C), 1, stream), rand((B, N, C), 2), rand((B, N, C), 3, stream)
    par = {n: rand(s, 4 + i, torch.float32) for i, (n, s) in enumerate(
        dict(gate=(B, groups, C), scale=(B, groups, C), shift=(B, groups, C), weight=(C,), bias=(C,),
             post_weight=(C,)).items())}
    par["scale"][0, 0, 0], par["weight"][0] = float("inf"), float("nan")   # not read: they make no h
    a = bsa.NormArgs(C, groups, bsa.BSA_BF16 if stream == torch.bfloat16 else bsa.BSA_F32, bsa.BSA_NORM_NONE,
                     bsa.BSA_NORM_RMS, 1e-6, 1.0, *(par[n].data_ptr() for n in
                                                    ("gate", "scale", "shift", "weight", "bias", "post_weight")))
    names = ("gate", "scale", "shift", "weight", "bias", "post_weight")
    out = {n: torch.full_like(par[n], float("nan")) for n in names}
    dx, dy = torch.full_like(x, float("nan")), torch.full_like(y, float("nan"))
    ws = torch.empty(bsa._lib.bsa_norm_bwd_workspace_size(plan.handle, ctypes.byref(a)), dtype=torch.uint8, device="cuda")
    rc = bsa._lib.bsa_residual_norm_bwd(plan.handle, ctypes.byref(a), None, dxo.data_ptr(), x.data_ptr(), y.data_ptr(),
                                        dx.data_ptr(), dy.data_ptr(), *(out[n].data_ptr() for n in names),
                                        ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == bsa.BSA_OK
    torch.cuda.synchronize()
    for n in ("scale", "shift", "weight", "bias"):
        assert (out[n] == 0).all(), n
    plain = bsa.residual_norm_backward(plan, None, dxo, x, y, gate=par["gate"], post_weight=par["post_weight"],
                                       norm=bsa.BSA_NORM_NONE, post_norm=bsa.BSA_NORM_RMS)
    for got, want in ((dx, plain.dx), (dy, plain.dy), (out["gate"], plain.dgate), (out["post_weight"], plain.dpost_weight)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("C", [24, 129, 1536])
@pytest.mark.parametrize("groups", [1, 2, 6])
def test_norm_modulate_reads_no_gate_and_no_post_weight(bsa, groups, C):
    """One struct of arguments for both norm operators: what norm_modulate and its gradient do not read may hold
    anything (here NaN, one group of it)."""
    B, N = 2, 6
    plan = plan_of(bsa, B, N, 1, 64)
    x, dh = rand((B, N, C), 1, torch.float32), rand((B, N, C), 2)
    par = dict(scale=rand((B, groups, C), 3, torch.float32), shift=rand((B, groups, C), 4, torch.float32),
               weight=rand((C,), 5, torch.float32), bias=rand((C,), 6, torch.float32))
    h, grads = bsa.norm_modulate(plan, x, **par), bsa.norm_modulate_backward(plan, dh, x, **par)
    nan = torch.full((B * N * C,), float("nan"), device="cuda")
    p = {n: t.data_ptr() for n, t in par.items()}
    a = bsa.NormArgs(C, groups, bsa.BSA_F32, bsa.BSA_NORM_LAYER, bsa.BSA_NORM_NONE, 1e-6, float("nan"), nan.data_ptr(),
                     p["scale"], p["shift"], p["weight"], p["bias"], nan.data_ptr())
    s = torch.cuda.current_stream().cuda_stream
    h2, dx = torch.empty_like(h), torch.empty_like(x)
    assert bsa._lib.bsa_norm_modulate(plan.handle, ctypes.byref(a), x.data_ptr(), h2.data_ptr(), s) == bsa.BSA_OK
    out = {n: torch.empty_like(t) for n, t in par.items()}
    ws = torch.empty(bsa._lib.bsa_norm_bwd_workspace_size(plan.handle, ctypes.byref(a)), dtype=torch.uint8, device="cuda")
    assert bsa._lib.bsa_norm_modulate_bwd(plan.handle, ctypes.byref(a), dh.data_ptr(), x.data_ptr(), dx.data_ptr(),
                                          *(out[n].data_ptr() for n in par), ws.data_ptr(), ws.numel(), s) == bsa.BSA_OK
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(dx, grads.dx)
    for n in par:
        assert torch.equal(out[n], getattr(grads, "d" + n)), n


# ------------------------------------------------------------------ cross attention

# rows and states: the tensor-core kernel with one and with several key tiles, and the split kernel
@pytest.mark.parametrize("N,M", [(200, 40), (200, 300), (3, 40), (1, 700)])
def test_a_query_row_of_nan_stays_nan(bsa, N, M):
    """All scores of a row are NaN: so are its output and its lse.  -inf is the sign of a row without valid states."""
    B, H, d = 2, 2, 64
    q, k, v = rand((B, N, H, d), 1), rand((B, M, H, d), 2), rand((B, M, H, d), 3)
    plan = plan_of(bsa, B, N, H, d)
    for kw in ({}, dict(kv_len=torch.tensor([M - 3, 0], dtype=torch.int32).cuda()),
               dict(key_mask=(torch.arange(B * M).view(B, M) >= 33).cuda())):
        o, lse = bsa.cross_attn(plan, q, k, v, return_lse=True, **kw)
        q2 = q.clone()
        q2[:, 0, 1, 5] = float("nan")
        o2, lse2 = bsa.cross_attn(plan, q2, k, v, return_lse=True, **kw)
        assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
        for b in range(B):
            if "kv_len" in kw and b == 1:
                assert not o2[b].any() and torch.isneginf(lse2[b]).all()
                continue
            assert torch.isnan(o2[b, 0, 1]).all() and torch.isnan(lse2[b, 1, 0])
            o2[b, 0, 1], lse2[b, 1, 0] = o[b, 0, 1], lse[b, 1, 0]
        assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("N,M", [(200, 40), (200, 300), (3, 40), (1, 700)])
def test_a_query_row_of_scores_minus_infinity_is_empty(bsa, N, M):
    B, H, d = 1, 2, 64
    q, k, v = rand((B, N, H, d), 1).abs() + 0.5, rand((B, M, H, d), 2), rand((B, M, H, d), 3)
    k[:, :, 1] = float("-inf")                                         # the second head: q > 0, so every score is -inf
    o, lse = bsa.cross_attn(plan_of(bsa, B, N, H, d), q, k, v, return_lse=True)
    assert not o[:, :, 1].any() and torch.isneginf(lse[:, 1]).all()
    assert torch.isfinite(o[:, :, 0].float()).all() and torch.isfinite(lse[:, 0]).all()


# one key tile, several, and enough rows that the key side's work is split into shares
@pytest.mark.parametrize("N,M", [(150, 40), (150, 300), (2000, 200)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gradients_of_what_does_not_count_are_zero(bsa, bad, N, M):
    """Query rows without a valid state and states that do not count get zero gradients, whatever d_o holds there."""
    B, H, d = 3, 2, 64
    q, k, v, do = rand((B, N, H, d), 1), rand((B, M, H, d), 2), rand((B, M, H, d), 3), rand((B, N, H, d), 4)
    mask = torch.arange(B * M).view(B, M) % 3 != 1
    mask[1] = False                                                    # batch entry 1: no state counts
    mask = mask.cuda()
    plan = plan_of(bsa, B, N, H, d)
    o, lse = bsa.cross_attn(plan, q, k, v, key_mask=mask, return_lse=True)
    want = bsa.cross_attn_backward(plan, do, q, k, v, o, lse, key_mask=mask)
    do2 = do.clone()
    do2[1] = bad
    got = bsa.cross_attn_backward(plan, do2, q, k, v, o, lse, key_mask=mask)
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b) and not a[1].any()
    do2[2, 7] = bad                                                    # a row whose states count: theirs are not finite
    _, dk, dv = bsa.cross_attn_backward(plan, do2, q, k, v, o, lse, key_mask=mask)
    assert not dk[~mask].any() and not dv[~mask].any()
    assert not torch.isfinite(dv[2][mask[2]].float()).all()


# ------------------------------------------------------------------------ a whole block

@pytest.mark.parametrize("p", [0.4, 1.0])
def test_dit_block_is_its_parts(bsa, p):
    """Bit for bit the calls one after the other, with routing that drops blocks, and with q, k and v as views of one
    fused projection."""
    B, H, d, T, Hs, Ws, M, Hkv = 2, 2, 64, 2, 17, 19, 23, 1
    N, C = T * Hs * Ws, H * d
    plan = bsa.Plan(B, H, T, Hs, Ws, d, 64)
    x = rand((B, N, C), 1, torch.float32)
    mod = [rand((B, T, C), 2 + i, torch.float32, 0.3) for i in range(6)]
    wqkv, w = rand((C, 3 * C), 10, scale=2 * C ** -0.5), [rand((C, C), 11 + i, scale=C ** -0.5) for i in range(4)]
    kc, vc = rand((B, M, Hkv, d), 20), rand((B, M, Hkv, d), 21)

    def fused(h):
        return (h @ wqkv).view(B, N, 3, H, d).unbind(2)

    def heads(t):
        return t.reshape(B, N, H, d)

    def flat(t):
        return t.reshape(B, N, C)

    args = dict(attn_out=lambda o: flat(o) @ w[0], cross_q=lambda h: heads(h @ w[1]), cross_out=lambda o: flat(o) @ w[2],
                ffn=lambda h: h @ w[3], k_ctx=kc, v_ctx=vc, p=p, k_floor=1)
    got = bsa.dit_block(plan, x, mod, qkv=fused, **args)
    dense = bsa.dit_block(plan, x, mod, qkv=lambda h: tuple(t.contiguous() for t in fused(h)), **args)
    t1, s1, g1, t2, s2, g2 = mod
    h = bsa.norm_modulate(plan, x, scale=s1, shift=t1)
    q, k, v = (t.contiguous() for t in fused(h))
    row_ptr, col_idx, _, nnz = bsa.route(plan, q, k, p, 1)
    assert (int(nnz.item()) < plan.rows * plan.nb) == (p < 1)
    y = args["attn_out"](bsa.sparse_attn(plan, q, k, v, row_ptr, col_idx))
    a, h = bsa.residual_norm(plan, x, y, gate=g1)
    y = args["cross_out"](bsa.cross_attn(plan, args["cross_q"](h), kc, vc))
    a, h = bsa.residual_norm(plan, a, y, scale=s2, shift=t2)
    want = bsa.residual_norm(plan, a, args["ffn"](h), gate=g2, norm=bsa.BSA_NORM_NONE)[0]
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
    assert torch.equal(dense, want)
    assert torch.equal(got, want)


@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("C", [5128, 5632, 5640, 8192, 8200, 10240, 10248, 11264, 11272, 5121, 8193, 10241])
def test_norms_on_both_sides_of_each_variant_s_widths(bsa, C, stream):
    """The widths at which the launch takes another kernel (threads, rows in the ring, no ring), in both directions."""
    for groups in ("frame", "token"):
        case = norm_case(bsa, 1, 2, 7, C, groups, stream, "layer", "rms", ALL, seed=C, res_scale=0.75)
        residual_both(bsa, case, seed=C)
    plan, x, t, kw, opt, store, F = norm_case(bsa, 1, 2, 7, C, "frame", stream, "rms", None, ALL, seed=C, residual=False)
    h, dh = bsa.norm_modulate(plan, x, **t, **kw), rand(x.shape, C + 1)
    check_boundary(None, h, f64(x), t, opt, store)
    check_boundary_grad(bsa.norm_modulate_backward(plan, dh, x, **t, **kw), f64(x), f64(dh), None, t, opt, F, store)



@pytest.mark.parametrize("C", [200, 1219, 1536, 5632, 8200])
@pytest.mark.parametrize("groups", ["frame", "token"])
@pytest.mark.parametrize("post", [None, "layer"])
def test_residual_norm_gradient_in_place(bsa, post, groups, C):
    """dx over dx_out and dy over y, as the header allows: the kernel reads the next rows before it writes this one."""
    plan, x, t, kw, opt, store, F = norm_case(bsa, 2, 3, 50, C, groups, "f32", "layer", post, ALL, seed=C)
    y, par = t["y"], {n: v for n, v in t.items() if n != "y"}
    dh, dxo = rand(x.shape, C + 1), rand(x.shape, C + 2, torch.float32)
    want = bsa.residual_norm_backward(plan, dh, dxo, x, y, **par, **kw)
    names = ("gate", "scale", "shift", "weight", "bias", "post_weight")
    a = bsa.NormArgs(C, F, bsa.BSA_F32, kw["norm"], kw["post_norm"], kw["eps"], kw["res_scale"],
                     *(par[n].data_ptr() for n in names))
    ws = torch.empty(bsa._lib.bsa_norm_bwd_workspace_size(plan.handle, ctypes.byref(a)), dtype=torch.uint8, device="cuda")
    out = {n: torch.empty_like(par[n]) for n in names}
    dx, dy = dxo.clone(), y.clone()
    rc = bsa._lib.bsa_residual_norm_bwd(plan.handle, ctypes.byref(a), dh.data_ptr(), dx.data_ptr(), x.data_ptr(),
                                        dy.data_ptr(), dx.data_ptr(), dy.data_ptr(), *(out[n].data_ptr() for n in names),
                                        ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == bsa.BSA_OK
    torch.cuda.synchronize()
    assert torch.equal(dx, want.dx) and torch.equal(dy, want.dy)
    for n in names:
        assert torch.equal(out[n], getattr(want, "d" + n)), n


# ------------------------------------------------------------------------ large and many

def gpu_rand(shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), dtype=dtype, device="cuda")


def test_cross_attention_of_queries_past_32_bits(bsa):
    """q, o, d_o and dq of more than 2^31 elements: the last rows against a call on those rows alone."""
    H, d, M, n = 16, 128, 70, 384
    N = 2 ** 31 // (H * d) + 3 * 128 + 5
    q, do = gpu_rand((1, N, H, d), 1), gpu_rand((1, N, H, d), 2)
    k, v = gpu_rand((1, M, H, d), 3), gpu_rand((1, M, H, d), 4)
    plan, tail = plan_of(bsa, 1, N, H, d), plan_of(bsa, 1, n, H, d)
    o, lse = bsa.cross_attn(plan, q, k, v, return_lse=True)
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
    q1, do1 = q[:, -n:].contiguous(), do[:, -n:].contiguous()
    o1, lse1 = bsa.cross_attn(tail, q1, k, v, return_lse=True)
    assert torch.equal(o[:, -n:], o1) and torch.equal(lse[:, :, -n:], lse1)
    # only the last rows have a gradient: theirs is dq, and all of dk and dv
    do[:, :-n] = 0
    dq, dk, dv = bsa.cross_attn_backward(plan, do, q, k, v, o, lse)
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
    dq1, dk1, dv1 = bsa.cross_attn_backward(tail, do1, q1, k, v, o1, lse1)
    assert torch.equal(dq[:, -n:], dq1) and not dq[:, :-n].any()
    # The same sums in other shares: two roundings to bf16 (2^-8 each), and fp32 sums of n terms whose absolute values
    # add up to about 5 (dv: sum P |do|; dk: sum |dS| |q| / sqrt(d)) and nowhere to 40: n 2^-24 40 < 1e-3.
    for a, b in ((dk, dk1), (dv, dv1)):
        assert ((a - b).float().abs() <= 2 ** -7 * b.float().abs() + 1e-3).all()


@pytest.mark.parametrize("N", [1, 130])
def test_cross_attention_of_states_past_32_bits(bsa, N):
    """k and v of more than 2^31 elements; only the last states count."""
    B, H, d, n = 2, 8, 128, 300
    M = 2 ** 30 // (H * d) + 77
    k, v = gpu_rand((B, M, H, d), 1), gpu_rand((B, M, H, d), 2)
    q = gpu_rand((B, N, H, d), 3)
    mask = torch.zeros(B, M, dtype=torch.bool, device="cuda")
    mask[:, -n:] = True
    plan = plan_of(bsa, B, N, H, d)
    o, lse = bsa.cross_attn(plan, q, k, v, key_mask=mask, return_lse=True)
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
    check_cross(o, lse, q, k[:, -n:], v[:, -n:], ob.valid_states(B, n))


def test_norms_past_32_bits(bsa):
    """Streams of more than 2^31 elements: the last rows against a call on those rows alone."""
    C, n, G = 4096, 64, 5
    N = G * (2 ** 31 // C // G + 40)
    x, y = gpu_rand((1, N, C), 1), gpu_rand((1, N, C), 2)
    par = {name: gpu_rand((1, G, C), 3 + i, torch.float32) for i, name in enumerate(("gate", "scale", "shift"))}
    last = {name: t[:, -1:].contiguous() for name, t in par.items()}
    plan, tail = plan_of(bsa, 1, N, 1, 64), plan_of(bsa, 1, n, 1, 64)
    xo, h = bsa.residual_norm(plan, x, y, **par)
    x1, y1 = x[:, -n:].contiguous(), y[:, -n:].contiguous()
    xo1, h1 = bsa.residual_norm(tail, x1, y1, **last)
    assert torch.equal(xo[:, -n:], xo1) and torch.equal(h[:, -n:], h1)
    del x
    g = bsa.residual_norm_backward(plan, h, None, xo, y, **par)
    g1 = bsa.residual_norm_backward(tail, h1, None, xo1, y1, **last)
    assert torch.equal(g.dx[:, -n:], g1.dx) and torch.equal(g.dy[:, -n:], g1.dy)


def test_cross_attention_of_more_heads_than_a_grid_s_third_extent(bsa):
    """Few rows and 66 000 key heads: not the split kernel's call."""
    B, M, d = 66000, 3, 64
    q, k, v, do = (gpu_rand((B, n, 1, d), i) for i, n in enumerate((1, M, M, 1)))
    lens = (torch.arange(B, device="cuda") % (M + 1)).int()
    plan = plan_of(bsa, B, 1, 1, d)
    o, lse = bsa.cross_attn(plan, q, k, v, kv_len=lens, return_lse=True)
    grads = bsa.cross_attn_backward(plan, do, q, k, v, o, lse, kv_len=lens)
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
    on = ob.valid_states(B, M, lens.cpu().numpy())
    check_cross(o, lse, q, k, v, on)
    check_cross_grad(grads, q, k, v, on, do)


# ------------------------------------------------------------------------ streams and graphs

def test_streams_by_object_and_by_handle(bsa):
    """stream= takes torch's streams and raw handles, the default stream's 0 among them."""
    B, N, H, M, d, C = 1, 300, 2, 100, 64, 136
    plan = plan_of(bsa, B, N, H, d)
    q, k, v, do = (rand((B, n, H, d), i) for i, n in enumerate((N, M, M, N)))
    x, y = rand((B, N, C), 7), rand((B, N, C), 8)

    def step(s):
        o, lse = bsa.cross_attn(plan, q, k, v, return_lse=True, stream=s)
        xo, h = bsa.residual_norm(plan, x, y, stream=s)
        return (o, lse, *bsa.cross_attn_backward(plan, do, q, k, v, o, lse, stream=s), xo, h,
                *bsa.residual_norm_backward(plan, h, xo, xo, y, stream=s)[:2])

    want = step(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, torch.cuda.default_stream(), 0):
        got = step(stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_one_plan_on_two_streams_at_once(bsa):
    B, N, H, M, d = 2, 900, 3, 260, 128
    plan = plan_of(bsa, B, N, H, d)
    q, k, v, do = (rand((B, n, H, d), i) for i, n in enumerate((N, M, M, N)))
    mask = (torch.arange(B * M).view(B, M) % 5 != 0).cuda()

    def step(s=None, **kw):
        o, lse = bsa.cross_attn(plan, q, k, v, return_lse=True, stream=s, **kw)
        return (o, lse, *bsa.cross_attn_backward(plan, do, q, k, v, o, lse, stream=s, **kw))

    want = step(), step(key_mask=mask)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [(i, step(streams[i], **(dict(key_mask=mask) if i else {}))) for _ in range(10) for i in range(2)]
    torch.cuda.synchronize()
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
    for i, out in got:
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)


def test_captured_boundary_without_h(bsa):
    """A group per token and no h, captured: the zeros of dscale and dshift are part of the graph."""
    B, N, C = 2, 40, 264
    plan = plan_of(bsa, B, N, 1, 64)
    x, y, dxo = rand((B, N, C), 1), rand((B, N, C), 2), rand((B, N, C), 3)
    par = {n: rand((B, N, C), 4 + i, torch.float32) for i, n in enumerate(("gate", "scale", "shift"))}

    def step():
        return bsa.residual_norm_backward(plan, None, dxo, x, y, norm=bsa.BSA_NORM_NONE, **par)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (11, 12):
        dxo.copy_(rand(dxo.shape, seed))
        for t in out:
            if t is not None:
                t.fill_(float("nan"))
        g.replay()
        for a, b in zip(out, step()):
            assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
        assert not out.dscale.any() and not out.dshift.any()
