"""The block operators on the GPU against the fp64 oracle, element by element.

Every bound is derived before the run: a rounding to bf16 is off by at most 2^-8 of the value, fp32 by 2^-24; how the
terms of a formula carry them is written in oracle/block.py (cross attention) and at `norm_*` below.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_top_b200 import build
    build.build()
    import block_sparse_attention_top_b200 as m
    return m


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}, " \
        f"got {got[bad][0]} want {want[bad][0]} bound {np.broadcast_to(bound, want.shape)[bad][0]}"


def rand(shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


# ------------------------------------------------------------------ cross attention

# B, N, H, Hkv, M, d
SHAPES = [
    (1, 1, 1, 1, 1, 64), (1, 1, 2, 1, 33, 128), (2, 3, 4, 2, 7, 64), (1, 127, 2, 2, 128, 128), (1, 128, 1, 1, 129, 64),
    (2, 130, 6, 2, 77, 128), (1, 257, 3, 3, 257, 64), (3, 65, 2, 2, 300, 128), (1, 300, 2, 1, 513, 128),
    (1, 1, 5, 1, 1000, 128), (4, 2, 10, 2, 700, 64), (1, 5, 8, 1, 129, 128), (1, 513, 2, 2, 64, 64),
    (1, 640, 1, 1, 1030, 128), (1, 17, 16, 16, 63, 64),
]


def plan_of(bsa, B, N, H, d):
    return bsa.Plan(B, H, 1, 1, N, d, 64, bsa.BSA_ORDER_IDENTITY)


def masks_of(kind, B, M, seed=0):
    g = np.random.default_rng(seed + 17 * M + B)
    kv_len = key_mask = None
    if kind in ("len", "both"):
        kv_len = g.integers(0, M + 1, size=B)
        kv_len[0] = max(1, M - 1)
        if B > 1:
            kv_len[1] = 0
    if kind in ("mask", "both"):
        key_mask = g.random((B, M)) > 0.3
        key_mask[-1, : M // 2] = False
    return kv_len, key_mask


def run_cross(bsa, B, N, H, Hkv, M, d, kind, seed=0, grad=True, scale=1.0):
    q, do = rand((B, N, H, d), seed + 1, scale=scale), rand((B, N, H, d), seed + 2)
    k, v = rand((B, M, Hkv, d), seed + 3), rand((B, M, Hkv, d), seed + 4)
    kv_len, key_mask = masks_of(kind, B, M, seed)
    on = ob.valid_states(B, M, kv_len, key_mask)
    kw = dict(kv_len=None if kv_len is None else torch.from_numpy(kv_len.astype(np.int32)).cuda(),
              key_mask=None if key_mask is None else torch.from_numpy(key_mask).cuda())
    plan = plan_of(bsa, B, N, H, d)
    o, lse = bsa.cross_attn(plan, q, k, v, return_lse=True, **kw)
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
    check_cross(o, lse, q, k, v, on)
    if grad:
        grads = bsa.cross_attn_backward(plan, do, q, k, v, o, lse, **kw)
        assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK
        check_cross_grad(grads, q, k, v, on, do)
    return plan, (q, k, v, do), kw, (o, lse)


def check_cross(o, lse, q, k, v, on):
    want, wlse, absv, size = ob.cross_attention(f64(q), f64(k), f64(v), on)
    within(o, want, ob.cross_bound(want, absv, size, q.shape[3]), "o")
    got = f64(lse)
    empty = np.isneginf(wlse)
    assert np.array_equal(np.isneginf(got), empty)
    # the scores' error, the row sum's (2^-14 an exponential) and the logarithm's and sum's roundings
    bound = (q.shape[3] + 3) * ob.U32 * size + 2.0 ** -14 + 4 * ob.U32 * np.abs(np.where(empty, 0, wlse)) + 8 * ob.U32
    within(np.where(empty, 0, got), np.where(empty, 0, wlse), bound, "lse")


def check_cross_grad(grads, q, k, v, on, do):
    a = [f64(t) for t in (q, k, v)]
    want, _, absv, size = ob.cross_attention(*a, on)
    o_bound = ob.cross_bound(want, absv, size, q.shape[3])
    *wants, info = ob.cross_attention_grad(*a, on, f64(do))
    bounds = ob.cross_grad_bounds(a[0], f64(do), o_bound, info, k.shape[2])
    for got, w, b, n in zip(grads, wants, bounds, ("dq", "dk", "dv")):
        within(got, w, b, n)


@pytest.mark.parametrize("kind", ["all", "len", "mask", "both"])
@pytest.mark.parametrize("shape", SHAPES)
def test_cross_attention_and_gradient(bsa, shape, kind):
    run_cross(bsa, *shape, kind)


@pytest.mark.parametrize("M", [2, 3, 17, 64])
def test_cross_gradient_of_few_states_keeps_its_digits(bsa, M):
    """Sharp rows over few states: dS is a small difference, and D from the rounded o would cost a third of a bf16 step
    of the whole.  P and dS are rounded once (2^-8 at most, a third of that as a root mean square) and the result once,
    so the 2-norm of the error stays below 2^-8 of the result's."""
    B, N, H, d = 2, 260, 3, 128
    plan, (q, k, v, do), kw, (o, lse) = run_cross(bsa, B, N, H, H, M, d, "all", seed=3 + M, grad=False, scale=4.0)
    grads = bsa.cross_attn_backward(plan, do, q, k, v, o, lse)
    wants = ob.cross_attention_grad(f64(q), f64(k), f64(v), ob.valid_states(B, M), f64(do))[:3]
    for got, want, name in zip(grads, wants, ("dq", "dk", "dv")):
        assert np.linalg.norm(f64(got) - want) <= ob.U16 * np.linalg.norm(want), name


@pytest.mark.parametrize("scale", [0.01, 8.0])
def test_cross_attention_flat_and_sharp_scores(bsa, scale):
    run_cross(bsa, 1, 150, 2, 2, 300, 128, "all", seed=9, scale=scale)


def test_cross_attention_rising_scores(bsa):
    """Each key block's largest score is far above the last block's: the running maximum moves every time."""
    B, N, H, M, d = 1, 140, 2, 640, 64
    q = torch.ones(B, N, H, d, dtype=torch.bfloat16).cuda()
    k = (torch.arange(M).float() / 16 - 20).to(torch.bfloat16).view(1, M, 1, 1).expand(B, M, H, d).contiguous().cuda()
    v = rand((B, M, H, d), 5)
    plan = plan_of(bsa, B, N, H, d)
    for kk in (k, k.flip(1).contiguous()):
        o, lse = bsa.cross_attn(plan, q, kk, v, return_lse=True)
        check_cross(o, lse, q, kk, v, ob.valid_states(B, M))


@pytest.mark.parametrize("N,M", [(1, 40), (3, 200), (150, 40), (150, 300)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), torch.finfo(torch.bfloat16).min])
def test_cross_attention_garbage_behind_the_mask(bsa, bad, N, M):
    B, H, d = 2, 2, 128
    q, k, v, do = rand((B, N, H, d), 1), rand((B, M, H, d), 2), rand((B, M, H, d), 3), rand((B, N, H, d), 4)
    plan = plan_of(bsa, B, N, H, d)
    for kw in (dict(kv_len=torch.tensor([M - 9, 0], dtype=torch.int32).cuda()),
               dict(key_mask=(torch.arange(2 * M).view(2, M) % 3 != 1).cuda())):
        on = ob.valid_states(B, M, *(None if kw.get(n) is None else kw[n].cpu().numpy() for n in ("kv_len", "key_mask")))
        off = torch.from_numpy(~on).cuda()
        k2, v2 = k.clone(), v.clone()
        k2[off], v2[off] = bad, bad
        o, lse = bsa.cross_attn(plan, q, k2, v2, return_lse=True, **kw)
        o1, lse1 = bsa.cross_attn(plan, q, k, v, return_lse=True, **kw)
        assert torch.equal(o, o1) and torch.equal(lse, lse1)
        g2 = bsa.cross_attn_backward(plan, do, q, k2, v2, o, lse, **kw)
        g1 = bsa.cross_attn_backward(plan, do, q, k, v, o, lse, **kw)
        for a, b in zip(g2, g1):
            assert torch.equal(a, b)
        assert not g2[1][off].any() and not g2[2][off].any()
        check_cross_grad(g2, q, k, v, on, do)


def test_cross_attention_without_states(bsa):
    B, N, H, d = 2, 9, 3, 64
    q, do = rand((B, N, H, d), 1), rand((B, N, H, d), 2)
    kv = torch.empty(B, 0, H, d, dtype=torch.bfloat16, device="cuda")
    plan = plan_of(bsa, B, N, H, d)
    o, lse = bsa.cross_attn(plan, q, kv, kv, return_lse=True)
    assert not o.any() and torch.isneginf(lse).all()
    dq, dk, dv = bsa.cross_attn_backward(plan, do, q, kv, kv, o, lse)
    assert not dq.any() and dk.shape == kv.shape and dv.shape == kv.shape


def test_cross_attention_lengths_out_of_range_act_as_the_bound(bsa):
    B, N, H, M, d = 2, 40, 2, 50, 64
    q, k, v = rand((B, N, H, d), 1), rand((B, M, H, d), 2), rand((B, M, H, d), 3)
    plan = plan_of(bsa, B, N, H, d)
    a = bsa.cross_attn(plan, q, k, v, kv_len=torch.tensor([-5, 9999], dtype=torch.int32).cuda())
    b = bsa.cross_attn(plan, q, k, v, kv_len=torch.tensor([0, M], dtype=torch.int32).cuda())
    assert torch.equal(a, b) and not a[0].any()


@pytest.mark.parametrize("N,M", [(1, 90), (200, 150)])
def test_cross_attention_strided_inputs(bsa, N, M):
    """Views into fused projections: q out of [B,N,3,H,d], k and v out of [B,M,2,H,d], k head-major."""
    B, H, d = 2, 3, 64
    qq, kv = rand((B, N, 3, H, d), 1), rand((B, M, 2, H, d), 2)
    kh = rand((B, H, M, d), 3)
    plan = plan_of(bsa, B, N, H, d)
    do = rand((B, N, H, d), 4)
    for q, k, v in ((qq[:, :, 1], kv[:, :, 0], kv[:, :, 1]), (qq[:, :, 2], kh.transpose(1, 2), kv[:, :, 0])):
        o, lse = bsa.cross_attn(plan, q, k, v, return_lse=True)
        o1, lse1 = bsa.cross_attn(plan, q.contiguous(), k.contiguous(), v.contiguous(), return_lse=True)
        assert torch.equal(o, o1) and torch.equal(lse, lse1)
        for a, b in zip(bsa.cross_attn_backward(plan, do, q, k, v, o, lse),
                        bsa.cross_attn_backward(plan, do, q.contiguous(), k.contiguous(), v.contiguous(), o, lse)):
            assert torch.equal(a, b)


def test_cross_attention_refusals_with_a_plan(bsa):
    plan = plan_of(bsa, 2, 40, 4, 64)
    q, k = rand((2, 40, 4, 64), 1), rand((2, 8, 3, 64), 2)
    with pytest.raises(bsa.BsaError) as e:                              # 3 key heads, 4 query heads
        bsa.cross_attn(plan, q, k, k)
    assert e.value.status == bsa.BSA_EINVAL
    k = rand((2, 8, 4, 64), 2)
    with pytest.raises(bsa.BsaError) as e:                              # one state for both batch entries
        bsa.cross_attn(plan, q, k[:1].expand(2, -1, -1, -1), k)
    assert e.value.status == bsa.BSA_EUNSUPPORTED
    with pytest.raises(bsa.BsaError) as e:                              # rows off the 16-byte grid
        bsa.cross_attn(plan, q, rand((2, 8, 4, 68), 3)[..., :64], k)
    assert e.value.status == bsa.BSA_EUNSUPPORTED
    flat = rand((2 * 8 * 4 * 64 + 1,), 4)
    with pytest.raises(bsa.BsaError) as e:
        bsa.cross_attn(plan, q, flat[1:].view(2, 8, 4, 64), k)
    assert e.value.status == bsa.BSA_EINVAL
    o, lse = bsa.cross_attn(plan, q, k, k, return_lse=True)
    with pytest.raises(bsa.BsaError) as e:
        bsa.cross_attn_backward(plan, q, q, k, k, o, lse, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == bsa.BSA_EWORKSPACE


# ------------------------------------------------------------------------ the norms
#
# Row sums are at most 40 roundings deep (16 in a thread, 5 shuffles, 5 more over warps, the products around them), so
# a normalised value is off by at most 40 2^-24 X with X = r (mean|x| + |x|) + |xhat|, r = 1 / deviation, plus what
# x itself is off by.

K = 40 * ob.U32


def xhat_bound(x, xh, r, ex=0.0):
    ex = np.broadcast_to(ex, x.shape)
    X = r * (np.abs(x).mean(axis=-1, keepdims=True) + np.abs(x)) + np.abs(xh)
    return K * X + r * (ex + (1 + np.abs(xh)) * (ex * (1 + np.abs(xh))).mean(axis=-1, keepdims=True)), X


def rows(p, N):
    return 1.0 if p is None else p.repeat(N // p.shape[1], axis=1)


def check_boundary(got_x, got_h, x, t, opt, store):
    t = {k: f64(v) for k, v in t.items()}
    N, eps = x.shape[1], opt["eps"]
    wx, wh = ob.boundary(x, **t, **opt)
    ex = 0.0
    y = t.get("y")
    if y is not None:
        u, eu = y, 0.0
        if opt["post"]:
            u, r = ob.normalise(y, opt["post"], eps)
            eu = xhat_bound(y, u, r)[0]
        f = np.abs((1.0 if t.get("post_weight") is None else t["post_weight"]) * rows(t.get("gate"), N))
        ex = f * eu + 4 * ob.U32 * (f * np.abs(u) + np.abs(opt["res_scale"] * x))
        within(got_x, wx, store * np.abs(wx) + ex + 1e-37, "x_out")
    if opt["norm"] is None:
        assert got_h is None
        return
    xh, r = ob.normalise(wx, opt["norm"], eps)
    w = np.abs((1.0 if t.get("weight") is None else t["weight"])) * np.abs(1 + (0 if t.get("scale") is None else rows(t["scale"], N)))
    b = 0 if t.get("bias") is None else np.abs(t["bias"] * (1 + (0 if t.get("scale") is None else rows(t["scale"], N))))
    s = 0 if t.get("shift") is None else np.abs(rows(t["shift"], N))
    e = w * xhat_bound(wx, xh, r, ex)[0] + 8 * ob.U32 * (np.abs(xh) * w + b + s)
    within(got_h, wh, ob.U16 * np.abs(wh) + e + 1e-37, "h")


def check_boundary_grad(got, x, dh, dxo, t, opt, groups, store):
    t = {k: f64(v) for k, v in t.items()}
    B, N, C = x.shape
    eps = opt["eps"]
    want = ob.boundary_grad(x, dh, dxo, groups=groups, **t, **opt)

    def gsum(v):
        return np.broadcast_to(v, x.shape).reshape(B, groups, N // groups, C).sum(axis=2)

    Kc = (N + 64) * ob.U32                                   # column sums: at most a group's rows deep
    g = np.zeros_like(x) if dxo is None else dxo
    eg = 0.0
    bounds = {}
    if dh is not None:
        xh, r = ob.normalise(x, opt["norm"], eps)
        exh, X = xhat_bound(x, xh, r)
        one = np.abs(1 + (0 if t.get("scale") is None else rows(t["scale"], N)))
        w = 1.0 if t.get("weight") is None else np.abs(t["weight"])
        b = 0.0 if t.get("bias") is None else np.abs(t["bias"])
        ga = np.abs(dh) * one * w
        # three products of values 40 roundings deep, and their row means
        eg = 3 * K * r * (ga + ga.mean(axis=-1, keepdims=True) + X * (ga * X).mean(axis=-1, keepdims=True))
        full = dh * (1 if t.get("scale") is None else 1 + rows(t["scale"], N)) * (1.0 if t.get("weight") is None else t["weight"])
        head = full - xh * (full * xh).mean(axis=-1, keepdims=True)
        g = g + r * (head - head.mean(axis=-1, keepdims=True) if opt["norm"] == "layer" else head)
        eg = eg + 4 * ob.U32 * (np.abs(dxo) if dxo is not None else 0.0)
        bounds["dshift"] = Kc * gsum(np.abs(dh))
        bounds["dscale"] = gsum(np.abs(dh) * (w * (exh + Kc * np.abs(xh)) + Kc * b))
        bounds["dweight"] = ((B * N + 64) * ob.U32 * np.abs(dh * one * xh) + np.abs(dh) * one * exh).sum(axis=(0, 1))
        bounds["dbias"] = (B * N + 64) * ob.U32 * (np.abs(dh) * one).sum(axis=(0, 1))
    rs = 1.0
    if "y" in t:
        y = t["y"]
        yh, ry, eyh, Y = y, None, 0.0, np.abs(y)
        if opt["post"]:
            yh, ry = ob.normalise(y, opt["post"], eps)
            eyh, Y = xhat_bound(y, yh, ry)
        pw = 1.0 if t.get("post_weight") is None else np.abs(t["post_weight"])
        gt = np.abs(rows(t.get("gate"), N))
        bounds["dgate"] = gsum(pw * (np.abs(g) * (eyh + Kc * np.abs(yh)) + eg * np.abs(yh)))
        bounds["dpost_weight"] = (gt * (np.abs(g) * (eyh + (B * N + 64) * ob.U32 * np.abs(yh)) + eg * np.abs(yh))).sum(axis=(0, 1))
        ga, ea = np.abs(g) * gt * pw, eg * gt * pw + 4 * ob.U32 * np.abs(g) * gt * pw
        if opt["post"]:
            def mean(v):
                return np.broadcast_to(v, x.shape).mean(axis=-1, keepdims=True)
            ey = ry * (ea + mean(ea) + np.abs(yh) * mean(ea * np.abs(yh))) \
                + 3 * K * ry * (ga + mean(ga) + Y * mean(ga * Y))
        else:
            ey = ea
        bounds["dy"] = ob.U16 * np.abs(want["dy"]) + ey
        rs = abs(opt["res_scale"])
    bounds["dx"] = store * np.abs(want["dx"]) + rs * eg + 4 * ob.U32 * np.abs(want["dx"])
    names = {"dx"} | ({"dy"} if "y" in t else set()) | {"d" + n for n in t if n != "y" and t[n] is not None}
    for n, v in got._asdict().items():
        assert (v is not None) == (n in names), n
        if v is not None:
            within(v, want[n], bounds[n] * 1.01 + 1e-37, n)


KIND = {None: "BSA_NORM_NONE", "layer": "BSA_NORM_LAYER", "rms": "BSA_NORM_RMS"}


def norm_case(bsa, B, T, S, C, groups, stream, norm, post, params, seed=0, mean=0.0, res_scale=1.0, residual=True):
    """Plan, inputs and options of one case; params: which parameters are given."""
    N = T * S
    dt = torch.bfloat16 if stream == "bf16" else torch.float32
    F = {"batch": 1, "frame": T, "token": N}[groups]
    x = (rand((B, N, C), seed, torch.float32, 2.0) + mean).to(dt)
    t = dict(y=rand((B, N, C), seed + 1)) if residual else {}
    if residual and "gate" in params:
        t["gate"] = rand((B, F, C), seed + 2, torch.float32)
    if residual and "post_weight" in params:
        t["post_weight"] = rand((C,), seed + 3, torch.float32)
    if norm:
        for i, (n, shape) in enumerate(dict(scale=(B, F, C), shift=(B, F, C), weight=(C,), bias=(C,)).items()):
            if n in params:
                t[n] = rand(shape, seed + 4 + i, torch.float32)
    eps = 1e-5
    kw = dict(norm=getattr(bsa, KIND[norm]), eps=eps)
    if residual:
        kw.update(post_norm=getattr(bsa, KIND[post]), res_scale=res_scale)
    opt = dict(norm=norm, post=post, res_scale=res_scale, eps=eps)
    plan = bsa.Plan(B, 1, T, 1, S, 64, 64, bsa.BSA_ORDER_IDENTITY)
    F = F if {"gate", "scale", "shift"} & set(t) else 1
    return plan, x, t, kw, opt, (ob.U16 if stream == "bf16" else ob.U32), F


ALL = ("gate", "post_weight", "scale", "shift", "weight", "bias")
# B, T, tokens a frame, C
SIZES = [(1, 1, 1, 1), (1, 1, 1, 8), (2, 3, 5, 24), (1, 2, 9, 129), (2, 2, 7, 512), (1, 3, 50, 520), (1, 2, 33, 1219),
         (1, 5, 70, 1536), (1, 2, 12, 1856), (1, 1, 9, 2048), (1, 1, 9, 4096), (2, 1, 4, 5120), (1, 2, 3, 6151), (1, 1, 3, 16384), (1, 1, 2, 16383), (1, 1, 700, 72)]


def residual_both(bsa, case, seed=0):
    plan, x, t, kw, opt, store, F = case
    xo, h = bsa.residual_norm(plan, x, **t, **kw)
    check_boundary(xo, h, f64(x), t, opt, store)
    dh = None if opt["norm"] is None else rand(x.shape, seed + 20)
    dxo = rand(x.shape, seed + 21, x.dtype)
    gr = bsa.residual_norm_backward(plan, dh, dxo, xo, **t, **kw)
    check_boundary_grad(gr, f64(xo), f64(dh), f64(dxo), t, opt, F, store)


@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_residual_norm_sizes(bsa, size, stream):
    for groups in ("batch", "frame", "token"):
        residual_both(bsa, norm_case(bsa, *size, groups, stream, "layer", "rms", ALL, res_scale=0.75))


@pytest.mark.parametrize("norm,post", [("layer", None), ("rms", None), ("rms", "rms"), ("rms", "layer"), (None, None),
                                       (None, "layer")])
@pytest.mark.parametrize("params", [(), ("gate",), ("scale", "shift"), ("weight",), ("bias",), ("gate", "scale", "shift"),
                                    ("post_weight", "shift"), ALL])
def test_residual_norm_options(bsa, norm, post, params):
    residual_both(bsa, norm_case(bsa, 2, 3, 11, 200, "frame", "bf16", norm, post, params))
    residual_both(bsa, norm_case(bsa, 1, 2, 5, 1030, "frame", "f32", norm, post, params))


@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_norm_modulate_sizes(bsa, size, stream):
    for norm, groups in (("layer", "batch"), ("rms", "frame"), ("layer", "token")):
        plan, x, t, kw, opt, store, F = norm_case(bsa, *size, groups, stream, norm, None, ALL, residual=False)
        h = bsa.norm_modulate(plan, x, **t, **kw)
        check_boundary(None, h, f64(x), t, opt, store)
        dh = rand(x.shape, 30)
        gr = bsa.norm_modulate_backward(plan, dh, x, **t, **kw)
        check_boundary_grad(gr, f64(x), f64(dh), None, t, opt, F, store)


def test_norm_large_mean(bsa):
    """A mean a thousand times the deviation costs no more than the bound's mean|x| term."""
    plan, x, t, kw, opt, store, F = norm_case(bsa, 1, 1, 20, 1536, "batch", "f32", "layer", None, (), residual=False,
                                              mean=2000.0)
    check_boundary(None, bsa.norm_modulate(plan, x, **kw), f64(x), t, opt, store)


def test_norm_constant_and_zero_rows(bsa):
    plan, x, t, kw, opt, store, F = norm_case(bsa, 1, 1, 4, 96, "batch", "f32", "layer", None, ("shift",), residual=False)
    x[0, 0], x[0, 1] = 0.0, 5.0
    h = bsa.norm_modulate(plan, x, **t, **kw)
    check_boundary(None, h, f64(x), t, opt, store)
    assert torch.equal(h[0, 0], t["shift"][0, 0].bfloat16()) and torch.equal(h[0, 1], h[0, 0])


def test_residual_norm_backward_partial_inputs(bsa):
    plan, x, t, kw, opt, store, F = norm_case(bsa, 1, 2, 20, 136, "frame", "bf16", "layer", "rms", ALL)
    xo, _ = bsa.residual_norm(plan, x, **t, **kw)
    dh = rand(x.shape, 3)
    gr = bsa.residual_norm_backward(plan, dh, None, xo, **t, **kw)
    check_boundary_grad(gr, f64(xo), f64(dh), None, t, opt, F, store)


@pytest.mark.parametrize("C", [200, 1219, 1536])
def test_residual_norm_in_place(bsa, C):
    plan, x, t, kw, opt, store, F = norm_case(bsa, 1, 2, 40, C, "frame", "f32", "layer", "rms", ALL)
    xo, h = bsa.residual_norm(plan, x, **t, **kw)
    x2, y2 = x.clone(), t["y"].clone()
    a, b = bsa.residual_norm(plan, x2, **{**t, "y": y2}, **kw, x_out=x2, h_out=y2)
    assert a is x2 and b is y2 and torch.equal(x2, xo) and torch.equal(y2, h)


def test_norm_refusals_with_a_plan(bsa):
    plan, x, t, kw, opt, store, F = norm_case(bsa, 1, 2, 5, 64, "frame", "f32", "layer", None, ALL)
    y = t["y"]
    for call in (lambda: bsa.norm_modulate(plan, x, norm=7), lambda: bsa.norm_modulate(plan, x, eps=0.0),
                 lambda: bsa.norm_modulate(plan, x, norm=bsa.BSA_NORM_NONE),
                 lambda: bsa.norm_modulate(plan, x, scale=rand((1, 3, 64), 1, torch.float32)),          # 3 groups, 10 tokens
                 lambda: bsa.residual_norm_backward(plan, None, x, x, y),                                # dh is due
                 lambda: bsa.residual_norm_backward(plan, None, None, x, y, norm=bsa.BSA_NORM_NONE)):
        with pytest.raises(bsa.BsaError) as e:
            call()
        assert e.value.status == bsa.BSA_EINVAL
    with pytest.raises(bsa.BsaError) as e:
        bsa.norm_modulate(plan, rand((1, 10, 16385), 1))
    assert e.value.status == bsa.BSA_EUNSUPPORTED
    with pytest.raises(bsa.BsaError) as e:
        bsa.norm_modulate_backward(plan, y, x, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == bsa.BSA_EWORKSPACE


@pytest.mark.parametrize("M,kind", [(13, "mask"), (64, "all"), (1, "all"), (100, "len")])
def test_many_items_of_few_states(bsa, M, kind):
    """Several items to every SM, each with one or two key tiles: what an item leaves for the output warps (its rows'
    sums and maxima) stays until they have read it, however far the softmax warps run ahead."""
    B, N, H, Hkv, d = 2, 6216, 9, 3, 128
    sharp = torch.logspace(-2, 1, H, base=2).to(torch.bfloat16).cuda().view(1, 1, H, 1)
    q, do = rand((B, N, H, d), 71) * sharp, rand((B, N, H, d), 72)
    k, v = rand((B, M, Hkv, d), 73), rand((B, M, Hkv, d), 74)
    kv_len, key_mask = masks_of(kind, B, M, 5)
    on = ob.valid_states(B, M, kv_len, key_mask)
    kw = dict(kv_len=None if kv_len is None else torch.from_numpy(kv_len.astype(np.int32)).cuda(),
              key_mask=None if key_mask is None else torch.from_numpy(key_mask).cuda())
    plan = plan_of(bsa, B, N, H, d)
    o, lse = bsa.cross_attn(plan, q, k, v, return_lse=True, **kw)
    check_cross(o, lse, q, k, v, on)
    grads = bsa.cross_attn_backward(plan, do, q, k, v, o, lse, **kw)
    for _ in range(20):
        o2, lse2 = bsa.cross_attn(plan, q, k, v, return_lse=True, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for a, b in zip(grads, bsa.cross_attn_backward(plan, do, q, k, v, o, lse, **kw)):
            assert torch.equal(a, b)
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK


@pytest.mark.parametrize("which", ["dgate", "dscale", "dshift", "dweight", "dbias", "dpost_weight"])
@pytest.mark.parametrize("off", [4, 8])
def test_norm_gradients_refuse_outputs_off_the_16_byte_grid(bsa, which, off):
    """The C call takes any device pointers: what 16-byte stores could not write is refused before the launch."""
    import ctypes
    plan, x, t, kw, opt, store, F = norm_case(bsa, 1, 2, 5, 64, "token", "f32", "layer", None, ALL)
    lib, y = bsa._lib, t["y"]
    names = ["dgate", "dscale", "dshift", "dweight", "dbias", "dpost_weight"]
    out = {n: torch.empty(10 * 64 + 4, device="cuda") for n in names}
    ptr = {n: o.data_ptr() + (off if n == which else 0) for n, o in out.items()}
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    dx, dy = torch.empty_like(x), torch.empty_like(y)
    a = bsa.NormArgs(64, 10, bsa.BSA_F32, bsa.BSA_NORM_LAYER, bsa.BSA_NORM_NONE, 1e-6, 1.0)
    rc = lib.bsa_residual_norm_bwd(plan.handle, ctypes.byref(a), y.data_ptr(), x.data_ptr(), x.data_ptr(), y.data_ptr(),
                                   dx.data_ptr(), dy.data_ptr(), *(ptr[n] for n in names), ws.data_ptr(), ws.numel(), 0)
    assert rc == bsa.BSA_EINVAL
    if which in names[1:5]:
        rc = lib.bsa_norm_modulate_bwd(plan.handle, ctypes.byref(a), y.data_ptr(), x.data_ptr(), dx.data_ptr(),
                                       *(ptr[n] for n in names[1:5]), ws.data_ptr(), ws.numel(), 0)
        assert rc == bsa.BSA_EINVAL


# -------------------------------------------------------- streams, graphs, a whole block

def test_gradients_are_the_same_every_time(bsa):
    plan, (q, k, v, do), kw, (o, lse) = run_cross(bsa, 2, 300, 4, 2, 200, 64, "mask", grad=False)
    first = bsa.cross_attn_backward(plan, do, q, k, v, o, lse, **kw)
    plan2, x, t, kw2, opt, store, F = norm_case(bsa, 2, 2, 400, 520, "frame", "bf16", "layer", "rms", ALL)
    n1 = bsa.residual_norm_backward(plan2, t["y"], x, x, **t, **kw2)
    for _ in range(3):
        for a, b in zip(first, bsa.cross_attn_backward(plan, do, q, k, v, o, lse, **kw)):
            assert torch.equal(a, b)
        for a, b in zip(n1, bsa.residual_norm_backward(plan2, t["y"], x, x, **t, **kw2)):
            assert torch.equal(a, b)


def test_two_streams_at_once(bsa):
    """Two plans on two streams, many calls in flight, the same results as one after the other."""
    jobs = []
    for i in range(2):
        plan, (q, k, v, do), kw, (o, lse) = run_cross(bsa, 1, 500 + i, 4, 4, 300, 128, "len", seed=i, grad=False)
        g = bsa.cross_attn_backward(plan, do, q, k, v, o, lse, **kw)
        jobs.append((plan, q, k, v, do, kw, o, lse, g, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for plan, q, k, v, do, kw, o, lse, g, s in jobs:
            o2, l2 = bsa.cross_attn(plan, q, k, v, return_lse=True, stream=s, **kw)
            outs.append((o2, l2, *bsa.cross_attn_backward(plan, do, q, k, v, o2, l2, stream=s, **kw)))
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        _, _, _, _, _, _, o, lse, g, _ = jobs[i % 2]
        for a, b in zip(got, (o, lse, *g)):
            assert torch.equal(a, b)


def test_captured_and_replayed(bsa):
    """Two graphs that share one workspace, replayed in turn on new inputs."""
    B, N, H, M, d, C = 1, 200, 2, 150, 64, 128
    plan = plan_of(bsa, B, N, H, d)
    q, k, v, do = (rand((B, n, H, d), i) for i, n in enumerate((N, M, M, N)))
    x, y = rand((B, N, C), 7), rand((B, N, C), 8)
    gate = rand((B, 1, C), 9, torch.float32)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")

    def step():
        o, lse = bsa.cross_attn(plan, q, k, v, return_lse=True, workspace=ws)
        grads = bsa.cross_attn_backward(plan, do, q, k, v, o, lse, workspace=ws)
        xo, h = bsa.residual_norm(plan, x, y, gate=gate)
        return (o, *grads, xo, h, *(t for t in bsa.residual_norm_backward(plan, h, xo, xo, y, gate=gate, workspace=ws)
                                    if t is not None))

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for seed in (31, 32):
        for t in (q, k, v, do, x, y):
            t.copy_(rand(t.shape, seed + t.numel() % 97))
        for g, out in graphs:
            for t in out:
                t.fill_(float("nan"))
            g.replay()
        want = step()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("block", [64, 128])
def test_dit_block_against_the_oracle(bsa, block):
    """A whole block at p = 1 (dense self-attention): the path as a host model calls it."""
    B, H, d, T, Hs, Ws, M, Hkv = 2, 2, 64, 2, 9, 11, 23, 1
    N, C = T * Hs * Ws, H * d
    plan = bsa.Plan(B, H, T, Hs, Ws, d, block)
    x = rand((B, N, C), 1, torch.float32)
    mod = [rand((B, T, C), 2 + i, torch.float32, 0.3) for i in range(6)]
    w = [rand((C, C), 10 + i, scale=C ** -0.5) for i in range(7)]
    kc, vc = rand((B, M, Hkv, d), 20), rand((B, M, Hkv, d), 21)
    kv_len = torch.tensor([M, 5], dtype=torch.int32).cuda()
    cw, cb = rand((C,), 22, torch.float32), rand((C,), 23, torch.float32)

    def heads(t):
        return t.view(B, N, H, d)

    got = bsa.dit_block(plan, x, mod, qkv=lambda h: tuple(heads(h @ w[i]) for i in range(3)),
                        attn_out=lambda o: o.reshape(B, N, C) @ w[3], cross_q=lambda h: heads(h @ w[4]),
                        cross_out=lambda o: o.reshape(B, N, C) @ w[5], ffn=lambda h: h @ w[6], k_ctx=kc, v_ctx=vc,
                        p=1.0, k_floor=1, kv_len=kv_len, cross_weight=cw, cross_bias=cb)
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK and got.dtype == x.dtype
    W, m = [f64(t) for t in w], [f64(t) for t in mod]
    on = ob.valid_states(B, M, kv_len.cpu().numpy())
    xs = f64(x)
    h = ob.boundary(xs, scale=m[1], shift=m[0], norm="layer")[1]
    q, k, v = (heads(torch.from_numpy(h @ W[i])).numpy() for i in range(3))
    a = ob.cross_attention(q, k, v, ob.valid_states(B, N))[0].reshape(B, N, C)
    xs, h = ob.boundary(xs, y=a @ W[3], gate=m[2], weight=f64(cw), bias=f64(cb), norm="layer")
    c = ob.cross_attention(heads(torch.from_numpy(h @ W[4])).numpy(), f64(kc), f64(vc), on)[0].reshape(B, N, C)
    xs, h = ob.boundary(xs, y=c @ W[5], scale=m[4], shift=m[3], norm="layer")
    want = ob.boundary(xs, y=h @ W[6], gate=m[5], norm=None)[0]
    err = np.abs(f64(got) - want)
    # a chain of about ten bf16 roundings (2^-8 each) of values of size one: 3 standard deviations of their random
    # sum on average, and a worst element a few times that
    assert err.mean() <= 10 ** 0.5 * 3 * ob.U16 * np.abs(want).mean() and err.max() <= 0.25, (err.mean(), err.max())
