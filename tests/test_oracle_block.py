"""Pins of oracle/block.py: torch's float64 attention and differentiation, finite differences, and hand cases."""
import numpy as np
import pytest
import torch

from oracle import block as ob


def _case(seed=0, B=2, N=5, M=7, H=4, Hkv=2, d=6):
    g = np.random.default_rng(seed)
    q, k, v, do = (g.standard_normal(s) for s in ((B, N, H, d), (B, M, Hkv, d), (B, M, Hkv, d), (B, N, H, d)))
    on = ob.valid_states(B, M, kv_len=[M, 4], key_mask=g.random((B, M)) > 0.2)
    on[:, 0] = True
    return q, k, v, do, on


def _torch_attention(q, k, v, on):
    G = q.shape[2] // k.shape[2]
    t = [x.permute(0, 2, 1, 3) for x in (q, k.repeat_interleave(G, 2), v.repeat_interleave(G, 2))]
    o = torch.nn.functional.scaled_dot_product_attention(*t, attn_mask=torch.from_numpy(on)[:, None, None, :])
    return o.permute(0, 2, 1, 3)


def test_cross_attention_matches_torch_and_its_gradient():
    q, k, v, do, on = _case()
    tq, tk, tv = (torch.from_numpy(x).requires_grad_(True) for x in (q, k, v))
    to = _torch_attention(tq, tk, tv, on)
    o, lse, _, _ = ob.cross_attention(q, k, v, on)
    assert np.allclose(o, to.detach().numpy(), atol=1e-13)
    to.backward(torch.from_numpy(do))
    for got, t in zip(ob.cross_attention_grad(q, k, v, on, do)[:3], (tq, tk, tv)):
        assert np.allclose(got, t.grad.numpy(), atol=1e-12)
    s = np.einsum("nd,jd->nj", q[0, :, 0], k[0, :, 0]) / np.sqrt(q.shape[3])
    assert np.allclose(lse[0, 0], np.log(np.exp(s[:, on[0]]).sum(axis=1)))


def test_cross_attention_empty_rows_and_garbage_behind_the_mask():
    q, k, v, do, on = _case(1)
    on[1] = False
    k2, v2 = k.copy(), v.copy()
    k2[~on], v2[~on] = np.nan, np.inf
    o, lse, _, _ = ob.cross_attention(q, k2, v2, on)
    assert np.array_equal(o, ob.cross_attention(q, k, v, on)[0]) and not o[1].any() and np.all(lse[1] == -np.inf)
    dq, dk, dv, _ = ob.cross_attention_grad(q, k2, v2, on, do)
    assert not dq[1].any() and not dk[~on].any() and not dv[~on].any() and np.isfinite(dq).all()


def test_cross_gradient_by_differences():
    q, k, v, do, on = _case(2)
    grads = ob.cross_attention_grad(q, k, v, on, do)[:3]
    g = np.random.default_rng(3)
    for which, x in enumerate((q, k, v)):
        step = g.standard_normal(x.shape)
        args = [[q, k, v], [q, k, v]]
        args[0][which], args[1][which] = x + 1e-5 * step, x - 1e-5 * step
        hi, lo = (float((ob.cross_attention(*a, on)[0] * do).sum()) for a in args)
        assert (hi - lo) / 2e-5 == pytest.approx(float((grads[which] * step).sum()), rel=1e-6, abs=1e-7)


KINDS = [("layer", None), ("rms", None), ("layer", "rms"), ("rms", "layer"), (None, "rms"), (None, None)]


def _boundary_case(norm, post, groups, seed=0, B=2, N=6, C=9):
    g = np.random.default_rng(seed)
    t = dict(y=g.standard_normal((B, N, C)), gate=g.standard_normal((B, groups, C)), post_weight=g.standard_normal(C))
    if norm:
        t.update(scale=g.standard_normal((B, groups, C)), shift=g.standard_normal((B, groups, C)),
                 weight=g.standard_normal(C), bias=g.standard_normal(C))
    return 2 * g.standard_normal((B, N, C)) + 1, t, g


@pytest.mark.parametrize("norm,post", KINDS)
@pytest.mark.parametrize("groups", [1, 3, 6])
def test_boundary_gradient_by_differences(norm, post, groups):
    x, t, g = _boundary_case(norm, post, groups)
    opt = dict(norm=norm, post=post, res_scale=0.7)
    xo, h = ob.boundary(x, **t, **opt)
    dxo, dh = g.standard_normal(xo.shape), None if norm is None else g.standard_normal(xo.shape)

    def loss(x, t):
        a, b = ob.boundary(x, **t, **opt)
        return float((a * dxo).sum() + (0 if b is None else (b * dh).sum()))

    got = ob.boundary_grad(xo, dh, dxo, groups=groups, **t, **opt)
    for name, val in dict(x=x, **t).items():
        step = g.standard_normal(val.shape)
        lo, hi = ((x + s * step, t) if name == "x" else (x, {**t, name: val + s * step}) for s in (-1e-5, 1e-5))
        want = (loss(*hi) - loss(*lo)) / 2e-5
        assert float((got["d" + name] * step).sum()) == pytest.approx(want, rel=1e-5, abs=1e-6), name


def test_boundary_closed_forms():
    x = np.arange(24.0).reshape(1, 2, 12)
    _, h = ob.boundary(x, norm="layer", eps=1e-12)
    ln = torch.nn.functional.layer_norm(torch.from_numpy(x), (12,), eps=1e-12).numpy()
    assert np.allclose(h, ln)
    xo, h = ob.boundary(x, y=np.ones_like(x), gate=np.full((1, 2, 12), 3.0), norm=None, res_scale=2.0)
    assert h is None and np.array_equal(xo, 2 * x + 3)
