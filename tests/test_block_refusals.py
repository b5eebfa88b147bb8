"""Argument checks of the block operators that need no GPU: the C calls' null and range checks, and the binding's
type, shape, layout and device checks (on CPU tensors, with a stand-in for the plan)."""
import contextlib
import ctypes
import types
import warnings

import pytest
import torch


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_top_b200 import build
    build.build()
    import block_sparse_attention_top_b200 as m
    return m


def test_c_calls_refuse_a_null_plan(bsa):
    lib, na = bsa._lib, bsa.NormArgs(C=8, groups=1, dtype=0, norm=1, post_norm=0, eps=1e-6, res_scale=1.0)
    n = [None]
    assert lib.bsa_cross_attn(*n * 4, 4, 1, *n * 6, 0, None) == bsa.BSA_EINVAL
    assert lib.bsa_cross_attn_bwd(*n * 4, 4, 1, *n * 10, 0, None) == bsa.BSA_EINVAL
    assert lib.bsa_cross_attn_workspace_size(None, 4, 1, 1) == 0
    ref = ctypes.byref(na)
    assert lib.bsa_norm_modulate(None, ref, *n * 3) == bsa.BSA_EINVAL
    assert lib.bsa_residual_norm(None, ref, *n * 5) == bsa.BSA_EINVAL
    assert lib.bsa_norm_modulate_bwd(None, ref, *n * 8, 0, None) == bsa.BSA_EINVAL
    assert lib.bsa_residual_norm_bwd(None, ref, *n * 13, 0, None) == bsa.BSA_EINVAL
    assert lib.bsa_norm_bwd_workspace_size(None, ref) == 0


PLAN = types.SimpleNamespace(B=2, N=6, H=4, d=64, device=torch.device("cpu"), handle=None)


def _qkv(**over):
    t = dict(q=torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16), k=torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16),
             v=torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16))
    t.update(over)
    return t


BAD_CROSS = [
    dict(q=torch.zeros(2, 6, 4, 64)),                                              # type
    dict(q=torch.zeros(2, 7, 4, 64, dtype=torch.bfloat16)),                        # tokens
    dict(k=torch.zeros(2, 5, 128, dtype=torch.bfloat16)),                          # rank
    dict(v=torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)),                        # k and v differ
    dict(k=torch.zeros(2, 5, 64, 2, dtype=torch.bfloat16).transpose(2, 3)),        # channels not contiguous
    dict(kv_len=torch.zeros(2, dtype=torch.int64)),
    dict(kv_len=torch.zeros(3, dtype=torch.int32)),
    dict(key_mask=torch.zeros(2, 5)),
    dict(key_mask=torch.zeros(2, 10, dtype=torch.bool)[:, ::2]),
    dict(q=torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16, device="meta")),         # device
    dict(q=None),
]


@pytest.mark.parametrize("over", BAD_CROSS)
def test_cross_attention_refuses(bsa, over):
    with pytest.raises(ValueError):
        bsa.cross_attn(PLAN, **_qkv(**over))
    with pytest.raises(ValueError):
        bsa.cross_attn_backward(PLAN, do=torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16),
                                o=torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16), lse=torch.zeros(2, 4, 6), **_qkv(**over))


@pytest.mark.parametrize("name,bad", [("do", torch.zeros(2, 6, 4, 64)), ("lse", torch.zeros(2, 6, 4)),
                                      ("o", torch.zeros(2, 6, 4, 128, dtype=torch.bfloat16)[..., ::2])])
def test_cross_backward_refuses(bsa, name, bad):
    t = dict(do=torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16), o=torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16),
             lse=torch.zeros(2, 4, 6))
    t[name] = bad
    with pytest.raises(ValueError):
        bsa.cross_attn_backward(PLAN, **t, **_qkv())


X, Y = torch.zeros(2, 6, 24), torch.zeros(2, 6, 24, dtype=torch.bfloat16)
BAD_NORM = [
    dict(x=torch.zeros(2, 6, 24, dtype=torch.float16)), dict(x=torch.zeros(12, 24)), dict(x=torch.zeros(2, 6, 48)[..., ::2]),
    dict(scale=torch.zeros(2, 1, 24, dtype=torch.bfloat16)), dict(scale=torch.zeros(2, 24)),
    dict(scale=torch.zeros(2, 2, 24), shift=torch.zeros(2, 3, 24)), dict(scale=torch.zeros(2, 2, 24), shift=torch.zeros(2, 1, 24)),
    dict(scale=torch.zeros(1, 1, 24).expand(2, 1, 24)), dict(weight=torch.zeros(25)), dict(bias=torch.zeros(24, dtype=torch.float64)),
]


@pytest.mark.parametrize("over", BAD_NORM)
def test_norms_refuse(bsa, over):
    x = over.get("x", X)
    par = {k: v for k, v in over.items() if k != "x"}
    with pytest.raises(ValueError):
        bsa.norm_modulate(PLAN, x, **par)
    with pytest.raises(ValueError):
        bsa.norm_modulate_backward(PLAN, Y, x, **par)
    with pytest.raises(ValueError):
        bsa.residual_norm(PLAN, x, Y, **par)
    with pytest.raises(ValueError):
        bsa.residual_norm_backward(PLAN, Y, None, x, Y, **par)


def test_residual_refuses_branch_and_outputs(bsa):
    with pytest.raises(ValueError):
        bsa.residual_norm(PLAN, X, X)                                  # y is bf16
    with pytest.raises(ValueError):
        bsa.residual_norm(PLAN, X, Y, x_out=Y)
    with pytest.raises(ValueError):
        bsa.residual_norm(PLAN, X, Y, h_out=X)
    with pytest.raises(ValueError):
        bsa.residual_norm_backward(PLAN, Y, Y, X, Y)                   # dx_out has x's type


@pytest.mark.parametrize("bad", [torch.zeros(2, 6, 4, 64), torch.zeros(2, 7, 4, 64, dtype=torch.bfloat16),
                                 torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16, device="meta"), None])
@pytest.mark.parametrize("which", range(3))
def test_dit_block_refuses_what_qkv_returns(bsa, monkeypatch, which, bad):
    """The self-attention's calls take what they get; dit_block checks it first."""
    good = torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(bsa, "_On", lambda plan, stream: contextlib.nullcontext())
    monkeypatch.setattr(bsa, "norm_modulate", lambda *a, **k: Y)
    monkeypatch.setattr(bsa, "route", lambda *a, **k: pytest.fail("called"))
    with pytest.raises(ValueError):
        bsa.dit_block(PLAN, X, [None] * 6, qkv=lambda h: [bad if i == which else good for i in range(3)], attn_out=None,
                      cross_q=None, cross_out=None, ffn=None, k_ctx=None, v_ctx=None, p=1.0, k_floor=1)


def test_dit_block_runs_on_the_plan_s_device(bsa, monkeypatch):
    """route and sparse_attn launch on the current device: the block makes that the plan's, around every call."""
    inside, calls = [], []

    class On:
        def __init__(self, plan, stream):
            assert plan is PLAN and stream is None

        def __enter__(self):
            inside.append(True)

        def __exit__(self, *exc):
            inside.pop()

    def record(name, value):
        def call(*a, **k):
            assert inside, name
            calls.append(name)
            return value
        return call

    q = torch.zeros(2, 6, 4, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(bsa, "_On", On)
    for name, value in dict(norm_modulate=Y, route=(None,) * 4, sparse_attn=q, cross_attn=q, residual_norm=(X, Y)).items():
        monkeypatch.setattr(bsa, name, record(name, value))
    out = bsa.dit_block(PLAN, X, [None] * 6, qkv=record("qkv", (q, q, q)), attn_out=record("attn_out", Y),
                        cross_q=record("cross_q", q), cross_out=record("cross_out", Y), ffn=record("ffn", Y), k_ctx=q,
                        v_ctx=q, p=1.0, k_floor=1)
    assert out is X and not inside
    assert calls == ["norm_modulate", "qkv", "route", "sparse_attn", "attn_out", "residual_norm", "cross_q", "cross_attn",
                     "cross_out", "residual_norm", "ffn", "residual_norm"]


class Reached(Exception):
    """The checks are over: the call would launch."""


CALLS = [
    ("cross_attn", _qkv(), ()), ("norm_modulate", dict(x=X), ("scale", "shift", "weight", "bias")),
    ("residual_norm", dict(x=X, y=Y), ("gate", "scale", "shift", "weight", "bias", "post_weight")),
]


@pytest.mark.parametrize("name,inputs,params", CALLS)
def test_a_lost_gradient_is_said(bsa, monkeypatch, name, inputs, params):
    def on(plan, stream):
        raise Reached

    def call(**over):
        with pytest.raises(Reached):
            getattr(bsa, name)(PLAN, **{**inputs, **over})

    monkeypatch.setattr(bsa, "_On", on)
    given = {**inputs, **{n: torch.zeros(*((24,) if "weight" in n or n == "bias" else (2, 1, 24))) for n in params}}
    for which, t in given.items():
        t = t.clone().requires_grad_()
        with pytest.warns(UserWarning, match=f"{name}_backward"):
            call(**{which: t})
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            call(**{which: t.detach()})
            with torch.no_grad():
                call(**{which: t})
