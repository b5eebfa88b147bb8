"""Workloads of the operators around a video transformer block's self-attention: cross attention to an
encoder's states, and the norms at the block's boundaries fused with modulation, gate and residual.

Each case names one call (or, for training, a forward with its backward).  `run` computes it in plain torch
arithmetic (32 bits, rounded once to the output's type), or, where `own` is true, by the framework's calls;
`exact` is the definition in 64 bits.  Formulas (j a key, c a channel, n a token of group f):

  cross attention   S = q k^T / sqrt(d) over the valid keys, O = softmax(S) v, rows without a valid key are
                    zero; query head h reads key head h // (H / Hkv)
  its gradient      P = softmax(S), dv = P^T do, dS = P (do v^T - rowsum(do O)), dq = dS k / sqrt(d),
                    dk = dS^T q / sqrt(d); shared key heads sum over their query heads
  modulated norm    h = (norm(x) w + b)(1 + scale_f) + shift_f
  block boundary    x' = r x + gate_f (post_norm(y) w_post), then h as above from x'
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # text states of a 720p clip's block: every query token against 512 prompt states
        dict(name="cross_720p", op="cross", B=1, H=40, Hkv=40, d=128, T=21, Hs=45, Ws=80, M=512, keys="all"),
        # image-conditioned 480p clip: 257 states of an image encoder (an odd length)
        dict(name="cross_480p_image", op="cross", B=1, H=12, Hkv=12, d=128, T=21, Hs=30, Ws=52, M=257, keys="all"),
        # guidance in one batch: prompts of different lengths, padded, lengths given
        dict(name="cross_guided_ragged", op="cross", B=2, H=12, Hkv=12, d=128, T=6, Hs=30, Ws=52, M=512, keys="len"),
        # the smallest clip: launch latency counts
        dict(name="cross_tiny", op="cross", B=1, H=2, Hkv=2, d=64, T=4, Hs=16, Ws=16, M=77, keys="all"),
        # one new token of each of four sequences against a clip's states, shared key heads
        dict(name="cross_one_token", op="cross", B=4, H=40, Hkv=8, d=128, T=1, Hs=1, Ws=1, M=32760, keys="len"),
        # a training step of a 480p clip's cross attention
        dict(name="cross_train_480p", op="cross_train", B=1, H=12, Hkv=12, d=128, T=21, Hs=30, Ws=52, M=512, keys="all"),
        # a small ragged training batch: shared key heads, holes in the mask
        dict(name="cross_train_ragged", op="cross_train", B=2, H=12, Hkv=4, d=64, T=3, Hs=17, Ws=29, M=301, keys="mask"),
        # the boundary between two halves of a 720p block: gate and residual, then the next modulated norm
        dict(name="residual_720p", op="residual", B=1, T=21, Hs=45, Ws=80, C=5120, groups="batch", stream="bf16",
             norm="layer", affine=False, post="none", mod=True),
        # 480p with a 32-bit residual stream, one modulation per frame, norms before and after the block
        dict(name="residual_480p_sandwich", op="residual", B=1, T=21, Hs=30, Ws=52, C=1536, groups="frame",
             stream="f32", norm="rms", affine=True, post="rms", mod=True),
        # the first norm of the smallest clip: launch latency counts
        dict(name="modulate_tiny", op="modulate", B=1, T=4, Hs=16, Ws=16, C=128, groups="batch", stream="bf16",
             norm="layer", affine=False, post="none", mod=True),
        # the 720p boundary's backward pass
        dict(name="residual_bwd_720p", op="residual_bwd", B=1, T=21, Hs=45, Ws=80, C=5120, groups="batch",
             stream="bf16", norm="layer", affine=False, post="none", mod=True),
        # backward of an affine modulated norm at an odd width, one modulation per frame, 32-bit stream
        dict(name="modulate_bwd_odd", op="modulate_bwd", B=2, T=3, Hs=17, Ws=29, C=1219, groups="frame",
             stream="f32", norm="layer", affine=True, post="none", mod=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross_token", "cross_train", "residual", "modulate", "residual_bwd",
                     "modulate_bwd"])
    if op.startswith("cross"):
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12, 20])
        H = Hkv * rng.choice([1, 1, 1, 2, 3, 5] if Hkv <= 8 else [1, 1, 2])
        B = rng.randint(1, 4)
        keys = rng.choice(["all", "len", "mask"])
        if op == "cross_token":
            return dict(op="cross", B=B, H=H, Hkv=Hkv, d=d, T=1, Hs=1, Ws=rng.choice([1, 1, 2, 5]),
                        M=_log_int(rng, 1, 40000), keys=keys)
        M = _log_int(rng, 1, 1200)
        # at most a fifth of the largest listed case's pairs, and a bounded number of tokens
        most = 300e6 / (B * H * M)
        hi = max(30.0, min(40000.0, most))
        N = _log_int(rng, 20, hi)
        T = rng.randint(1, 21)
        Ws = rng.randint(1, 52)
        Hs = max(1, N // (T * Ws))
        return dict(op=op, B=B, H=H, Hkv=Hkv, d=d, T=T, Hs=Hs, Ws=Ws, M=M, keys=keys)
    B = rng.randint(1, 3)
    C = _log_int(rng, 48, 6000)
    if rng.random() < 0.5:
        C = max(64, C // 64 * 64)
    T = rng.randint(1, 21)
    Hs, Ws = rng.randint(1, 45), rng.randint(1, 52)
    while B * T * Hs * Ws * C > 120e6:
        T, Hs = max(1, T // 2), max(1, Hs // 2)
    post = rng.choice(["none", "rms", "layer"]) if op.startswith("residual") else "none"
    return dict(op=op, B=B, T=T, Hs=Hs, Ws=Ws, C=C, groups=rng.choice(["batch", "frame", "token"]),
                stream=rng.choice(["bf16", "f32"]), norm=rng.choice(["layer", "rms"]),
                affine=rng.random() < 0.5, post=post, mod=rng.random() < 0.8)


def _tokens(case):
    return case["T"] * case["Hs"] * case["Ws"]


def _groups(case):
    return {"batch": 1, "frame": case["T"], "token": _tokens(case)}[case["groups"]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev = "cuda"

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    st = dict(case=dict(case))
    B, N = case["B"], _tokens(case)
    if case["op"].startswith("cross"):
        H, Hkv, d, M = case["H"], case["Hkv"], case["d"], case["M"]
        # heads of different sharpness: scores have a standard deviation of 1/4 to 4
        s = torch.exp2(4 * uniform(H) - 2).to(torch.bfloat16).view(1, 1, H, 1)
        st["q"] = normal(B, N, H, d, dtype=torch.bfloat16) * s
        st["k"] = normal(B, M, Hkv, d, dtype=torch.bfloat16)
        st["v"] = normal(B, M, Hkv, d, dtype=torch.bfloat16)
        st["kv_len"] = st["key_mask"] = None
        if case["keys"] == "len":            # padded prompts: a third of the length up to all of it
            st["kv_len"] = (M * (1 + 2 * uniform(B)) / 3).ceil().clamp(1, M).to(torch.int32)
        elif case["keys"] == "mask":         # a padded tail and dropped states
            n = (M * (1 + 2 * uniform(B)) / 3).ceil().clamp(1, M)
            st["key_mask"] = (uniform(B, M) > 0.15) & (torch.arange(M, device=dev).view(1, M) < n.view(B, 1))
        if case["op"] == "cross_train":
            st["do"] = normal(B, N, H, d, dtype=torch.bfloat16)
    else:
        C, F = case["C"], _groups(case)
        dt = torch.bfloat16 if case["stream"] == "bf16" else torch.float32
        bwd = case["op"].endswith("_bwd")
        # a residual stream: channels of different size and mean
        st["x"] = (normal(B, N, C, dtype=dt) * (0.5 + 2 * uniform(C)).to(dt) + normal(C).to(dt) * 0.5)
        st["y"] = normal(B, N, C, dtype=torch.bfloat16) if case["op"].startswith("residual") else None
        st["gate"] = normal(B, F, C) * 0.5 if case["op"].startswith("residual") and case["mod"] else None
        st["scale"] = normal(B, F, C) * 0.3 if case["mod"] else None
        st["shift"] = normal(B, F, C) * 0.3 if case["mod"] else None
        st["weight"] = 1 + 0.2 * normal(C) if case["affine"] else None
        st["bias"] = 0.2 * normal(C) if case["affine"] and case["norm"] == "layer" else None
        st["post_weight"] = 1 + 0.2 * normal(C) if case["post"] != "none" else None
        if bwd:
            st["dh"] = normal(B, N, C, dtype=torch.bfloat16)
            st["dx_out"] = normal(B, N, C, dtype=dt) if case["op"] == "residual_bwd" else None
    if own:
        import block_sparse_attention_top_b200 as bsa
        heads = case.get("H", 1)
        st["plan"] = bsa.Plan(B, heads, case["T"], case["Hs"], case["Ws"], case.get("d", 64), 128,
                              bsa.BSA_ORDER_IDENTITY)
    return st


# ------------------------------------------------------------------- the framework's calls

def _run_own(st):
    import block_sparse_attention_top_b200 as bsa
    case, plan = st["case"], st["plan"]
    if case["op"] == "cross":
        return {"o": bsa.cross_attn(plan, st["q"], st["k"], st["v"], kv_len=st["kv_len"], key_mask=st["key_mask"])}
    if case["op"] == "cross_train":
        o, lse = bsa.cross_attn(plan, st["q"], st["k"], st["v"], kv_len=st["kv_len"], key_mask=st["key_mask"],
                                return_lse=True)
        dq, dk, dv = bsa.cross_attn_backward(plan, st["do"], st["q"], st["k"], st["v"], o, lse,
                                             kv_len=st["kv_len"], key_mask=st["key_mask"])
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    norms = {"none": bsa.BSA_NORM_NONE, "layer": bsa.BSA_NORM_LAYER, "rms": bsa.BSA_NORM_RMS}
    norm, post = norms[case["norm"]], norms[case["post"]]
    if case["op"] == "modulate":
        return {"h": bsa.norm_modulate(plan, st["x"], scale=st["scale"], shift=st["shift"], weight=st["weight"],
                                       bias=st["bias"], norm=norm, eps=EPS)}
    if case["op"] == "residual":
        x_out, h = bsa.residual_norm(plan, st["x"], st["y"], gate=st["gate"], scale=st["scale"], shift=st["shift"],
                                     weight=st["weight"], bias=st["bias"], post_weight=st["post_weight"],
                                     norm=norm, post_norm=post, eps=EPS)
        return {"x": x_out, "h": h}
    if case["op"] == "modulate_bwd":
        gr = bsa.norm_modulate_backward(plan, st["dh"], st["x"], scale=st["scale"], shift=st["shift"],
                                        weight=st["weight"], bias=st["bias"], norm=norm, eps=EPS)
    else:                                    # here x is the boundary's output, as the forward pass left it
        gr = bsa.residual_norm_backward(plan, st["dh"], st["dx_out"], st["x"], st["y"], gate=st["gate"],
                                        scale=st["scale"], shift=st["shift"], weight=st["weight"], bias=st["bias"],
                                        post_weight=st["post_weight"], norm=norm, post_norm=post, eps=EPS)
    return {k: v for k, v in gr._asdict().items() if v is not None}


# ------------------------------------------------------------------------- the plain form

def _valid(st):
    """[B, 1, 1, M] truth values of the keys that count, or None where all do."""
    M = st["k"].shape[1]
    if st["kv_len"] is not None:
        return (torch.arange(M, device="cuda").view(1, M) < st["kv_len"].view(-1, 1)).view(-1, 1, 1, M)
    if st["key_mask"] is not None:
        return st["key_mask"].view(-1, 1, 1, M)
    return None


def _cross_plain(st):
    q, k, v = st["q"], st["k"], st["v"]
    B, N, H, d = q.shape
    M, Hkv = k.shape[1], k.shape[2]

    def rows(t):                             # [B, N, H, d] -> [B, Hkv, (H / Hkv) N, d] in 32 bits
        return t.float().permute(0, 2, 1, 3).reshape(B, Hkv, H // Hkv * N, d)

    def back(t, dtype):
        return t.reshape(B, H, N, d).permute(0, 2, 1, 3).to(dtype).contiguous()

    qf, kf, vf = rows(q), k.float().permute(0, 2, 1, 3), v.float().permute(0, 2, 1, 3)
    rd = 1.0 / math.sqrt(d)
    s = torch.matmul(qf, kf.transpose(2, 3)) * rd
    valid = _valid(st)
    if valid is not None:
        s = torch.where(valid, s, -math.inf)
    m = s.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(3, keepdim=True)
    p = p / torch.where(l == 0, 1.0, l)
    o = torch.matmul(p, vf)
    if "do" not in st:
        return {"o": back(o, q.dtype)}
    lse = (m + torch.log(l)).reshape(B, H, N)
    do = rows(st["do"])
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = p * (torch.matmul(do, vf.transpose(2, 3)) - (do * o).sum(3, keepdim=True))
    dq = torch.matmul(ds, kf) * rd
    dk = torch.matmul(ds.transpose(2, 3), qf) * rd

    def key_side(t):
        return t.permute(0, 2, 1, 3).to(k.dtype).contiguous()

    return {"o": back(o, q.dtype), "lse": lse, "dq": back(dq, q.dtype), "dk": key_side(dk), "dv": key_side(dv)}


def _spread(p, N):
    """[B, F, C] group parameters as [B, N, C] rows (a view where one group covers the batch entry)."""
    B, F, C = p.shape
    return p.unsqueeze(2).expand(B, F, N // F, C).reshape(B, N, C) if F > 1 else p


def _norm(x, kind):
    """(normalised rows, 1 / deviation) in the input's precision."""
    if kind == "layer":
        x = x - x.mean(2, keepdim=True)
    r = torch.rsqrt((x * x).mean(2, keepdim=True) + EPS)
    return x * r, r


def _affine(st, xh, dtype):
    u = xh
    if st["weight"] is not None:
        u = u * st["weight"].to(dtype)
    if st["bias"] is not None:
        u = u + st["bias"].to(dtype)
    return u


def _modulated(st, xh, N, dtype):
    u = _affine(st, xh, dtype)
    if st["scale"] is not None:
        u = u * (1 + _spread(st["scale"].to(dtype), N))
    if st["shift"] is not None:
        u = u + _spread(st["shift"].to(dtype), N)
    return u


def _norm_grad(g, xh, r, kind):
    """Gradient through the normalisation: r (g - xh mean(g xh) [- mean(g)])."""
    t = g - xh * (g * xh).mean(2, keepdim=True)
    return r * (t - g.mean(2, keepdim=True) if kind == "layer" else t)


def _group_sum(t, F):
    B, N, C = t.shape
    return t.view(B, F, N // F, C).sum(2)


def _boundary(st, dtype, out_types):
    case = st["case"]
    x = st["x"].to(dtype)
    B, N, C = x.shape
    F = _groups(case)
    if not case["op"].endswith("_bwd"):
        out = {}
        if st["y"] is not None:
            u = st["y"].to(dtype)
            if case["post"] != "none":
                u = _norm(u, case["post"])[0] * st["post_weight"].to(dtype)
            x = x + (u * _spread(st["gate"].to(dtype), N) if st["gate"] is not None else u)
            out["x"] = x.to(st["x"].dtype if out_types else dtype)
        out["h"] = _modulated(st, _norm(x, case["norm"])[0], N, dtype).to(torch.bfloat16 if out_types else dtype)
        return out
    dh = st["dh"].to(dtype)
    xh, r = _norm(x, case["norm"])
    out = {}
    a, s = _group_sum(dh * xh, F), _group_sum(dh, F)          # both [B, F, C]
    one = 1 + st["scale"].to(dtype) if st["scale"] is not None else torch.ones((), dtype=dtype, device="cuda")
    w = st["weight"].to(dtype) if st["weight"] is not None else None
    if st["scale"] is not None:
        out["dscale"] = a if w is None else a * w
        if st["bias"] is not None:
            out["dscale"] = out["dscale"] + s * st["bias"].to(dtype)
    if st["shift"] is not None:
        out["dshift"] = s
    if w is not None:
        out["dweight"] = (a * one).sum((0, 1))
    if st["bias"] is not None:
        out["dbias"] = (s * one).sum((0, 1))
    g = dh if w is None else dh * w
    if st["scale"] is not None:
        g = g * _spread(one, N)
    dx = _norm_grad(g, xh, r, case["norm"])
    if st["y"] is not None:
        dx = dx + st["dx_out"].to(dtype)
        y = st["y"].to(dtype)
        yh, ry = _norm(y, case["post"]) if case["post"] != "none" else (y, None)
        pw = st["post_weight"].to(dtype) if st["post_weight"] is not None else None
        t = _group_sum(dx * yh, F)
        if st["gate"] is not None:
            out["dgate"] = t if pw is None else t * pw
        if pw is not None:
            out["dpost_weight"] = (t * st["gate"].to(dtype) if st["gate"] is not None else t).sum((0, 1))
        gy = dx * _spread(st["gate"].to(dtype), N) if st["gate"] is not None else dx
        if pw is not None:
            gy = _norm_grad(gy * pw, yh, ry, case["post"])
        out["dy"] = gy.to(torch.bfloat16 if out_types else dtype)
    out["dx"] = dx.to(st["x"].dtype if out_types else dtype)
    return out


def run(st):
    if own:
        return _run_own(st)
    if st["case"]["op"].startswith("cross"):
        return _cross_plain(st)
    return _boundary(st, torch.float32, True)


# ------------------------------------------------------------------------------- 64 bits

def _cross_exact(st):
    """Head by head and in slabs of queries, so that the 64-bit scores stay small."""
    q, k, v = st["q"], st["k"], st["v"]
    B, N, H, d = q.shape
    M, Hkv = k.shape[1], k.shape[2]
    f64 = torch.float64
    train = "do" in st
    out = {"o": torch.zeros(B, N, H, d, dtype=f64, device="cuda")}
    if train:
        out["lse"] = torch.full((B, H, N), -math.inf, dtype=f64, device="cuda")
        out["dq"] = torch.zeros_like(out["o"])
        out["dk"] = torch.zeros(B, M, Hkv, d, dtype=f64, device="cuda")
        out["dv"] = torch.zeros_like(out["dk"])
    for b in range(B):
        keep = torch.arange(M, device="cuda")
        if st["kv_len"] is not None:
            keep = keep[keep < st["kv_len"][b]]
        if st["key_mask"] is not None:
            keep = keep[st["key_mask"][b]]
        if keep.numel() == 0:
            continue
        for h in range(H):
            hk = h * Hkv // H
            kh, vh = k[b, keep, hk].to(f64), v[b, keep, hk].to(f64)
            for n in range(0, N, 16384):
                qh = q[b, n:n + 16384, h].to(f64)
                e = (qh @ kh.T) / d ** 0.5
                top = e.max(1, keepdim=True).values
                w = (e - top).exp()
                tot = w.sum(1, keepdim=True)
                w = w / tot
                out["o"][b, n:n + 16384, h] = w @ vh
                if train:
                    out["lse"][b, h, n:n + 16384] = (top + tot.log())[:, 0]
                    gh = st["do"][b, n:n + 16384, h].to(f64)
                    gw = gh @ vh.T
                    ge = w * (gw - (w * gw).sum(1, keepdim=True)) / d ** 0.5
                    out["dq"][b, n:n + 16384, h] = ge @ kh
                    out["dk"][b, keep, hk] += ge.T @ qh
                    out["dv"][b, keep, hk] += w.T @ gh
    return out


def _boundary_exact(st):
    """The forward pass as written in the head of this file; gradients by torch's differentiation of it."""
    case = st["case"]
    f64 = torch.float64
    B, N, C = st["x"].shape
    F = _groups(case)
    names = ["x", "y", "gate", "scale", "shift", "weight", "bias", "post_weight"]
    t = {n: st[n].to(f64) for n in names if st.get(n) is not None}
    bwd = case["op"].endswith("_bwd")
    if bwd:
        t = {n: a.requires_grad_(True) for n, a in t.items()}

    def per_token(a):
        return a.repeat_interleave(N // F, dim=1)

    def normed(a, kind):
        if kind == "layer":
            mean = a.mean(-1, keepdim=True)
            return (a - mean) / ((a - mean).pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        return a / (a.pow(2).mean(-1, keepdim=True) + EPS).sqrt()

    def branch():
        u = t["y"] if case["post"] == "none" else normed(t["y"], case["post"]) * t["post_weight"]
        return per_token(t["gate"]) * u if "gate" in t else u

    def head(x):
        u = normed(x, case["norm"])
        u = u * t["weight"] if "weight" in t else u
        u = u + t["bias"] if "bias" in t else u
        u = u * (1 + per_token(t["scale"])) if "scale" in t else u
        return u + per_token(t["shift"]) if "shift" in t else u

    if not bwd:
        x = t["x"] + branch() if "y" in t else t["x"]
        return {**({"x": x} if "y" in t else {}), "h": head(x)}
    # x is the boundary's output: its total gradient is what arrives on it and what the head sends back,
    # and it passes on to the residual input unchanged and to the branch through the gate
    h = head(t["x"])
    leaves = [n for n in t if n in ("x", "scale", "shift", "weight", "bias")]
    got = dict(zip(leaves, torch.autograd.grad(h, [t[n] for n in leaves], st["dh"].to(f64))))
    if "y" in t:
        got["x"] = got["x"] + st["dx_out"].to(f64)
        leaves = [n for n in t if n in ("y", "gate", "post_weight")]
        got.update(zip(leaves, torch.autograd.grad(branch(), [t[n] for n in leaves], got["x"])))
    return {"d" + n: a for n, a in got.items()}


def exact(case, seed):
    if case["op"].startswith("cross"):
        pairs = case["B"] * case["H"] * _tokens(case) * case["M"]
        if pairs * case["d"] > 4e11:         # over about 20 seconds with the copies back
            return None
    st = prepare(case, seed)
    return _cross_exact(st) if case["op"].startswith("cross") else _boundary_exact(st)


def work(case):
    B, N = case["B"], _tokens(case)
    if case["op"].startswith("cross"):
        H, Hkv, d, M = case["H"], case["Hkv"], case["d"], case["M"]
        keys = M if case["keys"] == "all" else 2 * M / 3       # lengths are between a third and all
        qo, kv = B * N * H * d * 2, B * keys * Hkv * d * 2
        if case["op"] == "cross":
            return {"bytes": 2 * qo + 2 * kv, "flops": 4 * B * H * N * keys * d}
        # forward: q, k, v in, o, lse out; backward: q, k, v, o, do, lse in, dq, dk, dv out
        return {"bytes": 6 * qo + 6 * kv + 8 * B * H * N, "flops": 14 * B * H * N * keys * d}
    C, F = case["C"], _groups(case)
    s = 2 if case["stream"] == "bf16" else 4
    rows, par = B * N * C, B * F * C * 4
    mods = (2 if case["mod"] else 0) + (1 if case["mod"] and case["op"].startswith("residual") else 0)
    if case["op"] == "modulate":
        return {"bytes": rows * (s + 2) + mods * par, "flops": 8 * rows}
    if case["op"] == "residual":
        return {"bytes": rows * (s + 2 + s + 2) + mods * par, "flops": 14 * rows}
    if case["op"] == "modulate_bwd":
        return {"bytes": rows * (2 + s + s) + 2 * mods * par, "flops": 16 * rows}
    return {"bytes": rows * (2 + s + s + 2 + s + 2) + 2 * mods * par, "flops": 24 * rows}
