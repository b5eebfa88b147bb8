"""fp64 oracle of the operators around a block's self-attention: cross attention to an encoder's states and the
norms at the block's boundaries, with their gradients written out from the formulas (include/bsa.h).

Arrays are numpy float64.  Besides each result the attention functions return the sums of absolute terms that
error bounds are made of.
"""
import numpy as np


def valid_states(B, M, kv_len=None, key_mask=None):
    """Boolean [B, M]: the states that count."""
    on = np.ones((B, M), dtype=bool)
    if kv_len is not None:
        on &= np.arange(M)[None, :] < np.asarray(kv_len).reshape(B, 1)
    if key_mask is not None:
        on &= np.asarray(key_mask).astype(bool)
    return on


def _probabilities(q, k, on):
    """P [B,H,N,M] (0 where a state does not count), lse [B,H,N], and max_j sum_c |q_c k_jc| / sqrt(d)."""
    B, N, H, d = q.shape
    G = H // k.shape[2]
    kh = np.where(on[:, :, None, None], k, 0.0).repeat(G, axis=2)
    s = np.einsum("bnhd,bjhd->bhnj", q, kh) / np.sqrt(d)
    s = np.where(on[:, None, None, :], s, -np.inf)
    if s.shape[3] == 0:
        return s, np.full((B, H, N), -np.inf), np.zeros((B, H, N))
    m = s.max(axis=3, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(s - m)
    l = e.sum(axis=3, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[..., 0]
    size = np.einsum("bnhd,bjhd->bhnj", np.abs(q), np.abs(kh)).max(axis=3) / np.sqrt(d)
    return e / np.where(l == 0, 1.0, l), lse, size


def cross_attention(q, k, v, on):
    """o [B,N,H,d], lse [B,H,N], sum_j P|v| [B,N,H,d] and the score size [B,H,N]."""
    P, lse, size = _probabilities(q, k, on)
    G = q.shape[2] // k.shape[2]
    vh = np.where(on[:, :, None, None], v, 0.0).repeat(G, axis=2)
    return (np.einsum("bhnj,bjhd->bnhd", P, vh), lse, np.einsum("bhnj,bjhd->bnhd", P, np.abs(vh)), size)


def cross_attention_grad(q, k, v, on, do):
    """dq, dk, dv and the pieces of their error bounds (see cross_grad_bounds)."""
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    G = H // Hkv
    rd = 1.0 / np.sqrt(d)
    P, _, size = _probabilities(q, k, on)
    kh = np.where(on[:, :, None, None], k, 0.0).repeat(G, axis=2)
    vh = np.where(on[:, :, None, None], v, 0.0).repeat(G, axis=2)
    dP = np.einsum("bnhd,bjhd->bhnj", do, vh)
    D = (P * dP).sum(axis=3, keepdims=True)
    dS = P * (dP - D)

    def share(t):                                        # sum over the query heads of a key head
        return t.reshape(B, t.shape[1], Hkv, G, d).sum(axis=3)

    dq = np.einsum("bhnj,bjhd->bnhd", dS, kh) * rd
    dk = share(np.einsum("bhnj,bnhd->bjhd", dS, q)) * rd
    dv = share(np.einsum("bhnj,bnhd->bjhd", P, do))
    return dq, dk, dv, dict(P=P, dP=dP, dS=dS, kh=kh, vh=vh, size=size)


U16, U32 = 2.0 ** -8, 2.0 ** -24


def cross_bound(o, absv, size, d):
    """Elementwise bound of o: P and o rounded once to bf16 (2^-8 each); a score is off by at most
    (d + 3) 2^-24 of its absolute sum, an exponential by 2^-14 more, numerator and row sum alike."""
    e = 2 * ((d + 3) * U32 * size + 2.0 ** -14)                     # [B,H,N]
    e = np.moveaxis(e, 1, 2)[..., None]
    return (U16 * np.abs(o) + (U16 + e) * absv) * 1.01 + 1e-37


def cross_grad_bounds(q, do, o_bound, info, Hkv):
    """Elementwise bounds of dq, dk, dv: P and dS are rounded to bf16 (2^-8), P is off by e as in cross_bound,
    dP by (d + 1) 2^-24 of its absolute sum, D by sum_c |do| times the bound of o (D is made from the o the
    forward pass returned); sums over N G terms and the last rounding."""
    P, dP, dS, kh, vh, size = (info[n] for n in ("P", "dP", "dS", "kh", "vh", "size"))
    B, N, H, d = q.shape
    G = H // Hkv
    e = 2 * ((d + 3) * U32 * size + 2.0 ** -14)[..., None]          # [B,H,N,1]
    absdp = np.einsum("bnhd,bjhd->bhnj", np.abs(do), np.abs(vh))
    ddp = (d + 1) * U32 * absdp + np.moveaxis((np.abs(do) * o_bound).sum(axis=3), 1, 2)[..., None]
    ds = (U16 + e) * np.abs(dS) + P * ddp * (1 + U16)
    acc = (N * G + 4) * U32
    rd = 1.0 / np.sqrt(d)

    def share(t):
        return t.reshape(B, t.shape[1], Hkv, G, d).sum(axis=3)

    bq = np.einsum("bhnj,bjhd->bnhd", ds, np.abs(kh)) * rd
    bk = share(np.einsum("bhnj,bnhd->bjhd", ds + acc * np.abs(dS), np.abs(q))) * rd
    bv = share(np.einsum("bhnj,bnhd->bjhd", (U16 + e + acc) * P, np.abs(do)))
    dq = np.einsum("bhnj,bjhd->bnhd", dS, kh) * rd
    dk = share(np.einsum("bhnj,bnhd->bjhd", dS, q)) * rd
    dv = share(np.einsum("bhnj,bnhd->bjhd", P, do))
    return tuple((b + U16 * np.abs(t)) * 1.01 + 1e-37 for b, t in ((bq, dq), (bk, dk), (bv, dv)))


# ---- norms ----

def normalise(x, kind, eps):
    """(normalised rows, 1 / deviation); kind "layer" or "rms"."""
    c = x - x.mean(axis=-1, keepdims=True) if kind == "layer" else x
    r = 1.0 / np.sqrt((c * c).mean(axis=-1, keepdims=True) + eps)
    return c * r, r


def _rows(p, N):
    """[B, groups, C] as [B, N, C]."""
    return p.repeat(N // p.shape[1], axis=1)


def boundary(x, y=None, gate=None, scale=None, shift=None, weight=None, bias=None, post_weight=None, norm="layer",
             post=None, res_scale=1.0, eps=1e-6):
    """(x_out, h); norm None: h is None; y None: x_out is x."""
    N = x.shape[1]
    if y is not None:
        u = y if post is None else normalise(y, post, eps)[0]
        u = u if post_weight is None else u * post_weight
        u = u if gate is None else u * _rows(gate, N)
        x = res_scale * x + u
    if norm is None:
        return x, None
    h = normalise(x, norm, eps)[0]
    h = h if weight is None else h * weight
    h = h if bias is None else h + bias
    h = h if scale is None else h * (1 + _rows(scale, N))
    return x, h if shift is None else h + _rows(shift, N)


def _through(g, xh, r, kind):
    t = g - xh * (g * xh).mean(axis=-1, keepdims=True)
    return r * (t - g.mean(axis=-1, keepdims=True) if kind == "layer" else t)


def boundary_grad(x_out, dh=None, dx_out=None, y=None, gate=None, scale=None, shift=None, weight=None, bias=None,
                  post_weight=None, norm="layer", post=None, res_scale=1.0, eps=1e-6, groups=1):
    """Gradients by name (dx, dy, dgate, dscale, dshift, dweight, dbias, dpost_weight), those that exist."""
    B, N, C = x_out.shape

    def gsum(t):
        return t.reshape(B, groups, N // groups, C).sum(axis=2)

    out = {}
    g = np.zeros_like(x_out) if dx_out is None else dx_out.copy()
    one = 1.0 if scale is None else 1 + _rows(scale, N)
    if dh is not None:
        xh, r = normalise(x_out, norm, eps)
        u = xh if weight is None else xh * weight
        u = u if bias is None else u + bias
        out["dscale"], out["dshift"] = gsum(dh * u), gsum(dh)
        out["dweight"], out["dbias"] = (dh * one * xh).sum(axis=(0, 1)), (dh * one).sum(axis=(0, 1))
        g = g + _through(dh * one * (1.0 if weight is None else weight), xh, r, norm)
    if y is not None:
        yh, ry = (y, None) if post is None else normalise(y, post, eps)
        pw = 1.0 if post_weight is None else post_weight
        gt = 1.0 if gate is None else _rows(gate, N)
        out["dgate"], out["dpost_weight"] = gsum(g * yh * pw), (g * gt * yh).sum(axis=(0, 1))
        gy = g * gt * pw
        out["dy"] = gy if post is None else _through(gy, yh, ry, post)
        g = res_scale * g
    out["dx"] = g
    return out
