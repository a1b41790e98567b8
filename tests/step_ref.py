"""Plain forms in 64 bits of the tuning step's operators (SwiGLU experts, rows
kept in 8 bits, slots and tokens, the norms around a block), and the error that
their fp32 arithmetic may make: each function returns values and bounds.

U is half a step of fp32, relative (one rounding).  The sigmoid of the SwiGLU
epilogues is off by at most 7 + 1.2 |g| steps of 2^-23 (held to that in
test_gpu_swiglu_sigmoid.py); silu_error allows 12 + 2.4 |g|, for it and for
1 - sigmoid next to it."""
import numpy as np
import torch

from tests import grouped_ref as ref

U = 2.0 ** -24


def near(got, want, err, what=""):
    """Elementwise: `err`, then the output type's rounding of a value that far off."""
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    over = (g - want).abs() - (err + ref.half_step(got.dtype, want.abs() + err))
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()} off, worst by {over.max():.3e}"


# ------------------------------------------------------------------ SwiGLU
def silu_error(g):
    """Relative error of sigmoid(g) and 1 - sigmoid(g) as the kernels take them."""
    return (2 * (2 + 1.2 * g.abs()) + 4 + 4) * 2 * U


def swiglu(p, dp):
    """(h, its error) of p [M][2I] that is known to dp."""
    g, u, eg, eu = p[:, 0::2], p[:, 1::2], dp[:, 0::2], dp[:, 1::2]
    a = g * torch.sigmoid(g)
    h = a * u
    # |silu'| <= 1.1
    err = 1.1 * eg * (u.abs() + eu) + a.abs() * eu + h.abs() * (silu_error(g) + 4 * U)
    return h, err


def swiglu_back(dh, edh, p):
    """((dp, error), (h, error)) of dh known to edh."""
    g, u = p[:, 0::2], p[:, 1::2]
    s, t = torch.sigmoid(g), torch.sigmoid(-g)
    a = g * s
    phi = s + a * t
    e = silu_error(g) + 4 * U
    dp, err = torch.zeros_like(p), torch.zeros_like(p)
    dp[:, 0::2], dp[:, 1::2] = dh * u * phi, dh * a
    # dh's error, and that of phi's two terms (the second has both factors' errors)
    err[:, 0::2] = edh * (u * phi).abs() + (dh.abs() + edh) * u.abs() * (s + 2 * (a * t).abs()) * e
    err[:, 1::2] = edh * a.abs() + (dh.abs() + edh) * a.abs() * e
    return (dp, err), (a * u, (a * u).abs() * e)


# ---------------------------------------------------------- rows in 8 bits
def e4m3_table():
    """The values of the codes 0 .. 126."""
    c = np.arange(127)
    return np.where(c < 8, c * 2.0 ** -9, (8 + c % 8) * np.exp2((c >> 3) - 10.0))


def act8_save(x):
    """(codes, scale bytes) of float64 rows, from the definition."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(axis=2)
    v = np.where(bad[..., None], 0.0, b)
    m = np.abs(v).max(axis=2)
    e = np.full(m.shape, -126)
    for k in range(-125, 128):
        e = np.where(m > 448.0 * 2.0 ** (k - 1), k, e)
    q = np.abs(v) * np.exp2(-e.astype(np.float64))[..., None]
    table = e4m3_table()
    lo = np.clip(np.searchsorted(table, q, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    dl, dh = q - table[lo], table[hi] - q
    code = np.where((dh < dl) | ((dh == dl) & (lo % 2 == 1)), hi, lo)
    code = code + np.where(np.signbit(v), 128, 0)
    code = np.where(bad[..., None], 0x7f, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def act8_load(codes, byte):
    c = codes.astype(np.int64)
    v = np.append(e4m3_table(), np.nan)[c & 127] * np.where(c >> 7, -1.0, 1.0)
    s = np.where(byte == 0, 0.0, np.exp2(byte.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)


# -------------------------------------------------------- slots and tokens
def combine(y, inv, weights):
    """(sum, sum of magnitudes), slots outside y left out."""
    T, K = inv.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(out)
    for k in range(K):
        s = inv[:, k].long()
        live = ((s >= 0) & (s < y.shape[0])).double()[:, None]
        w = weights[:, k:k + 1].double() if weights is not None else torch.ones_like(live)
        v = live * w * y[s.clamp(0, y.shape[0] - 1)].double()
        out += v
        mag += v.abs()
    return out, mag


def spread(dout, inv, weights, y, M):
    """(dy, which rows it has, dweights, sum of magnitudes of dweights' terms)."""
    T, K = inv.shape
    dy = torch.zeros(M, dout.shape[1], dtype=torch.float64, device=dout.device)
    there = torch.zeros(M, dtype=torch.bool, device=dout.device)
    dw = torch.zeros(T, K, dtype=torch.float64, device=dout.device)
    mag = torch.zeros_like(dw)
    for k in range(K):
        s = inv[:, k].long()
        live = (s >= 0) & (s < M)
        w = weights[live, k:k + 1].double() if weights is not None else 1.0
        dy[s[live]] = w * dout[live].double()
        there[s[live]] = True
        if y is not None:
            t = dout[live].double() * y[s[live]].double()
            dw[live, k], mag[live, k] = t.sum(dim=1), t.abs().sum(dim=1)
    return dy, there, dw, mag


# ------------------------------------------------------------------- norms
def depth(H):
    """Additions that a row's sum passes one after the other, with its terms' own roundings: pieces
    of at most 64 a thread, the pieces, a CTA's threads."""
    return 64 + H // 16384 + 48


def norm(f, r, w_post, gate, post, alpha, beta, eps):
    """((r' before it is stored, error), s0)."""
    n = torch.zeros_like(r)
    s0 = torch.ones(r.shape[0], 1, dtype=torch.float64, device=r.device)
    if f is not None:
        if post:
            s0 = 1 / torch.sqrt(f.square().mean(dim=1, keepdim=True) + eps)
        n = f * s0
        if w_post is not None:
            n = n * w_post
        if gate is not None:
            n = n * gate[:, None]
        n = beta * n
    out = alpha * r + n
    err = n.abs() * (depth(r.shape[1]) / 2 + 8) * U + ((alpha * r).abs() + out.abs()) * 2 * U
    return out, err, s0


def pre(v, w_pre, eps):
    """((x, error), s1) of the residual as it is stored."""
    s1 = 1 / torch.sqrt(v.square().mean(dim=1, keepdim=True) + eps)
    x = v * s1
    if w_pre is not None:
        x = x * w_pre
    return x, x.abs() * (depth(v.shape[1]) / 2 + 8) * U, s1


def norm_back(dx, dr2, f, v, w_post, w_pre, gate, s0, s1, post, alpha, beta):
    """{name: (gradient, error)}."""
    like = v if dr2 is None else dr2
    T, H = like.shape
    one = torch.ones(H, dtype=torch.float64, device=like.device)
    wpre, wpost = (one if w is None else w for w in (w_pre, w_post))
    g = torch.ones(T, 1, dtype=torch.float64, device=like.device) if gate is None else gate[:, None]
    d = torch.zeros_like(like) if dr2 is None else dr2.clone()
    ed = 2 * U * d.abs()
    n = depth(H) + 8
    out = {}
    if dx is not None:
        gx = dx * wpre
        m = (gx * v).sum(dim=1, keepdim=True)
        em = n * U * (gx * v).abs().sum(dim=1, keepdim=True)
        c = s1 ** 3 * m / H
        d = d + s1 * gx - c * v
        ed = ed + 6 * U * ((s1 * gx).abs() + (c * v).abs() + d.abs()) + s1 ** 3 / H * em * v.abs()
    out["dresid"] = (alpha * d, abs(alpha) * ed + 2 * U * (alpha * d).abs())
    # a column's sums: rows of a piece, a CTA's pieces, the CTAs
    rows = min(T, 640 + T // 4096) + 8
    if dx is not None:
        t = dx * v * s1
        out["dw_pre"] = (t.sum(dim=0), rows * U * t.abs().sum(dim=0))
    dn, edn = beta * g * d, abs(beta) * g.abs() * (ed + 3 * U * d.abs())
    if f is None:
        out["df"] = (dn, edn)
        return out
    t = d * wpost * f
    q = t.sum(dim=1, keepdim=True)
    eq = (ed * (wpost * f).abs() + n * U * t.abs()).sum(dim=1, keepdim=True)
    out["dgate"] = ((beta * s0 * q)[:, 0], (abs(beta) * s0 * (eq + 4 * U * q.abs()))[:, 0])
    if not post:
        out["df"] = (dn, edn)
        return out
    t = dn * f * s0
    out["dw_post"] = (t.sum(dim=0), (edn * (f * s0).abs() + rows * U * t.abs()).sum(dim=0))
    c = beta * g * s0 ** 3 * q / H
    ec = abs(beta) * g.abs() * s0 ** 3 * eq / H + 6 * U * c.abs()
    df = s0 * dn * wpost - c * f
    out["df"] = (df, s0 * (edn + 3 * U * dn.abs()) * wpost.abs() + ec * f.abs()
                 + 3 * U * ((c * f).abs() + df.abs()))
    return out
