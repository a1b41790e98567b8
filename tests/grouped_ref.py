"""Plain forms in 64 bits of the grouped products and the 4-bit block
formats, and the tolerances that follow from their arithmetic."""
import numpy as np
import torch

VEC = {0: 32, 1: 16}                                   # STRATA_FP4_MX, STRATA_FP4_NV
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32)


def spans(offsets):
    o = [int(v) for v in offsets]
    return list(zip(o[:-1], o[1:]))


def mm(x, w, offsets):
    """(sum, sum of magnitudes) of the forward product, float64; rows of no group are zero."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    m = torch.zeros_like(y)
    for e, (a, b) in enumerate(spans(offsets)):
        y[a:b] = x[a:b].double() @ w[e].double().T
        m[a:b] = x[a:b].double().abs() @ w[e].double().abs().T
    return y, m


def dx(dy, w, offsets):
    return mm(dy, w.transpose(1, 2), offsets)


def dw(dy, x, offsets):
    E = len(offsets) - 1
    y = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    m = torch.zeros_like(y)
    for e, (a, b) in enumerate(spans(offsets)):
        y[e] = dy[a:b].double().T @ x[a:b].double()
        m[e] = dy[a:b].double().abs().T @ x[a:b].double().abs()
    return y, m


def half_step(dtype, ref):
    """Half a step of the output type at |ref|: eps / 2 relative, at least half the smallest one."""
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def sum_error(n, mags):
    """n fp32 additions, each off by at most one step (2^-23, truncation
    included) of a partial sum that the magnitudes' sum bounds; plus the
    products' own rounding, none for 16-bit and smaller factors."""
    return n * 2.0 ** -23 * mags


def check(got, ref, mags, n, what=""):
    """Elementwise: the sum's error bound, then the output's rounding of a
    value that far off.  And over all values: the errors of n additions with
    random signs grow like sqrt(n) steps, far inside 1e-5 for n <= 4096."""
    g, dt = got.double(), got.dtype
    assert torch.isfinite(g).all(), f"{what}: not finite"
    err = sum_error(n, mags)
    tol = err + half_step(dt, ref.abs() + err)
    over = (g - ref).abs() - tol
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} values off, worst by {over.max():.3e}"
    norm = float(ref.norm())
    if norm > 0:
        rel = float((g - ref).norm()) / norm
        assert rel <= torch.finfo(dt).eps / 2 + 1e-5, f"{what}: rel {rel:.3e}"


# ------------------------------------------------------------ 4-bit formats
def quantize(x, fmt, scale_exp=0):
    """(codes uint8 [R][C], scale bytes uint8 [R][C / V]) of float64 rows, from the definition."""
    vec = VEC[fmt]
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    b = x.reshape(R, C // vec, vec) * 2.0 ** -scale_exp
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    if fmt == 0:
        e = np.maximum(np.frexp(amax)[1] - 1 - 2, -127)
        s = np.where(amax > 0, np.exp2(e.astype(np.float64)), 0.0)
        byte = np.where(amax > 0, e + 127, 0)
        byte = np.where(bad, 255, byte)
    else:
        v = np.minimum(amax / 6, 448.0)
        step = np.exp2(np.maximum(np.frexp(v)[1] - 1, -6).astype(np.float64) - 3)
        s = np.rint(v / step) * step                    # rint: ties to even
        ex = np.frexp(s)[1] - 1
        byte = np.where(ex < -6, s * 512, (ex + 7) * 8 + (s / np.exp2(ex.astype(np.float64)) - 1) * 8)
        byte = np.where(bad, 0x7f, np.where(s > 0, byte, 0))
    q = np.abs(b) / np.where(s > 0, s, 1.0)[..., None]
    q = np.where((s > 0)[..., None], q, 0.0)
    q = np.where(q < 2, np.rint(2 * q) / 2, np.where(q < 4, np.rint(q), 2 * np.rint(q / 2)))
    code = np.searchsorted(GRID, np.minimum(q, 6.0))
    # the sign stays, a zero's too: e2m1 has a negative zero
    code = code + np.where(np.signbit(b) & (s > 0)[..., None], 8, 0)
    return code.reshape(R, C).astype(np.uint8), byte.astype(np.uint8)


def values(codes, byte, fmt, scale_exp=0):
    vec = VEC[fmt]
    v = np.concatenate([GRID, -GRID])[codes]
    b = byte.astype(np.float64)
    if fmt == 0:
        s = np.where(byte == 255, np.nan, np.exp2(b - 127))
    else:
        e, m = byte >> 3, (byte & 7).astype(np.float64)
        s = np.where(e > 0, (8 + m) * np.exp2(e.astype(np.float64) - 10), m * 2.0 ** -9)
        s = np.where((byte & 0x7f) == 0x7f, np.nan, s)
    return v * np.repeat(s, vec, axis=1) * 2.0 ** scale_exp


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def tile_places(counts, cols, fmt):
    """(byte place of each scale, row by row of the groups in order; bytes in all the blocks)."""
    vec = VEC[fmt]
    words, n = -(-cols // (4 * vec)), cols // vec
    place, block = [], 0
    c = np.arange(n)
    for cnt in counts:
        for r in range(cnt):
            place.append(((block + r // 128) * words + c // 4) * 512 + (r % 32) * 16
                         + (r % 128 // 32) * 4 + c % 4)
        block += -(-cnt // 128)
    return np.array(place, dtype=np.int64).reshape(-1, n), block * words * 512


def tiled(byte, counts, cols, fmt, nbytes, fill=0):
    place, used = tile_places(counts, cols, fmt)
    out = np.full(nbytes, fill, dtype=np.uint8)
    out[:used] = 0
    out[place] = byte
    return out
