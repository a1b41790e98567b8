"""The 4-bit block formats and their grouped product on the GPU: codes and
scales bit for bit, products against 64-bit plain forms."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import grouped_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FMT = [pytest.param(0, id="mx"), pytest.param(1, id="nv")]
COUNTS = {
    "one": [1],
    "token": [0, 1, 1, 0, 0, 1, 0, 1],
    "edges": [127, 128, 129, 0, 1, 257],
    "empty": [0, 0],
    "many": [(5 * e) % 7 for e in range(300)],
}


def _done(ws):
    assert q.moe_get_device_status(ws) == q.STRATA_OK


def _rows(M, C, dtype, seed, fmt):
    """Rows whose blocks cover what the formats meet: ordinary values, wide ranges inside a block,
    exact ties between codes, zeros, one value alone, tiny and large scales."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((M, C))
    vec = ref.VEC[fmt]
    kind = g.integers(0, 7, (M, C // vec)).repeat(vec, axis=1)
    x = np.where(kind == 1, x * np.exp2(g.integers(-12, 6, (M, C))), x)
    ties = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 4, 0.5])
    x = np.where(kind == 2, np.sign(x) * ties[g.integers(0, 10, (M, C))], x)
    x = np.where(kind == 3, 0.0, x)
    x = np.where(kind == 4, x * np.exp2(-9.0), x)
    x = np.where(kind == 5, x * 300.0, x)
    x = np.where(kind == 6, np.where(g.random((M, C)) < 0.1, x, 0.0), x)
    return torch.from_numpy(x).to(DT[dtype])


def _bufs(M, C, fmt, groups, ragged=True, fill=0xAB):
    return (torch.full((M, C // 2), fill, dtype=torch.uint8, device="cuda"),
            torch.full((max(q.moe_fp4_scale_bytes(fmt, M, C, groups, ragged), 16),), fill,
                       dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("C", [32, 96, 256, 1120])
@pytest.mark.parametrize("name", COUNTS)
def test_quantize_bit_exact(name, C, dtype, fmt):
    counts = COUNTS[name]
    M, spare = sum(counts), 5
    ex = 3 if fmt else 0
    x = _rows(M + spare, C, dtype, 3, fmt)
    codes, sb = ref.quantize(x.double().numpy(), fmt, ex)
    qd, sc = _bufs(M + spare, C, fmt, len(counts))
    ws, off = q.make_grouped_workspace(), ref.offsets_of(counts).cuda()
    q.moe_fp4_quantize(x.cuda(), qd, sc, fmt, ws, offsets=off, scale_exp=ex)
    got = qd.cpu().numpy()
    assert np.array_equal(ref.unpack(got[:M]), codes[:M])
    assert (got[M:] == 0xAB).all()
    place, used = ref.tile_places(counts, C, fmt)
    scb = sc.cpu().numpy()
    assert np.array_equal(scb[place], sb[:M])
    assert (scb[used:] == 0xAB).all()
    # the last word of a row is filled with zeros
    vec = ref.VEC[fmt]
    n = C // vec
    if n % 4 and M:
        tail = place[:, -1:] - (n - 1) % 4 + np.arange(n % 4, 4)
        assert (scb[tail] == 0).all()
    # and back to values
    for odt in (DT[dtype], torch.float32):
        v = torch.full((M + spare, C), 7.0, dtype=odt, device="cuda")
        q.moe_fp4_dequantize(qd, sc, v, fmt, ws, offsets=off, scale_exp=ex)
        want = torch.from_numpy(ref.values(codes[:M], sb[:M], fmt, ex)).to(odt)
        assert torch.equal(v[:M].cpu(), want)
        assert (v[M:] == 7).all()
    _done(ws)


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_equal_groups_are_weights(fmt):
    E, N, K = 3, 136, 160
    w = _rows(E * N, K, "bf16", 4, fmt)
    codes, sb = ref.quantize(w.double().numpy(), fmt)
    qd, sc = _bufs(E * N, K, fmt, E, ragged=False)
    ws = q.make_grouped_workspace()
    q.moe_fp4_quantize(w.cuda(), qd, sc, fmt, ws, n_groups=E)
    place, used = ref.tile_places([N] * E, K, fmt)
    assert used == sc.numel()
    assert np.array_equal(ref.unpack(qd.cpu().numpy()), codes)
    assert np.array_equal(sc.cpu().numpy()[place], sb)
    v = torch.zeros(E * N, K, device="cuda")
    q.moe_fp4_dequantize(qd, sc, v, fmt, ws, n_groups=E)
    assert torch.equal(v.cpu().double(), torch.from_numpy(ref.values(codes, sb, fmt)))
    _done(ws)


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_gathers_by_perm(fmt):
    T, K, C = 37, 3, 192
    g = np.random.default_rng(0)
    ids = np.sort(np.stack([g.choice(6, K, replace=False) for _ in range(T)]), axis=1).reshape(-1)
    perm = np.argsort(ids, kind="stable").astype(np.int32)
    counts = np.bincount(ids, minlength=6)
    x = _rows(T, C, "bf16", 6, fmt)
    codes, sb = ref.quantize(x.double().numpy(), fmt)
    qd, sc = _bufs(T * K, C, fmt, 6)
    ws, off = q.make_grouped_workspace(), ref.offsets_of(counts).cuda()
    q.moe_fp4_quantize(x.cuda(), qd, sc, fmt, ws, offsets=off, perm=torch.from_numpy(perm).cuda(),
                       top_k=K)
    place, _ = ref.tile_places(counts, C, fmt)
    assert np.array_equal(ref.unpack(qd.cpu().numpy()), codes[perm // K])
    assert np.array_equal(sc.cpu().numpy()[place], sb[perm // K])
    _done(ws)
    # entries out of range read as zeros and are reported; the others are unharmed
    perm[[0, 50]] = [T * K, -3]
    q.moe_fp4_quantize(x.cuda(), qd, sc, fmt, ws, offsets=off, perm=torch.from_numpy(perm).cuda(),
                       top_k=K)
    got = ref.unpack(qd.cpu().numpy())
    ok = np.ones(T * K, dtype=bool)
    ok[[0, 50]] = False
    assert np.array_equal(got[ok], codes[perm[ok] // K]) and (got[~ok] == 0).all()
    assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", DT)
def test_quantize_extremes(fmt, dtype):
    """Blocks with infinities and NaNs read back as NaN and harm no neighbour; the smallest and
    largest magnitudes of each type."""
    f = torch.finfo(DT[dtype])
    x = torch.ones(8, 128, dtype=DT[dtype])
    x[0, 3], x[1, 40], x[2, 127] = float("nan"), float("inf"), float("-inf")
    x[3] = f.max
    x[4] = f.smallest_normal
    x[5] = f.smallest_normal * f.eps                    # the smallest subnormal
    x[6, ::2] = -f.max
    x[7, :64] = f.smallest_normal * f.eps * 3
    codes, sb = ref.quantize(x.double().numpy(), fmt)
    qd, sc = _bufs(8, 128, fmt, 1, ragged=False)
    ws = q.make_grouped_workspace()
    q.moe_fp4_quantize(x.cuda(), qd, sc, fmt, ws)
    place, _ = ref.tile_places([8], 128, fmt)
    got, gs = ref.unpack(qd.cpu().numpy()), sc.cpu().numpy()[place]
    assert np.array_equal(gs, sb)
    assert np.array_equal(got, codes)
    v = torch.zeros(8, 128, device="cuda")
    q.moe_fp4_dequantize(qd, sc, v, fmt, ws)
    want = torch.from_numpy(ref.values(codes, sb, fmt)).float()
    assert torch.equal(v.cpu().isnan(), want.isnan())
    assert torch.equal(v.cpu().nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("ex", [-64, -8, 0, 11, 64])
def test_nv_scale_exp(ex):
    x = (torch.randn(20, 64, generator=torch.Generator().manual_seed(1)) * 2.0 ** ex)
    for dt in (torch.bfloat16, torch.float32):
        xd = x.to(dt)
        codes, sb = ref.quantize(xd.double().numpy(), 1, ex)
        qd, sc = _bufs(20, 64, 1, 1, ragged=False)
        ws = q.make_grouped_workspace()
        q.moe_fp4_quantize(xd.cuda(), qd, sc, 1, ws, scale_exp=ex)
        place, _ = ref.tile_places([20], 64, 1)
        assert np.array_equal(ref.unpack(qd.cpu().numpy()), codes)
        assert np.array_equal(sc.cpu().numpy()[place], sb)
        v = torch.zeros(20, 64, device="cuda")
        q.moe_fp4_dequantize(qd, sc, v, 1, ws, scale_exp=ex)
        assert torch.equal(v.cpu().double(), torch.from_numpy(ref.values(codes, sb, 1, ex)))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("ex", [0, -5, 17])
def test_nv_every_scale_and_border(dtype, ex):
    """A block for each e4m3 scale whose elements are that scale's seven borders, the values beside
    them in the type, and the values themselves; and blocks whose largest magnitude is a border
    between two scales, or beside one."""
    if dtype == "fp16" and ex == 17:
        pytest.skip("outside fp16's range")
    dt = DT[dtype]
    s = np.array([m * 2.0 ** -9 for m in range(1, 8)]
                 + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if e < 15 or m < 7])
    s = s[(s * 6 * 2.0 ** ex < float(torch.finfo(dt).max)) & (s * 2.0 ** ex > 2.0 ** -12)]
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for off in (0, -1, 1):
        v = torch.from_numpy(s[:, None] * borders * 2.0 ** ex).to(dt)
        bits = v.view(torch.int32 if dt == torch.float32 else torch.int16)
        v = (bits + off).view(dt).double().numpy()
        rows.append(np.concatenate([6 * s[:, None] * 2.0 ** ex, v, -v, s[:, None] * 2.0 ** ex], axis=1))
    mids = (s[1:] + s[:-1]) / 2
    top = torch.from_numpy(6 * mids * 2.0 ** ex).to(dt)
    bits = top.view(torch.int32 if dt == torch.float32 else torch.int16)
    for off in (0, -1, 1):
        t = (bits + off).view(dt).double().numpy()
        rows.append(np.concatenate([t[:, None], np.outer(mids * 2.0 ** ex, np.linspace(-5, 5, 15))], axis=1))
    x = torch.from_numpy(np.concatenate(rows)).to(dt)
    x = torch.cat([x, x.flip(1)], dim=1)                # 32 columns: two blocks a row
    R = x.shape[0]
    codes, sb = ref.quantize(x.double().numpy(), 1, ex)
    qd, sc = _bufs(R, 32, 1, 1, ragged=False)
    ws = q.make_grouped_workspace()
    q.moe_fp4_quantize(x.cuda(), qd, sc, 1, ws, scale_exp=ex)
    place, _ = ref.tile_places([R], 32, 1)
    assert np.array_equal(sc.cpu().numpy()[place], sb)
    assert np.array_equal(ref.unpack(qd.cpu().numpy()), codes)


# -------------------------------------------------------------- the product
def _operand(counts, K, fmt, seed, ragged, fill=0xFF):
    """Random codes and scales of groups of rows: (packed, tiled on the GPU, float64 values).
    Unused scale bytes hold `fill` (NaN in both formats)."""
    g = np.random.default_rng(seed)
    M = sum(counts)
    codes = g.integers(0, 16, (M, K), dtype=np.uint8)
    n = K // ref.VEC[fmt]
    sb = (g.integers(121, 131, (M, n)) if fmt == 0 else g.integers(0x20, 0x48, (M, n))).astype(np.uint8)
    nbytes = max(q.moe_fp4_scale_bytes(fmt, M, K, len(counts), ragged), 16)
    place, used = ref.tile_places(counts, K, fmt)
    t = np.full(nbytes, fill, dtype=np.uint8)
    t[place] = sb
    if n % 4 and M:                                     # the row's last word is zero-filled
        t[place[:, -1:] - (n - 1) % 4 + np.arange(n % 4, 4)] = 0
    return (torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(t).cuda(),
            torch.from_numpy(ref.values(codes, sb, fmt)).cuda())


MM = {
    "one_row": ([1], 64, 64),
    "token": ([0, 1, 1, 0, 0, 1, 0, 1], 512, 384),
    "edges": ([127, 128, 129, 0, 1, 257], 256, 136),
    "one_group": ([700], 1024, 520),
    "empty": ([0, 0, 0], 128, 128),
    "odd": ([3, 64, 17, 0, 65], 160, 1002),
    "narrow": ([9, 0, 40], 32, 2),
    "odd_k": ([130, 2], 96, 66),
    "long": ([40, 300, 7], 2560, 264),
    "many": ([(7 * e) % 11 for e in range(300)], 128, 72),
}


def _swiglu(p, mags, n):
    """float64 SwiGLU of interleaved gate / up and the error bound it inherits: |silu'| <= 1.1, plus
    the fp32 exponential (2 ulp, of an argument off by half an ulp), sum, quotient and product."""
    g, u, e = p[:, 0::2], p[:, 1::2], ref.sum_error(n, mags)
    s = g * torch.sigmoid(g)
    tol = 1.1 * e[:, 0::2] * (u.abs() + e[:, 1::2]) + s.abs() * e[:, 1::2]
    y = s * u
    return y, tol + (8 + g.abs()) * 2.0 ** -23 * y.abs()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("out", DT)
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("name", MM)
def test_grouped_mm_fp4(name, fmt, out, swiglu):
    counts, K, N = MM[name]
    E, M, spare = len(counts), sum(counts), 9
    xq, xs, xv = _operand(counts, K, fmt, 1, True)
    xq = torch.cat([xq, torch.full((spare, K // 2), 0x77, dtype=torch.uint8, device="cuda")])
    need = q.moe_fp4_scale_bytes(fmt, M + spare, K, E, True)
    xs = torch.cat([xs, torch.full((max(need - xs.numel(), 0),), 0xFF, dtype=torch.uint8, device="cuda")])
    wq, wsc, wv = _operand([N] * E, K, fmt, 2, False)
    off, ws = ref.offsets_of(counts).cuda(), q.make_grouped_workspace()
    g = torch.Generator(device="cuda").manual_seed(2)
    # alpha brings the sums near one, so that fp16 holds them and SwiGLU bends
    alpha = (1 + torch.rand(E, generator=g, device="cuda")) / (16 * K ** 0.5)
    y = torch.full((M + spare, N // 2 if swiglu else N), 7.0, dtype=DT[out], device="cuda")
    q.moe_grouped_mm_fp4(xq, xs, wq.view(E, N, K // 2), wsc, off, y, fmt, ws, alpha=alpha, swiglu=swiglu)
    assert (y[M:] == 7).all()
    p, mags = ref.mm(xv, wv.view(E, N, K), off)
    rows = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))
    p, mags = p * alpha.double()[rows][:, None], mags * alpha.double()[rows][:, None]
    n = K + 2                                           # the sums, and alpha's product
    if not swiglu:
        ref.check(y[:M], p, mags, n, name)
    else:
        want, tol = _swiglu(p, mags, n)
        got = y[:M].double()
        assert torch.isfinite(got).all()
        tol = tol + ref.half_step(DT[out], want.abs() + tol)
        assert ((got - want).abs() <= tol).all()
        if M:
            assert float((got - want).norm() / want.norm()) <= torch.finfo(DT[out]).eps / 2 + 1e-5
    # alpha left out is alpha of one
    one, none = torch.empty_like(y, dtype=torch.float32), torch.empty_like(y, dtype=torch.float32)
    one.fill_(3)
    none.fill_(3)
    q.moe_grouped_mm_fp4(xq, xs, wq.view(E, N, K // 2), wsc, off, one, fmt, ws,
                         alpha=torch.ones(E, device="cuda"), swiglu=swiglu)
    q.moe_grouped_mm_fp4(xq, xs, wq.view(E, N, K // 2), wsc, off, none, fmt, ws, swiglu=swiglu)
    assert torch.equal(one, none)
    _done(ws)


@pytest.mark.parametrize("fmt", FMT)
def test_nan_blocks_stay_in_their_row(fmt):
    counts, K, N = [127, 130, 2], 256, 160
    xq, xs, xv = _operand(counts, K, fmt, 1, True, fill=0)
    wq, wsc, wv = _operand([N] * 3, K, fmt, 2, False, fill=0)
    place, _ = ref.tile_places(counts, K, fmt)
    for r in (126, 127, 258):
        xs[int(place[r, 3])] = 255 if fmt == 0 else 0x7f
    place, _ = ref.tile_places([N] * 3, K, fmt)
    wsc[int(place[N + 7, 0])] = 255 if fmt == 0 else 0x7f
    off, ws = ref.offsets_of(counts).cuda(), q.make_grouped_workspace()
    y = torch.zeros(259, N, device="cuda")
    q.moe_grouped_mm_fp4(xq, xs, wq.view(3, N, K // 2), wsc, off, y, fmt, ws)
    want = torch.zeros(259, N, dtype=torch.bool, device="cuda")
    want[[126, 127, 258]] = True
    want[127:257, 7] = True
    assert torch.equal(y.isnan(), want)


@pytest.mark.parametrize("fmt", FMT)
def test_bad_offsets(fmt):
    K, N = 64, 48
    xq, xs, _ = _operand([9], K, fmt, 1, True)
    xs = torch.cat([xs, xs, xs, xs])
    wq, wsc, _ = _operand([N] * 3, K, fmt, 2, False)
    ws = q.make_grouped_workspace()
    for bad in ([0, 5, 3, 9], [-1, 4, 6, 9], [0, 4, 9, 10], [9, 6, 4, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y = torch.zeros(9, N, device="cuda")
        q.moe_grouped_mm_fp4(xq, xs, wq.view(3, N, K // 2), wsc, off, y, fmt, ws)
        assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
        x = torch.ones(9, K, device="cuda")
        q.moe_fp4_quantize(x, xq.clone(), xs.clone(), fmt, ws, offsets=off)
        assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
        q.moe_fp4_dequantize(xq, xs, x, fmt, ws, offsets=off)
        assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE


@pytest.mark.parametrize("T", [1, 5, 40, 150])
@pytest.mark.parametrize("fmt", FMT)
def test_layer_with_4bit_experts(fmt, T):
    """The routed layer with 4-bit experts, as its stage calls make it: route, permute, quantise
    into slot order, gate/up with SwiGLU, quantise, down, combine; captured once and replayed."""
    from workloads import gen
    d = gen.LayerDims(hidden=256, n_experts=12, top_k=3, inter=256, shared_inter=256)
    layer = q.DeviceLayer(gen.draw_layer(d, 0))
    H, I, E, K = d.hidden, d.inter, d.n_experts, d.top_k
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    gw, dws = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((E, 2 * I, H), (E, H, I)))
    ex = -6 if fmt else 0
    gws = q.make_grouped_workspace()

    def weights(w):
        n = w.shape[0] * w.shape[1]
        wq, sc = _bufs(n, w.shape[2], fmt, E, ragged=False)
        q.moe_fp4_quantize(0.02 * w.view(n, -1).float(), wq, sc, fmt, gws, n_groups=E, scale_exp=ex)
        v = torch.zeros(n, w.shape[2], device="cuda")
        q.moe_fp4_dequantize(wq, sc, v, fmt, gws, n_groups=E, scale_exp=ex)
        return wq.view(*w.shape[:2], -1), sc, v.view(w.shape).double()
    uq, us, uv = weights(gw)
    dq, ds, dv = weights(dws)
    M = T * K
    ids, perm, inv = (torch.zeros(M, dtype=torch.int32, device="cuda") for _ in range(3))
    w, sig = torch.zeros(T, K, device="cuda"), torch.zeros(T, device="cuda")
    counts, off = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
    xq, xs = _bufs(M, H, fmt, E)
    hq, hs = _bufs(M, I, fmt, E)
    h, y = (torch.zeros(M, n, dtype=torch.bfloat16, device="cuda") for n in (I, H))
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    ws = q.make_workspace(d, T)
    alpha = torch.full((E,), 2.0 ** ex, device="cuda")

    def run():
        q.moe_route(d, layer, x, ids.view(T, K), w, sig, ws)
        q.moe_permute(d, ids.view(T, K), counts, off, perm, inv, ws)
        q.moe_fp4_quantize(x, xq, xs, fmt, gws, offsets=off, perm=perm, top_k=K)
        q.moe_grouped_mm_fp4(xq, xs, uq, us, off, h, fmt, gws, alpha=alpha, swiglu=True)
        q.moe_fp4_quantize(h, hq, hs, fmt, gws, offsets=off)
        q.moe_grouped_mm_fp4(hq, hs, dq, ds, off, y, fmt, gws, alpha=alpha)
        q.moe_combine(d, layer, x, y, inv, w, sig, out, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(2):
        if k:
            x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        if k == 0:
            assert torch.equal(out, first)
        src = (perm // K).long().cpu().numpy()
        c, b = ref.quantize(x.double().cpu().numpy(), fmt)
        xv = torch.from_numpy(ref.values(c, b, fmt)).cuda()[torch.from_numpy(src).cuda()]
        p, mags = ref.mm(xv, uv, off)
        hv, tol = _swiglu(p, mags, H + 2)
        assert ((h.double() - hv).abs() <= tol + ref.half_step(torch.bfloat16, hv.abs() + tol)).all()
        c, b = ref.quantize(h.double().cpu().numpy(), fmt)
        assert np.array_equal(ref.unpack(hq.cpu().numpy()), c)
        p, mags = ref.mm(torch.from_numpy(ref.values(c, b, fmt)).cuda(), dv, off)
        ref.check(y, p, mags, I + 2)
        # the combine of these slots: the int4 shared expert alone (no routed part) added
        zero = torch.zeros_like(out)
        q.moe_combine(d, layer, x, torch.zeros_like(y), inv, w, sig, zero, ws)
        routed = (y.double()[inv.long()].view(T, K, H) * w.double()[..., None]).sum(1)
        want = routed + zero.double()
        # both outputs round once to bf16
        tol = ref.half_step(torch.bfloat16, want.abs()) + ref.half_step(torch.bfloat16, zero.double()) + 1e-4
        assert ((out.double() - want).abs() <= 1.01 * tol).all()
    _done(ws)
    _done(gws)


def test_binding_refusals():
    xq, xs, _ = _operand([4, 4], 64, 1, 1, True)
    wq, wsc, _ = _operand([32, 32], 64, 1, 2, False)
    wq = wq.view(2, 32, 32)
    off, ws = ref.offsets_of([4, 4]).cuda(), q.make_grouped_workspace()
    y = torch.zeros(8, 32, device="cuda")
    with pytest.raises(TypeError):
        q.moe_grouped_mm_fp4(xq.int(), xs, wq, wsc, off, y, 1, ws)
    with pytest.raises(ValueError, match="shape"):
        q.moe_grouped_mm_fp4(xq, xs, wq, wsc, off, y, 1, ws, swiglu=True)
    with pytest.raises(ValueError, match="offsets"):
        q.moe_grouped_mm_fp4(xq, xs, wq, wsc, off[:2].contiguous(), y, 1, ws)
    with pytest.raises(q.StrataError):
        q.moe_grouped_mm_fp4(xq, xs[:16], wq, wsc, off, y, 1, ws)
    with pytest.raises(q.StrataError):
        q.moe_fp4_quantize(torch.zeros(8, 48, device="cuda"), torch.zeros(8, 24, dtype=torch.uint8,
                                                                          device="cuda"), xs, 1, ws)
    with pytest.raises(TypeError):
        q.moe_fp4_quantize(torch.zeros(8, 64, dtype=torch.int32, device="cuda"), xq, xs, 1, ws)
    with pytest.raises(ValueError, match="perm"):
        q.moe_fp4_quantize(torch.zeros(8, 64, device="cuda"), xq, xs, 1, ws,
                           perm=torch.zeros(8, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("out", DT)
def test_swiglu_of_gates_far_below_zero(out):
    """Gates from -110 to 110, each with an up value that brings the result near one where a power of
    two up to 2^120 can: e^-g passes 2^126 at -87.3 and leaves fp32 at -88.7, the result does not."""
    gates = np.arange(-220, 221) / 2.0
    I, K = len(gates), 32
    silu = gates / (1 + np.exp(-gates))
    up = np.clip(-np.round(np.log2(np.abs(silu) + 1e-60)), -100, 120)
    codes = np.zeros((2 * I, K), dtype=np.uint8)
    byte = np.full((2 * I, 1), 127, dtype=np.uint8)
    for i, g in enumerate(gates):                       # the gate row adds up to g
        left = abs(g)
        for k in range(K):
            c = int(np.searchsorted(ref.GRID, min(left, 6.0), side="right")) - 1
            codes[2 * i, k] = c + (8 if g < 0 and c else 0)
            left -= ref.GRID[c]
        assert left == 0
        codes[2 * i + 1, 0] = 2                         # one times the scale
        byte[2 * i + 1] = 127 + int(up[i])
    wsc = torch.from_numpy(ref.tiled(byte, [2 * I], K, 0, q.moe_fp4_scale_bytes(0, 2 * I, K))).cuda()
    xs = torch.from_numpy(ref.tiled(np.full((1, 1), 127), [1], K, 0, 512)).cuda()
    xq = torch.full((1, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    off, ws = ref.offsets_of([1]).cuda(), q.make_grouped_workspace()
    y = torch.full((1, I), 7.0, dtype=DT[out], device="cuda")
    q.moe_grouped_mm_fp4(xq, xs, torch.from_numpy(ref.pack(codes)).cuda()[None], wsc, off, y, 0, ws,
                         swiglu=True)
    u = np.exp2(up)
    want = torch.from_numpy(silu * u)
    # the exponential: 2 + 1.173 |g| steps (__expf's bound; expf's is smaller) and, below its normal
    # range, two of the smallest ones; 8 steps for the rest
    tol = torch.from_numpy((10 + 1.173 * np.abs(gates)) * 2.0 ** -23 * np.abs(silu * u)
                           + np.abs(gates) * u * 2.0 ** -148)
    tol = tol + ref.half_step(DT[out], want.abs() + tol)
    err = (y[0].double().cpu() - want).abs()
    bad = torch.nonzero(~(err <= tol)).flatten()
    assert not len(bad), [(gates[i], float(y[0, i]), float(want[i])) for i in bad[:8]]
    _done(ws)


@pytest.mark.parametrize("fmt", FMT)
def test_rows_before_the_first_group(fmt):
    """Rows before the first and behind the last group hold NaN and stay as they were; the groups' row
    blocks of scales are counted from the first group."""
    counts, first, spare, C, N = [130, 0, 1, 40], 5, 7, 160, 96
    M = first + sum(counts) + spare
    live = slice(first, M - spare)
    x = _rows(M, C, "bf16", 8, fmt)
    codes, sb = ref.quantize(x[live].double().numpy(), fmt)
    x[:first], x[M - spare:] = float("nan"), float("nan")
    off, ws = ref.offsets_of(counts, first).cuda(), q.make_grouped_workspace()
    qd, sc = _bufs(M, C, fmt, len(counts))
    q.moe_fp4_quantize(x.cuda(), qd, sc, fmt, ws, offsets=off)
    place, used = ref.tile_places(counts, C, fmt)
    got, scb = qd.cpu().numpy(), sc.cpu().numpy()
    assert np.array_equal(ref.unpack(got[live]), codes) and np.array_equal(scb[place], sb)
    assert (got[:first] == 0xAB).all() and (got[M - spare:] == 0xAB).all() and (scb[used:] == 0xAB).all()
    v = torch.full((M, C), 7.0, device="cuda")
    q.moe_fp4_dequantize(qd, sc, v, fmt, ws, offsets=off)
    values = torch.from_numpy(ref.values(codes, sb, fmt)).cuda()
    assert torch.equal(v[live].double(), values)
    assert (v[:first] == 7).all() and (v[M - spare:] == 7).all()
    wq, wsc, wv = _operand([N] * len(counts), C, fmt, 2, False)
    y = torch.full((M, N), 7.0, device="cuda")
    q.moe_grouped_mm_fp4(qd, sc, wq.view(len(counts), N, C // 2), wsc, off, y, fmt, ws)
    want, mags = ref.mm(values, wv.view(len(counts), N, C), ref.offsets_of(counts))
    ref.check(y[live], want, mags, C)
    assert (y[:first] == 7).all() and (y[M - spare:] == 7).all()
    _done(ws)
