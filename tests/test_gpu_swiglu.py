"""SwiGLU in the grouped products' epilogues, forward and backward, against 64-bit
plain forms: every kernel's borders, p kept in both forms, masks and refusals."""
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import grouped_ref as ref
from tests import step_ref as step

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}

# rows of each group; K (the other width of the product), I
SHAPES = {
    "one_row": ([1], 64, 32),
    "token": ([0, 1, 1, 0, 0, 1, 0, 1], 512, 192),
    "few_rows": ([0, 5, 0, 3], 1032, 77),
    "nine_rows": ([4, 5], 264, 48),
    "empty_ends": ([0, 0, 5, 0, 130, 0], 256, 160),
    "tile_edges": ([127, 128, 129, 1, 255, 257], 192, 72),
    "one_group": ([700], 1024, 264),
    "all_empty": ([0, 0, 0], 128, 64),
    "odd_wide": ([3, 64, 17, 0, 65], 200, 505),
    "narrow": ([9, 0, 40], 8, 8),
    "unaligned": ([5, 33, 0, 2], 37, 51),
    "unaligned_few": ([1, 0, 2], 37, 3),
    "one_by_one": ([2, 30], 1, 1),
    "long": ([40, 300, 7], 2560, 136),
    "longer": ([3, 140], 4168, 272),
    # reductions of several pieces in long groups, and in many groups of one tile
    "long_wide": ([900, 1200, 40], 2184, 520),
    "long_each": ([100 + e % 7 for e in range(60)], 2184, 520),
    "many": ([(7 * e) % 11 for e in range(300)], 128, 40),
    "long_groups": ([1500, 0, 777, 2048, 1], 320, 136),
    "long_even": ([1024, 512], 512, 512),
    "few_tiles": ([40, 1], 4096, 144),
    "one_tile": ([100], 1048, 50),
    "mid_groups": ([300, 129, 0, 1, 256, 255, 400, 350], 200, 80),
    "long_many": ([640 + 37 * (e % 5) for e in range(40)], 256, 200),
}
KEPT = ["none", "16", "8"]


def _case(name, dtype, spare=0, first=0):
    counts, K, I = SHAPES[name]
    g = torch.Generator(device="cuda").manual_seed(17 + len(name))
    E, M = len(counts), first + sum(counts) + spare

    def draw(*s, scale=1.0):
        return (scale * torch.randn(*s, generator=g, device="cuda")).to(DT[dtype])
    # p of unit size, so that gates pass through SwiGLU's bend
    return dict(x=draw(M, K), w=draw(E, 2 * I, K, scale=K ** -0.5), dy=draw(M, K), wd=draw(E, K, I, scale=K ** -0.5),
                p=draw(M, 2 * I, scale=1.5), off=ref.offsets_of(counts, first).cuda(), ws=q.make_grouped_workspace(),
                M=M, K=K, I=I, n=sum(counts), first=first)


def _fill(*s, dtype, value=7):
    return torch.full(s, value, dtype=dtype, device="cuda")


def _done(ws):
    assert q.moe_get_device_status(ws) == q.STRATA_OK


def _check_kept8(pq, ps, p, err, rows):
    """Each block's scale is the one of its largest value or, where the sums' error lies across the
    border, its neighbour; each value is within half a step of its own, or of the scale's smallest."""
    vals = torch.from_numpy(step.act8_load(pq.cpu().numpy(), ps.cpu().numpy())).cuda()[rows]
    b, want, e = ps[rows].double(), p[rows], err[rows]
    m, em = (t.abs().unflatten(1, (-1, 32)).amax(dim=2) for t in (want, e))
    s = torch.exp2(b - 127)
    assert ((m - em <= 448 * s) & ((m + em > 224 * s) | (b == 1))).all()
    half = torch.maximum(2.0 ** -4 * (want.abs() + e), (2.0 ** -10 * s).repeat_interleave(32, dim=1))
    assert ((vals - want).abs() <= half + e).all()


@pytest.mark.parametrize("kept", KEPT)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("name", SHAPES)
def test_forward(name, dtype, kept):
    c = _case(name, dtype)
    if kept == "8" and c["I"] % 16:
        pytest.skip("8 bits need a width of a multiple of 32")
    h = _fill(c["M"], c["I"], dtype=DT[dtype])
    p = ps = None
    if kept != "none":
        p = _fill(c["M"], 2 * c["I"], dtype=DT[dtype] if kept == "16" else torch.uint8)
        ps = _fill(c["M"], 2 * c["I"] // 32, dtype=torch.uint8) if kept == "8" else None
    q.moe_grouped_swiglu(c["x"], c["w"], c["off"], h, c["ws"], p=p, p_scales=ps)
    want, mags = ref.mm(c["x"], c["w"], c["off"])
    err = ref.sum_error(c["K"], mags)
    step.near(h, *step.swiglu(want, err), what=name)
    if kept == "16":
        ref.check(p, want, mags, c["K"], name)
    elif kept == "8":
        _check_kept8(p, ps, want, err, torch.arange(c["M"], device="cuda"))
    again = torch.empty_like(h)
    q.moe_grouped_swiglu(c["x"], c["w"], c["off"], again, c["ws"], p=p, p_scales=ps)
    assert torch.equal(h, again)
    _done(c["ws"])


def _kept(c, kept):
    """(p or its codes, scales, the values they stand for)."""
    if kept != "8":
        return c["p"], None, c["p"].double()
    pq = torch.zeros(c["M"], 2 * c["I"], dtype=torch.uint8, device="cuda")
    ps = torch.zeros(c["M"], 2 * c["I"] // 32, dtype=torch.uint8, device="cuda")
    q.moe_act8_save(c["p"], pq, ps)
    return pq, ps, torch.from_numpy(step.act8_load(pq.cpu().numpy(), ps.cpu().numpy())).cuda()


@pytest.mark.parametrize("kept", KEPT[1:])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("name", SHAPES)
def test_backward(name, dtype, kept):
    c = _case(name, dtype)
    if kept == "8" and c["I"] % 16:
        pytest.skip("8 bits need a width of a multiple of 32")
    p, ps, vals = _kept(c, kept)
    dp, h = _fill(c["M"], 2 * c["I"], dtype=DT[dtype]), _fill(c["M"], c["I"], dtype=DT[dtype])
    q.moe_grouped_swiglu_bwd(c["dy"], c["wd"], p, c["off"], dp, c["ws"], p_scales=ps, h=h)
    dh, mags = ref.dx(c["dy"], c["wd"], c["off"])
    want_dp, want_h = step.swiglu_back(dh, ref.sum_error(c["K"], mags), vals)
    step.near(dp, *want_dp, what=name + " dp")
    step.near(h, *want_h, what=name + " h")
    alone = torch.empty_like(dp)
    q.moe_grouped_swiglu_bwd(c["dy"], c["wd"], p, c["off"], alone, c["ws"], p_scales=ps)
    assert torch.equal(dp, alone)
    _done(c["ws"])


@pytest.mark.parametrize("name", ["token", "few_rows", "empty_ends", "tile_edges", "odd_wide", "unaligned",
                                  "long_groups", "few_tiles"])
def test_rows_of_no_group_keep_what_they_held(name):
    """Rows before the first group and behind the last hold NaN in every input."""
    c = _case(name, "bf16", spare=37, first=3)
    out = torch.ones(c["M"], dtype=torch.bool, device="cuda")
    out[3:3 + c["n"]] = False
    for t in ("x", "dy", "p"):
        c[t][out] = float("nan")
    h, p = _fill(c["M"], c["I"], dtype=torch.bfloat16), _fill(c["M"], 2 * c["I"], dtype=torch.bfloat16)
    h2, dp = h.clone(), p.clone()
    q.moe_grouped_swiglu(c["x"], c["w"], c["off"], h, c["ws"], p=p)
    q.moe_grouped_swiglu_bwd(c["dy"], c["wd"], c["p"], c["off"], dp, c["ws"], h=h2)
    for t in (h, p, h2, dp):
        assert (t[out] == 7).all()
    live = ~out
    want, mags = ref.mm(c["x"], c["w"], c["off"])
    step.near(h[live], *(t[live] for t in step.swiglu(want, ref.sum_error(c["K"], mags))))
    dh, mags = ref.dx(c["dy"], c["wd"], c["off"])
    (want, err), _ = step.swiglu_back(dh[live], ref.sum_error(c["K"], mags)[live], c["p"][live].double())
    step.near(dp[live], want, err)
    if c["I"] % 16 == 0:
        pq = _fill(c["M"], 2 * c["I"], dtype=torch.uint8)
        ps = _fill(c["M"], 2 * c["I"] // 32, dtype=torch.uint8)
        q.moe_grouped_swiglu(c["x"], c["w"], c["off"], h, c["ws"], p=pq, p_scales=ps)
        assert (pq[out] == 7).all() and (ps[out] == 7).all()
    _done(c["ws"])


@pytest.mark.parametrize("name", ["few_rows", "nine_rows", "unaligned", "one_group"])
def test_gates_far_out_and_rows_with_infinities(name):
    """Gates of -110 to 110 (one product a row, exact), up values of up to 2^100; an infinity or a NaN
    stays in its row."""
    counts, K, I = SHAPES[name]
    c = _case(name, "bf16")
    M = c["M"]
    gates = torch.linspace(-110, 110, I, device="cuda").bfloat16()
    c["x"].zero_()
    c["x"][:, 0] = 1
    c["w"].zero_()
    c["w"][:, 0::2, 0] = gates
    c["w"][:, 1::2, 0] = torch.where(torch.arange(I, device="cuda") % 2 == 0, 1.0, 2.0 ** 100).bfloat16()
    c["x"][M // 2, 0] = float("inf")
    c["x"][M // 3, 0] = float("nan")
    h = _fill(M, I, dtype=torch.bfloat16)
    q.moe_grouped_swiglu(c["x"], c["w"], c["off"], h, c["ws"])
    live = torch.ones(M, dtype=torch.bool, device="cuda")
    live[M // 2] = live[M // 3] = False
    p = (c["x"][live, :1].double() * c["w"][0, :, 0].double())
    want, err = step.swiglu(p, torch.zeros_like(p))
    # e^g of gates below -87.3 is denormal: off by a step of 2^-149 where it is taken
    err = err + 2.0 ** -148 * p[:, 1::2].abs() * 110
    step.near(h[live], want, err)
    assert torch.isnan(h[M // 3]).all()
    _done(c["ws"])


def test_back_through_gates_far_out():
    g = torch.linspace(-110, 110, 64, device="cuda").bfloat16()
    p = torch.ones(9, 128, device="cuda", dtype=torch.bfloat16)
    p[:, 0::2] = g
    dy = torch.ones(9, 8, device="cuda", dtype=torch.bfloat16)
    w = torch.full((1, 8, 64), 0.125, device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    dp, ws = torch.empty_like(p), q.make_grouped_workspace()
    q.moe_grouped_swiglu_bwd(dy, w, p, off, dp, ws)
    one = torch.ones(9, 64, device="cuda", dtype=torch.float64)
    (want, err), _ = step.swiglu_back(one, 0 * one, p.double())
    step.near(dp, want, err + 2.0 ** -148 * 110)


@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [0, 4, 8, 11], [-1, 2, 4, 9]])
@pytest.mark.parametrize("K", [64, 37])
def test_bad_offsets_empty_the_call(bad, K):
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    x = torch.ones(10, K, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(3, 64, K, dtype=torch.bfloat16, device="cuda")
    for rows in (10, 8):
        ws = q.make_grouped_workspace()
        h = _fill(rows, 32, dtype=torch.bfloat16)
        q.moe_grouped_swiglu(x[:rows], w, off, h, ws)
        assert (h == 7).all() and q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
        dp = _fill(rows, 2 * K, dtype=torch.bfloat16)
        q.moe_grouped_swiglu_bwd(torch.ones(rows, 64, dtype=torch.bfloat16, device="cuda"),
                                 w, _fill(rows, 2 * K, dtype=torch.bfloat16), off, dp, ws)
        assert (dp == 7).all() and q.moe_get_device_status(ws) == q.STRATA_EBADROUTE


@pytest.mark.parametrize("shift", [8, 24])
@pytest.mark.parametrize("name", ["token", "empty_ends", "one_group", "few_tiles"])
def test_tensors_aligned_to_16_bytes_only(name, shift):
    """Every tensor starts 16 (48) bytes behind an aligned address."""
    c = _case(name, "bf16")

    def moved(t):
        buf = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        v = buf[shift:].view(t.shape)
        v.copy_(t)
        return v
    out = {}
    for kind, f in (("plain", lambda t: t), ("moved", moved)):
        h, p = f(_fill(c["M"], c["I"], dtype=torch.bfloat16)), f(_fill(c["M"], 2 * c["I"], dtype=torch.bfloat16))
        dp, h2 = f(p.clone()), f(h.clone())
        q.moe_grouped_swiglu(f(c["x"]), f(c["w"]), c["off"], h, c["ws"], p=p)
        q.moe_grouped_swiglu_bwd(f(c["dy"]), f(c["wd"]), f(c["p"]), c["off"], dp, c["ws"], h=h2)
        out[kind] = [h, p, dp, h2]
    for a, b in zip(out["plain"], out["moved"]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("K", [4096, 1 << 15])
@pytest.mark.parametrize("rows", [6, 40])
def test_long_sums_of_one_sign(K, rows):
    """p of terms of one sign: in pieces, each off by at most 2e-5 of the sum (a truncating accumulator
    of the whole length loses 1e-7 of it with every 16 terms: 2e-4 at 2^15)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.rand(rows, K, generator=g, device="cuda") + 0.5).half()
    w = ((torch.rand(1, 32, K, generator=g, device="cuda") + 0.5) * (2.0 / K)).half()
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    h, p = (torch.empty(rows, n, dtype=torch.float16, device="cuda") for n in (16, 32))
    q.moe_grouped_swiglu(x, w, off, h, q.make_grouped_workspace(), p=p)
    want, mags = ref.mm(x, w, off)
    err = 2e-5 * mags
    step.near(p, want, err)
    step.near(h, *step.swiglu(want, err))


def test_captured_with_other_offsets_and_a_workspace_each():
    """Two captured graphs on two streams, replayed together with new offsets and inputs."""
    c = [_case("mid_groups", "bf16"), _case("token", "bf16")]
    outs, graphs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for k, s in zip(c, streams):
        k["h"], k["pk"] = _fill(k["M"], k["I"], dtype=torch.bfloat16), _fill(k["M"], 2 * k["I"], dtype=torch.bfloat16)
        k["dp"] = k["pk"].clone()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            def step_once(k=k):
                q.moe_grouped_swiglu(k["x"], k["w"], k["off"], k["h"], k["ws"], p=k["pk"])
                q.moe_grouped_swiglu_bwd(k["dy"], k["wd"], k["pk"], k["off"], k["dp"], k["ws"])
            step_once()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step_once()
            graphs.append(g)
    torch.cuda.synchronize()
    for k in c:                                  # the same rows in reversed groups
        n = (k["off"][1:] - k["off"][:-1]).flip(0)
        k["off"][1:] = n.cumsum(0)
        k["x"].mul_(-0.5)
    torch.cuda.synchronize()
    for g, s in zip(graphs * 3, streams * 3):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for k in c:
        want, mags = ref.mm(k["x"], k["w"], k["off"])
        err = ref.sum_error(k["K"], mags)
        step.near(k["h"], *step.swiglu(want, err))
        dh, mags = ref.dx(k["dy"], k["wd"], k["off"])
        (dp, err), _ = step.swiglu_back(dh, ref.sum_error(k["K"], mags), k["pk"].double())
        step.near(k["dp"], dp, err)
        _done(k["ws"])


def test_binding_refuses():
    c = _case("token", "bf16")
    h, dp = torch.empty(c["M"], c["I"], dtype=torch.bfloat16, device="cuda"), torch.empty_like(c["p"])
    u8 = torch.empty(c["M"], 2 * c["I"], dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError, match="one type"):
        q.moe_grouped_swiglu(c["x"], c["w"].half(), c["off"], h, c["ws"])
    with pytest.raises(TypeError, match="p must be"):
        q.moe_grouped_swiglu(c["x"], c["w"], c["off"], h, c["ws"], p=u8)
    with pytest.raises(ValueError, match="p_scales"):
        q.moe_grouped_swiglu(c["x"], c["w"], c["off"], h, c["ws"], p=u8, p_scales=u8)
    with pytest.raises(ValueError, match="contiguous"):
        q.moe_grouped_swiglu(c["x"], c["w"].transpose(1, 2).contiguous().transpose(1, 2), c["off"], h, c["ws"])
    with pytest.raises(ValueError, match="gate and an up"):
        q.moe_grouped_swiglu(c["x"], c["w"][:, :3].contiguous(), c["off"], h, c["ws"])
    with pytest.raises(ValueError, match="entries"):
        q.moe_grouped_swiglu_bwd(c["dy"], c["wd"], c["p"], c["off"][:4].contiguous(), dp, c["ws"])
    with pytest.raises(ValueError, match="h must"):
        q.moe_grouped_swiglu_bwd(c["dy"], c["wd"], c["p"], c["off"], dp, c["ws"], h=dp)
    with pytest.raises(ValueError, match="one device|workspace's device"):
        q.moe_grouped_swiglu(c["x"].cpu(), c["w"], c["off"], h, c["ws"])
