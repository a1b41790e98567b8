"""Products grouped by expert on the GPU against 64-bit plain forms."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_fwd_gb300 as q
from tests import grouped_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# rows of each group; K, N.  One row, no rows, rows around the tile heights, all rows in one
# group, widths that are no multiple of any tile, of 8, and long reductions.
SHAPES = {
    "one_row": ([1], 64, 64),
    "token": ([0, 1, 1, 0, 0, 1, 0, 1], 512, 384),
    "empty_ends": ([0, 0, 5, 0, 130, 0], 256, 320),
    "tile_edges": ([127, 128, 129, 1, 255, 257], 192, 136),
    "one_group": ([700], 1024, 520),
    "all_empty": ([0, 0, 0], 128, 128),
    "odd_wide": ([3, 64, 17, 0, 65], 200, 1000),
    "narrow": ([9, 0, 40], 8, 8),
    "unaligned": ([5, 33, 0, 2], 37, 51),
    "unaligned_k": ([130, 1], 66, 64),
    "one_by_one": ([2, 3], 1, 1),
    "long": ([40, 300, 7], 2560, 264),
    "many": ([(7 * e) % 11 for e in range(300)], 128, 72),
    # long groups (512 rows on average and more), some of them ragged, empty or a single row
    "long_groups": ([1500, 0, 777, 2048, 1], 320, 264),
    "long_even": ([1024, 512], 512, 1024),
    # few tiles and long reductions, in every direction; the last parts of a split are short
    "few_tiles": ([40, 1], 4096, 264),
    "few_tiles_back": ([33, 0, 12], 200, 3016),
    "one_tile": ([100], 1048, 100),
    "narrow_out": ([60, 9, 130], 1992, 3),
    "narrow_many": ([(5 * e) % 9 for e in range(200)], 1048, 4),
    "mid_groups": ([300, 129, 0, 1, 256, 255, 400, 350], 200, 144),
    "long_many": ([640 + 37 * (e % 5) for e in range(40)], 256, 392),
}
SEED = 11


def _case(name, dtype, spare=0, first=0, scale=1.0):
    counts, K, N = SHAPES[name]
    g = torch.Generator(device="cuda").manual_seed(SEED + len(name))
    E, M = len(counts), first + sum(counts) + spare

    def draw(*s):
        return (scale * torch.randn(*s, generator=g, device="cuda")).to(DT[dtype])
    return (draw(M, K), draw(E, N, K), draw(M, N), ref.offsets_of(counts, first).cuda(),
            q.make_grouped_workspace())


def _done(ws):
    assert q.moe_get_device_status(ws) == q.STRATA_OK


TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")]


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("name", SHAPES)
def test_forward(name, dtype, out):
    x, w, _, off, ws = _case(name, dtype)
    y = torch.full((x.shape[0], w.shape[1]), 7.0, dtype=DT[out], device="cuda")
    q.moe_grouped_mm(x, w, off, y, ws)
    want, mags = ref.mm(x, w, off)
    ref.check(y, want, mags, w.shape[2], name)
    _done(ws)


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("name", SHAPES)
def test_dx(name, dtype, out):
    x, w, dy, off, ws = _case(name, dtype)
    dx = torch.full(x.shape, 7.0, dtype=DT[out], device="cuda")
    q.moe_grouped_mm_dx(dy, w, off, dx, ws)
    want, mags = ref.dx(dy, w, off)
    ref.check(dx, want, mags, w.shape[1], name)
    _done(ws)


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("name", SHAPES)
def test_dw(name, dtype, out):
    x, w, dy, off, ws = _case(name, dtype)
    dw = torch.full(w.shape, 7.0, dtype=DT[out], device="cuda")
    q.moe_grouped_mm_dw(dy, x, off, dw, ws)
    want, mags = ref.dw(dy, x, off)
    ref.check(dw, want, mags, max(SHAPES[name][0]), name)
    again = torch.empty_like(dw)
    q.moe_grouped_mm_dw(dy, x, off, again, ws)
    assert torch.equal(dw, again)
    _done(ws)


def test_no_rows():
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = q.make_grouped_workspace()
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(3, 32, 64, dtype=torch.bfloat16, device="cuda")
    q.moe_grouped_mm(x, w, off, torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), ws)
    dw = torch.full((3, 32, 64), 5.0, device="cuda")
    q.moe_grouped_mm_dw(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), x, off, dw, ws)
    assert torch.equal(dw, torch.zeros_like(dw))
    _done(ws)


def test_few_rows_of_no_group_and_nan():
    """The kernel for a few rows: rows of no group, and a row of NaN beside finite ones."""
    counts, first, spare = [1, 0, 2, 1], 1, 2
    off = ref.offsets_of(counts, first).cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(7, 520, generator=g, device="cuda").half()
    w = torch.randn(4, 37, 520, generator=g, device="cuda").half()
    x[0], x[5:] = float("nan"), float("nan")
    y = torch.full((7, 37), 7.0, dtype=torch.float16, device="cuda")
    ws = q.make_grouped_workspace()
    q.moe_grouped_mm(x, w, off, y, ws)
    want, mags = ref.mm(x, w, off)
    assert (y[0] == 7).all() and (y[5:] == 7).all()
    ref.check(y[1:5], want[1:5], mags[1:5], 520)
    x[2, 519] = float("inf")
    q.moe_grouped_mm(x, w, off, y, ws)
    assert not torch.isfinite(y[2]).any()
    ref.check(y[[1, 3, 4]], want[[1, 3, 4]], mags[[1, 3, 4]], 520)
    for bad in ([1, 2, 1, 4, 5], [1, 2, 2, 4, 8]):
        y.fill_(7)
        q.moe_grouped_mm(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), y, ws)
        assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE and (y == 7).all()


@pytest.mark.parametrize("name", ["tile_edges", "token", "odd_wide", "unaligned", "narrow_out", "few_tiles",
                                  "long_groups"])
def test_rows_of_no_group_are_neither_read_nor_written(name):
    """Rows before the first and behind the last group hold NaN; outputs there stay."""
    first, spare = 3, 70
    x, w, dy, off, ws = _case(name, "bf16", spare=spare, first=first)
    M = x.shape[0]
    for t in (x, dy):
        t[:first] = float("nan")
        t[M - spare:] = float("nan")
    y = torch.full((M, w.shape[1]), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full(w.shape, 7.0, device="cuda")
    q.moe_grouped_mm(x, w, off, y, ws)
    q.moe_grouped_mm_dx(dy, w, off, dx, ws)
    q.moe_grouped_mm_dw(dy, x, off, dw, ws)
    live = slice(first, M - spare)
    for got, (want, mags), n in ((y, ref.mm(x, w, off), w.shape[2]), (dx, ref.dx(dy, w, off), w.shape[1])):
        assert (got[:first] == 7).all() and (got[M - spare:] == 7).all()
        ref.check(got[live], want[live], mags[live], n, name)
    want, mags = ref.dw(dy, x, off)
    ref.check(dw, want, mags, max(SHAPES[name][0]), name)
    _done(ws)


def test_a_row_of_nan_stays_in_its_row_and_group():
    x, w, dy, off, ws = _case("tile_edges", "bf16")
    rows = [int(off[2]) - 1, int(off[3])]               # the last row of a group, a group of one
    for t in (x, dy):
        t[rows[0]] = float("nan")
        t[rows[1], 5] = float("inf")
    y = torch.zeros(x.shape[0], w.shape[1], device="cuda")
    dx = torch.zeros(x.shape, device="cuda")
    dw = torch.zeros(w.shape, device="cuda")
    q.moe_grouped_mm(x, w, off, y, ws)
    q.moe_grouped_mm_dx(dy, w, off, dx, ws)
    q.moe_grouped_mm_dw(dy, x, off, dw, ws)
    rest = torch.ones(x.shape[0], dtype=torch.bool, device="cuda")
    rest[rows] = False
    for got in (y, dx):
        assert torch.isfinite(got[rest]).all() and got[rows[0]].isnan().all()
        assert not torch.isfinite(got[rows[1]]).any()
    touched = [1, 3]
    assert all(torch.isfinite(dw[e]).all() == (e not in touched) for e in range(6))
    assert dw[1].isnan().all()
    _done(ws)


@pytest.mark.parametrize("name", ["token", "tile_edges"])
def test_gradients_against_differences(name):
    """With values on a grid of 1/8 every product and sum below 2^24 / 64 is exact, so the forward's
    difference quotient in a direction equals the gradient's product with it, bit for bit."""
    counts, K, N = SHAPES[name]
    g = torch.Generator(device="cuda").manual_seed(5)

    def draw(*s):
        return (torch.randint(-16, 17, s, generator=g, device="cuda") / 8).to(torch.bfloat16)
    E, M = len(counts), sum(counts)
    off, ws = ref.offsets_of(counts).cuda(), q.make_grouped_workspace()
    x, w, c, px, pw = draw(M, K), draw(E, N, K), draw(M, N), draw(M, K), draw(E, N, K)

    def loss(x, w):
        y = torch.zeros(M, N, device="cuda")
        q.moe_grouped_mm(x, w, off, y, ws)
        return (y.double() * c.double()).sum()
    dx = torch.zeros(M, K, device="cuda")
    dw = torch.zeros(E, N, K, device="cuda")
    q.moe_grouped_mm_dx(c, w, off, dx, ws)
    q.moe_grouped_mm_dw(c, x, off, dw, ws)
    assert (loss(x + px, w) - loss(x - px, w)) / 2 == (dx.double() * px.double()).sum()
    assert (loss(x, w + pw) - loss(x, w - pw)) / 2 == (dw.double() * pw.double()).sum()
    _done(ws)


@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [-1, 4, 6, 9], [0, 4, 9, 10], [9, 6, 4, 0],
                                 [0, 9, 0, 9]], ids=str)
def test_bad_offsets_are_reported_and_harmless(bad):
    """Backward or outside offsets: the call is reported and treats every group as empty."""
    x = torch.randn(9, 64, device="cuda").bfloat16()
    w = torch.randn(3, 32, 64, device="cuda").bfloat16()
    off, ws = torch.tensor(bad, dtype=torch.int32, device="cuda"), q.make_grouped_workspace()
    y = torch.full((9, 32), 7.0, device="cuda")
    dx = torch.full((9, 64), 7.0, device="cuda")
    dw = torch.full((3, 32, 64), 7.0, device="cuda")
    for call in (lambda: q.moe_grouped_mm(x, w, off, y, ws),
                 lambda: q.moe_grouped_mm_dx(y.bfloat16(), w, off, dx, ws),
                 lambda: q.moe_grouped_mm_dw(y.bfloat16(), x, off, dw, ws)):
        call()
        assert q.moe_get_device_status(ws) == q.STRATA_EBADROUTE
        assert q.moe_get_device_status(ws) == q.STRATA_OK
    assert (y == 7).all() and (dx == 7).all() and (dw == 0).all()


def test_graph_replays_follow_the_offsets():
    """Captured once; replayed with other offsets and inputs in the same buffers."""
    K, N, M = 256, 192, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(5, N, K, generator=g, device="cuda").bfloat16()
    off, ws = ref.offsets_of([10, 0, 200, 60, 30]).cuda(), q.make_grouped_workspace()
    y, dx, dw = (torch.zeros(s, device="cuda") for s in ((M, N), (M, K), (5, N, K)))
    dy = torch.randn(M, N, generator=g, device="cuda").bfloat16()

    def step():
        q.moe_grouped_mm(x, w, off, y, ws)
        q.moe_grouped_mm_dx(dy, w, off, dx, ws)
        q.moe_grouped_mm_dw(dy, x, off, dw, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for counts in ([300, 0, 0, 0, 0], [1, 2, 3, 4, 5], [0, 0, 129, 171, 0]):
        off.copy_(ref.offsets_of(counts))
        x.copy_(torch.randn(M, K, generator=g, device="cuda"))
        y.fill_(7)
        graph.replay()
        n = sum(counts)
        want, mags = ref.mm(x, w, off)
        ref.check(y[:n], want[:n], mags[:n], K)
        assert (y[n:] == 7).all()
        want, mags = ref.dx(dy, w, off)
        ref.check(dx[:n], want[:n], mags[:n], N)
        want, mags = ref.dw(dy, x, off)
        ref.check(dw, want, mags, max(counts))
    _done(ws)


def test_two_streams_with_a_workspace_each():
    args = [_case(n, "bf16") for n in ("long", "tile_edges")]
    streams = [torch.cuda.Stream() for _ in args]
    outs = [torch.zeros(a[0].shape[0], a[1].shape[1], device="cuda") for a in args]
    torch.cuda.synchronize()
    for _ in range(10):
        for (x, w, _, off, ws), s, y in zip(args, streams, outs):
            q.moe_grouped_mm(x, w, off, y, ws, stream=s)
    torch.cuda.synchronize()
    for (x, w, _, off, ws), y in zip(args, outs):
        want, mags = ref.mm(x, w, off)
        ref.check(y, want, mags, w.shape[2])
        _done(ws)


def test_binding_refusals():
    x, w, dy, off, ws = _case("tile_edges", "bf16")
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        q.moe_grouped_mm(x.float(), w, off, y, ws)
    with pytest.raises(TypeError):
        q.moe_grouped_mm(x, w.half(), off, y, ws)
    with pytest.raises(TypeError):
        q.moe_grouped_mm(x, w, off, y.half(), ws)
    with pytest.raises(ValueError, match="shape"):
        q.moe_grouped_mm(x, w, off, y[:-1], ws)
    with pytest.raises(ValueError, match="contiguous"):
        q.moe_grouped_mm(x.repeat(1, 2)[:, ::2], w, off, y, ws)
    with pytest.raises(ValueError, match="offsets"):
        q.moe_grouped_mm(x, w, off[:-1].contiguous(), y, ws)
    with pytest.raises(ValueError, match="offsets"):
        q.moe_grouped_mm(x, w, off.long(), y, ws)
    with pytest.raises(ValueError, match="device"):
        q.moe_grouped_mm(x.cpu(), w, off, y, ws)
    with pytest.raises(q.StrataError) as e:
        q.moe_grouped_mm(x, w, off, y, ws[:256])
    assert e.value.status == q.STRATA_EINVAL
    with pytest.raises(q.StrataError):
        q.moe_grouped_mm(x, w, off, torch.zeros(y.numel() + 1, dtype=y.dtype, device="cuda")[1:]
                         .view(y.shape), ws)


def test_large_places():
    """Weights and outputs whose element places pass 2^31 in bytes and elements."""
    E, N, K = 1024, 1024, 2304                          # 2.4e9 weights
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    w[-1] = last
    x = torch.randn(5, K, generator=g, device="cuda").bfloat16()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 5
    ws = q.make_grouped_workspace()
    y = torch.zeros(5, N, device="cuda")
    q.moe_grouped_mm(x, w, off, y, ws)
    want, mags = ref.mm(x, last[None], torch.tensor([0, 5]))
    ref.check(y, want, mags, K)
    dx = torch.zeros(5, K, device="cuda")
    dy = torch.randn(5, N, generator=g, device="cuda").bfloat16()
    q.moe_grouped_mm_dx(dy, w, off, dx, ws)
    want, mags = ref.dx(dy, last[None], torch.tensor([0, 5]))
    ref.check(dx, want, mags, N)
    dw = w                                              # reused as the output
    q.moe_grouped_mm_dw(dy, x, off, dw, ws)
    want, mags = ref.dw(dy, x, torch.tensor([0, 5]))
    ref.check(dw[-1:], want, mags, 5)
    assert int(dw[:-1].count_nonzero()) == 0
    _done(ws)


@pytest.mark.parametrize("name", ["tile_edges", "few_tiles", "long_groups", "token"])
def test_a_timeout_latched_before_cuts_no_wait_short(name):
    """A workspace whose error word still holds an earlier call's timeout: the waits of these calls are
    their own, so the results are the same bits, and the code stays for moe_get_device_status."""
    x, w, dy, off, ws = _case(name, "bf16")
    E, M, K, N = w.shape[0], x.shape[0], x.shape[1], w.shape[1]
    fmt = q.FP4_NV
    xq, xs = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(
        q.moe_fp4_scale_bytes(fmt, M, K, E, True), dtype=torch.uint8, device="cuda")
    wq, wsc = torch.zeros(E * N, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(
        q.moe_fp4_scale_bytes(fmt, E * N, K, E), dtype=torch.uint8, device="cuda")
    results = []
    for code in (0, q.STRATA_ETIMEOUT):
        ws[:4].view(torch.int32).fill_(code)
        out = [torch.zeros(*s, dtype=dt, device="cuda") for dt in (torch.bfloat16, torch.float32)
               for s in ((M, N), (M, K), (E, N, K), (M, N))]
        for y, dx, dw, y4 in (out[:4], out[4:]):
            q.moe_grouped_mm(x, w, off, y, ws)
            q.moe_grouped_mm_dx(dy, w, off, dx, ws)
            q.moe_grouped_mm_dw(dy, x, off, dw, ws)
            q.moe_fp4_quantize(x, xq, xs, fmt, ws, offsets=off)
            q.moe_fp4_quantize(w.view(E * N, K), wq, wsc, fmt, ws, n_groups=E)
            q.moe_grouped_mm_fp4(xq, xs, wq.view(E, N, K // 2), wsc, off, y4, fmt, ws)
        assert q.moe_get_device_status(ws) == code
        results.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*results))
    _done(ws)
