"""The grouped products and the 4-bit block formats beside the int4 experts, as measured cases.

Operators (slots are the rows of moe_permute's order, group e holding rows
offsets[e] .. offsets[e + 1]):
  mm     y[s] = W[e] x[s]                     (bf16 / fp16, y in that type or fp32)
  dx     dx[s] = W[e]^T dy[s]                 (the gradient of mm's input)
  dw     dW[e] = sum over e's slots dy x^T    (the gradient of mm's weights)
  quant  rows to 4-bit blocks (e2m1 with a scale per 16 or 32) and back to values
  fp4    y[s] = alpha[e] W4[e] x4[s], optionally SwiGLU of interleaved gate/up rows
  ffn    quant, fp4 with SwiGLU, quant, fp4: the routed experts' whole FFN

Scales lie in tiles of 128 rows by 4 scales (512 bytes), the row blocks of a
group starting at a block of their own.
"""
import math

import torch

own = False

WORKSPACE_BYTES = 65536
VEC = {"mx": 32, "nv": 16}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
X_EXP, W_EXP = 0, -8        # powers of two the nv scales are taken relative to (0 for mx)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token's eight routed experts, gate/up rows of a 2048-hidden layer
        dict(name="mm_token", op="mm", dtype="bf16", out="bf16", E=256, top_k=8, T=1, K=2048, N=1024,
             spare=0),
        # a decode window of 16 tokens through the down product, fp32 sums kept
        dict(name="mm_window", op="mm", dtype="fp16", out="fp32", E=256, top_k=8, T=16, K=512, N=2048,
             spare=0),
        # a 2048-token prompt through gate/up
        dict(name="mm_prompt", op="mm", dtype="bf16", out="bf16", E=256, top_k=8, T=2048, K=2048,
             N=1024, spare=0),
        # a tuning step's input gradient over the same prompt
        dict(name="dx_prompt", op="dx", dtype="bf16", out="bf16", E=256, top_k=8, T=2048, K=2048,
             N=1024, spare=0),
        # few tokens, odd widths, buffers larger than the rows in use
        dict(name="dx_ragged", op="dx", dtype="fp16", out="fp32", E=32, top_k=4, T=251, K=1000, N=264,
             spare=37),
        # a tuning step's weight gradient: every expert written, most from few rows
        dict(name="dw_prompt", op="dw", dtype="bf16", out="bf16", E=256, top_k=8, T=2048, K=2048,
             N=1024, spare=0),
        # long batches over the toy layer's expert count: the weight gradient's sums in fp32
        dict(name="dw_long", op="dw", dtype="bf16", out="fp32", E=32, top_k=4, T=16384, K=2048, N=1024,
             spare=0),
        # one token's row quantised for its eight slots
        dict(name="quant_token", op="quant", dtype="bf16", fmt="nv", E=256, top_k=8, T=1, K=2048,
             spare=0),
        # a prompt's rows gathered into slot order and quantised
        dict(name="quant_prompt", op="quant", dtype="bf16", fmt="mx", E=256, top_k=8, T=2048, K=2048,
             spare=0),
        # one token through 4-bit gate/up
        dict(name="fp4_token", op="fp4", fmt="nv", out="bf16", swiglu=False, E=256, top_k=8, T=1,
             K=2048, N=1024, spare=0),
        # a prompt through 4-bit gate/up with SwiGLU
        dict(name="fp4_prompt", op="fp4", fmt="nv", out="bf16", swiglu=True, E=256, top_k=8, T=2048,
             K=2048, N=1024, spare=0),
        # the wider family geometry's experts, 300 tokens through the whole 4-bit FFN
        dict(name="ffn_wide", op="ffn", dtype="bf16", fmt="mx", out="bf16", E=512, top_k=10, T=300,
             K=2048, N=1024, spare=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mm", "mm", "dx", "dw", "quant", "fp4", "fp4", "ffn"])
    E = _log(rng, 1, 512)
    top_k = rng.randint(1, min(E, 10))
    T = _log(rng, 1, 2048)
    c = dict(op=op, E=E, top_k=top_k, T=T, spare=rng.choice([0, 0, rng.randint(1, 200)]))
    if op in ("quant", "fp4", "ffn"):
        c["fmt"] = rng.choice(["mx", "nv"])
        c["K"] = 32 * _log(rng, 1, 128)
    else:
        c["K"] = 8 * _log(rng, 2, 512)
    if op != "fp4":
        c["dtype"] = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("mm", "dx", "dw"):
        c["out"] = rng.choice([c["dtype"], "fp32"])
        c["N"] = _log(rng, 1, 2048) if op == "mm" else 8 * _log(rng, 1, 256)
    elif op == "fp4":
        c["out"] = rng.choice(["bf16", "fp16"])
        c["swiglu"] = rng.choice([False, True])
        c["N"] = (2 if c["swiglu"] else 1) * _log(rng, 1, 1024)
    elif op == "ffn":
        c["out"] = c["dtype"]
        c["N"] = 64 * _log(rng, 1, 16)
    # the listed cases' weights and products bound the drawn ones
    if "N" in c and E * c["N"] * c["K"] > 1 << 29:
        c["K"] = max(32, (1 << 29) // (E * c["N"]) // 32 * 32)
    if "N" in c:
        c["T"] = max(1, min(T, (1 << 35) // (top_k * c["N"] * c["K"])))
    return c


# ------------------------------------------------------------------ inputs
def _routing(c, gen):
    """Tokens routed top_k of E with a mild Zipf skew, in slot order."""
    E, k, T = c["E"], c["top_k"], c["T"]
    rank = torch.randperm(E, generator=gen, device="cuda") + 1
    logits = torch.randn(T, E, generator=gen, device="cuda") - 0.1815 * torch.log(rank.float())
    ids = logits.topk(k, dim=1).indices.sort(dim=1).values.reshape(-1)
    perm = torch.sort(ids, stable=True).indices.int()
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return perm, offsets, int(counts.max())


def _vec(c):
    return VEC[c["fmt"]]


def _tile_index(rows, cols, vec, first, block):
    """Byte place of every scale [rows][cols / vec]: `first` is each row's place in its group,
    `block` its group's first row block."""
    kw = -(-cols // (4 * vec))
    col = torch.arange(cols // vec, device="cuda")
    at = (block + first // 128).long()[:, None] * kw + col // 4
    r = (first % 128).long()[:, None]
    return at * 512 + (r % 32) * 16 + (r // 32) * 4 + col % 4


def _place(offsets, rows):
    """Each row's group, its place in the group, and its group's first row block."""
    r = torch.arange(rows, device="cuda", dtype=torch.int32)
    e = torch.searchsorted(offsets[1:].contiguous(), r, right=True).clamp(max=offsets.numel() - 2)
    blocks = (offsets[1:] - offsets[:-1] + 127) // 128
    return e, r - offsets[e], (blocks.cumsum(0) - blocks)[e]


def _ragged_scale_bytes(rows, cols, vec, groups):
    return (rows // 128 + min(groups, rows)) * -(-cols // (4 * vec)) * 512


def _pack4(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _weights4(c, N, K, gen):
    """Expert weights N(0, 0.02) as packed codes [E][N][K / 2] and tiled scales."""
    E, vec = c["E"], _vec(c)
    codes, sbytes, _ = _quant(0.02 * torch.randn(E * N, K, generator=gen, device="cuda"), c["fmt"],
                              W_EXP if c["fmt"] == "nv" else 0)
    r = torch.arange(E * N, device="cuda", dtype=torch.int32)
    blocks = -(-N // 128)
    tiled = torch.zeros(E * blocks * -(-K // (4 * vec)) * 512, dtype=torch.uint8, device="cuda")
    tiled[_tile_index(E * N, K, vec, r % N, r // N * blocks)] = sbytes
    return _pack4(codes).reshape(E, N, K // 2), tiled


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    perm, offsets, cap = _routing(c, gen)
    rows, K, N = c["T"] * c["top_k"] + c["spare"], c["K"], c.get("N", 0)
    st = dict(case=c, offsets=offsets, perm=perm, cap=cap, rows=rows,
              ws=torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"))

    def normal(*shape, dtype=None):
        return torch.randn(*shape, generator=gen, device="cuda").to(DT[dtype or c["dtype"]])

    if c["op"] in ("mm", "dx", "dw"):
        if c["op"] != "dx":
            st["x"] = normal(rows, K)
        if c["op"] != "mm":
            st["dy"] = normal(rows, N)
        if c["op"] != "dw":
            st["w"] = (0.02 * torch.randn(c["E"], N, K, generator=gen, device="cuda")).to(DT[c["dtype"]])
        shape = {"mm": (rows, N), "dx": (rows, K), "dw": (c["E"], N, K)}[c["op"]]
        st["y"] = torch.zeros(shape, dtype=DT[c["out"]], device="cuda")
        return st
    vec = _vec(c)
    st["xq"] = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
    st["xs"] = torch.zeros(_ragged_scale_bytes(rows, K, vec, c["E"]), dtype=torch.uint8, device="cuda")
    if c["op"] in ("quant", "ffn"):
        st["x"] = normal(c["T"], K)
    if c["op"] == "quant":
        st["y"] = torch.zeros(rows, K, dtype=DT[c["dtype"]], device="cuda")
        return st
    ex = W_EXP + X_EXP if c["fmt"] == "nv" else 0
    st["alpha"] = 2.0 ** ex * (1 + torch.rand(c["E"], generator=gen, device="cuda"))
    st["wq"], st["wsc"] = _weights4(c, N, K, gen)
    if c["op"] == "fp4":
        live = c["T"] * c["top_k"]
        codes, sbytes, _ = _quant(torch.randn(live, K, generator=gen, device="cuda"), c["fmt"], X_EXP)
        st["xq"][:live] = _pack4(codes)
        _, first, block = _place(offsets, live)
        st["xs"][_tile_index(live, K, vec, first, block)] = sbytes
        st["y"] = torch.zeros(rows, N // 2 if c["swiglu"] else N, dtype=DT[c["out"]], device="cuda")
    else:
        inter = N // 2
        st["w2q"], st["w2sc"] = _weights4(c, K, inter, gen)
        st["alpha2"] = torch.full_like(st["alpha"], 2.0 ** ex)
        st["h"] = torch.zeros(rows, inter, dtype=DT[c["dtype"]], device="cuda")
        st["hq"] = torch.zeros(rows, inter // 2, dtype=torch.uint8, device="cuda")
        st["hs"] = torch.zeros(_ragged_scale_bytes(rows, inter, vec, c["E"]), dtype=torch.uint8,
                               device="cuda")
        st["y"] = torch.zeros(rows, K, dtype=DT[c["out"]], device="cuda")
    return st


# ------------------------------------------------------------- plain forms
def _spread(a, st):
    """fp32 rows as [E][cap][.], short groups filled with zeros."""
    off = st["offsets"].long()
    idx = off[:-1, None] + torch.arange(st["cap"], device="cuda")
    live = idx < off[1:, None]
    return torch.where(live[..., None], a.float()[idx.clamp(max=a.shape[0] - 1)], 0.0)


def _collect(p, st, rows):
    """The rows of [E][cap][.] in slot order; rows behind the last group are zero."""
    off = st["offsets"]
    e, first, _ = _place(off, rows)
    live = torch.arange(rows, device="cuda") < off[-1]
    return torch.where(live[:, None], p[e, first.clamp(max=st["cap"] - 1)], 0.0)


def _pow2(e):
    """2^(e - 127) of scale bytes 1..254, exactly; 0 for byte 0, which only blocks of zeros have."""
    return (e.int() << 23).view(torch.float32)


def _quant(x, fmt, ex):
    """(codes, scale bytes, scale values relative to 2^ex) of fp32 rows; decisions are exact: every
    border times a scale has few bits, so no comparison rounds."""
    vec = VEC[fmt]
    ax = (x.abs() * 2.0 ** -ex).reshape(x.shape[0], -1, vec)
    amax = ax.amax(dim=2)
    if fmt == "mx":
        sbyte = (torch.frexp(amax).exponent - 1 - 2 + 127).clamp(0, 254)
        sbyte = torch.where(amax > 0, sbyte, 0)
        s = _pow2(sbyte)
    else:
        f8 = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        sbyte, s = f8.view(torch.uint8), f8.float()
    t = s[..., None]
    code = ((ax > 0.25 * t).byte() + (ax >= 0.75 * t).byte() + (ax > 1.25 * t).byte()
            + (ax >= 1.75 * t).byte() + (ax > 2.5 * t).byte() + (ax >= 3.5 * t).byte()
            + (ax > 5.0 * t).byte())
    code = torch.where(t > 0, code, torch.zeros_like(code)).reshape(x.shape)
    return code + 8 * (x < 0).byte(), sbyte.to(torch.uint8), s


def _values(codes, s, vec):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    grid = torch.cat([grid, -grid])
    return (grid[codes.int()].reshape(codes.shape[0], -1, vec) * s[..., None]).reshape(codes.shape)


def _unpack(q, tiled, index, fmt):
    """fp32 values (relative to 2^ex) of packed codes and tiled scales."""
    codes = torch.stack([q & 15, q >> 4], dim=-1).reshape(q.shape[0], -1)
    b = tiled[index]
    s = _pow2(b) if fmt == "mx" else b.view(torch.float8_e4m3fn).float()
    return _values(codes, s, VEC[fmt])


def _plain_weights(c, wq, wsc):
    E, N, K = wq.shape[0], wq.shape[1], 2 * wq.shape[2]
    r = torch.arange(E * N, device="cuda", dtype=torch.int32)
    index = _tile_index(E * N, K, _vec(c), r % N, r // N * -(-N // 128))
    return _unpack(wq.reshape(E * N, K // 2), wsc, index, c["fmt"]).reshape(E, N, K)


def _swiglu(p):
    g, u = p[..., 0::2], p[..., 1::2]
    return g / (1 + torch.exp(-g)) * u


def _plain(st):
    c, rows = st["case"], st["rows"]
    out = DT[c.get("out", c.get("dtype"))]
    if c["op"] == "mm":
        return _collect(torch.bmm(_spread(st["x"], st), st["w"].float().transpose(1, 2)), st, rows).to(out)
    if c["op"] == "dx":
        return _collect(torch.bmm(_spread(st["dy"], st), st["w"].float()), st, rows).to(out)
    if c["op"] == "dw":
        return torch.bmm(_spread(st["dy"], st).transpose(1, 2), _spread(st["x"], st)).to(out)
    vec = _vec(c)
    if c["op"] in ("quant", "ffn"):
        codes, _, s = _quant(st["x"].float()[st["perm"].long() // c["top_k"]], c["fmt"], X_EXP)
        x = _values(codes, s, vec) * 2.0 ** X_EXP
        x = torch.cat([x, x.new_zeros(rows - x.shape[0], x.shape[1])])
        if c["op"] == "quant":
            return x.to(out)
        x = x * 2.0 ** -X_EXP
    else:
        _, first, block = _place(st["offsets"], rows)
        index = _tile_index(rows, c["K"], vec, first, block).clamp(max=st["xs"].numel() - 1)
        x = _unpack(st["xq"], st["xs"], index, c["fmt"])
    p = torch.bmm(_spread(x, st), _plain_weights(c, st["wq"], st["wsc"]).transpose(1, 2))
    p = p * st["alpha"][:, None, None]
    if c["op"] == "fp4":
        return _collect(_swiglu(p) if c["swiglu"] else p, st, rows).to(out)
    h = _swiglu(p).to(DT[c["dtype"]]).float()
    codes, _, s = _quant(h.reshape(-1, h.shape[2]), c["fmt"], X_EXP)
    h = _values(codes, s, vec).reshape(h.shape)
    y = torch.bmm(h, _plain_weights(c, st["w2q"], st["w2sc"]).transpose(1, 2))
    return _collect(y * st["alpha2"][:, None, None], st, rows).to(out)


# ------------------------------------------------------------------ a pass
def run(state):
    if not own:
        return _plain(state)
    import quantized_moe_expert_fwd_gb300 as g
    st, c = state, state["case"]
    off, ws, y = st["offsets"], st["ws"], st["y"]
    if c["op"] == "mm":
        g.moe_grouped_mm(st["x"], st["w"], off, y, ws)
    elif c["op"] == "dx":
        g.moe_grouped_mm_dx(st["dy"], st["w"], off, y, ws)
    elif c["op"] == "dw":
        g.moe_grouped_mm_dw(st["dy"], st["x"], off, y, ws)
    else:
        fmt = g.FP4_MX if c["fmt"] == "mx" else g.FP4_NV
        if c["op"] in ("quant", "ffn"):
            g.moe_fp4_quantize(st["x"], st["xq"], st["xs"], fmt, ws, offsets=off, scale_exp=X_EXP,
                               perm=st["perm"], top_k=c["top_k"])
        if c["op"] == "quant":
            g.moe_fp4_dequantize(st["xq"], st["xs"], y, fmt, ws, offsets=off, scale_exp=X_EXP)
        elif c["op"] == "fp4":
            g.moe_grouped_mm_fp4(st["xq"], st["xs"], st["wq"], st["wsc"], off, y, fmt, ws,
                                 alpha=st["alpha"], swiglu=c["swiglu"])
        else:
            g.moe_grouped_mm_fp4(st["xq"], st["xs"], st["wq"], st["wsc"], off, st["h"], fmt, ws,
                                 alpha=st["alpha"], swiglu=True)
            g.moe_fp4_quantize(st["h"], st["hq"], st["hs"], fmt, ws, offsets=off, scale_exp=X_EXP)
            g.moe_grouped_mm_fp4(st["hq"], st["hs"], st["w2q"], st["w2sc"], off, y, fmt, ws,
                                 alpha=st["alpha2"])
    return y


def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    rows, K, N, E = c["T"] * c["top_k"], c["K"], c.get("N", 0), c["E"]
    # experts that T tokens of top_k picks touch, on average
    touched = E * (1 - (1 - c["top_k"] / E) ** c["T"])
    if c["op"] == "quant":
        # token rows in, codes and scales out and back in, values out
        return {"bytes": c["T"] * K * 2 + rows * K * (2 * (0.5 + 1 / _vec(c)) + 2), "flops": 0}
    flops = 2 * rows * K * N
    if c["op"] in ("mm", "dx"):
        a, y = (K, N) if c["op"] == "mm" else (N, K)
        return {"bytes": rows * (a * 2 + y * size[c["out"]]) + touched * N * K * 2, "flops": flops}
    if c["op"] == "dw":
        return {"bytes": rows * (K + N) * 2 + E * N * K * size[c["out"]], "flops": flops}
    per = 0.5 + 1 / _vec(c)
    if c["op"] == "fp4":
        y = N // 2 if c["swiglu"] else N
        return {"bytes": rows * (K * per + y * 2) + touched * N * K * per, "flops": flops}
    # token rows in, codes out and in, h out and in, its codes out and in, y out
    acts = c["T"] * K * 2 + rows * (2 * K * per + N // 2 * (4 + 2 * per) + K * 2)
    return {"bytes": acts + touched * 1.5 * N * K * per, "flops": flops * 3 // 2}


# ----------------------------------------------------------- in 64 bits
def _binade(v):
    """floor(log2 v) of float64 values from their exponent bits (-1023 for 0)."""
    return (v.view(torch.int64) >> 52) - 1023


def _two_to(e):
    return ((e.clamp(min=-1022) + 1023) << 52).view(torch.float64)


def _exact_quant(x, fmt, ex):
    """Values (relative to 2^ex) of float64 rows after the 4-bit rounding, from its definition."""
    vec = VEC[fmt]
    x = (x * 2.0 ** -ex).reshape(x.shape[0], -1, vec)
    amax = x.abs().amax(dim=2, keepdim=True)
    if fmt == "mx":
        s = _two_to(_binade(amax) - 2)
    else:
        v = (amax / 6).clamp(max=448)
        step = _two_to(_binade(v).clamp(min=-6) - 3)
        s = torch.round(v / step) * step
    q = torch.where(s > 0, x.abs() / s, torch.zeros_like(x))
    q = torch.where(q < 2, torch.round(2 * q) / 2,
                    torch.where(q < 4, torch.round(q), 2 * torch.round(q / 2))).clamp(max=6)
    return (torch.sign(x) * q * s).reshape(x.shape[0], -1)


def _exact_decode(q, tiled, fmt, groups):
    """float64 values of packed rows whose groups are (first row, rows) pairs in order."""
    vec = VEC[fmt]
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device="cuda").double() / 2
    codes = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.long, device="cuda")
    codes[:, 0::2], codes[:, 1::2] = (q & 15).long(), (q >> 4).long()
    v = mag[codes & 7] * (1 - 2 * (codes >> 3)).double()
    cols = codes.shape[1] // vec
    tiles = tiled.reshape(-1, -(-cols // 4), 32, 4, 4)
    s = torch.zeros(q.shape[0], cols, dtype=torch.uint8, device="cuda")
    block = 0
    for first, n in groups:
        nb = -(-n // 128)
        # [block][word][lane][quarter][byte] -> rows of quarter, lane; columns of word, byte
        t = tiles[block:block + nb].permute(0, 3, 2, 1, 4).reshape(nb * 128, 4 * tiles.shape[1])
        s[first:first + n] = t[:n, :cols]
        block += nb
    if fmt == "mx":
        sv = torch.exp2(s.double() - 127)
    else:
        e, m = (s >> 3).double(), (s & 7).double()
        sv = torch.where(e > 0, (8 + m) * torch.exp2(e - 10), m * 2.0 ** -9)
    return v * sv.repeat_interleave(vec, dim=1)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    off = st["offsets"].tolist()
    spans = [(off[e], off[e + 1] - off[e]) for e in range(c["E"])]
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    if c["op"] == "quant":
        src = (st["perm"] // c["top_k"]).long()
        y[:src.numel()] = _exact_quant(st["x"].double(), c["fmt"], X_EXP)[src] * 2.0 ** X_EXP
        return y
    if c["op"] in ("mm", "dx", "dw"):
        for e, (s, n) in enumerate(spans):
            at = slice(s, s + n)
            if n and c["op"] == "mm":
                y[at] = st["x"][at].double() @ st["w"][e].double().T
            elif n and c["op"] == "dx":
                y[at] = st["dy"][at].double() @ st["w"][e].double()
            elif n:
                y[e] = st["dy"][at].double().T @ st["x"][at].double()
        return y
    N, K = c["N"], c["K"]
    if c["op"] == "fp4":
        x = _exact_decode(st["xq"], st["xs"], c["fmt"], spans)
    else:
        src = (st["perm"] // c["top_k"]).long()
        x = _exact_quant(st["x"].double(), c["fmt"], X_EXP)[src] * 2.0 ** -X_EXP
    nb, kw = -(-N // 128), -(-K // (4 * _vec(c))) * 512
    if c["op"] == "ffn":
        nb2, kw2 = -(-K // 128), -(-(N // 2) // (4 * _vec(c))) * 512
    for e, (s, n) in enumerate(spans):
        if not n:
            continue
        w = _exact_decode(st["wq"][e], st["wsc"][e * nb * kw:(e + 1) * nb * kw], c["fmt"], [(0, N)])
        p = st["alpha"][e].double() * (x[s:s + n] @ w.T)
        if c["op"] == "ffn" or c["swiglu"]:
            g, u = p[:, 0::2], p[:, 1::2]
            p = u * g * torch.sigmoid(g)
        if c["op"] == "ffn":
            h = _exact_quant(p.to(DT[c["dtype"]]).double(), c["fmt"], X_EXP)
            w2 = _exact_decode(st["w2q"][e], st["w2sc"][e * nb2 * kw2:(e + 1) * nb2 * kw2], c["fmt"],
                               [(0, K)])
            p = st["alpha2"][e].double() * (h @ w2.T)
        y[s:s + n] = p
    return y
