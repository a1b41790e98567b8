"""A tuning step's operators around the bf16 / fp16 experts, as measured cases.

Operators (slots are the rows of moe_permute's order, group e holding rows
offsets[e] .. offsets[e + 1]; gate and up rows of W interleaved, 2i and 2i + 1):
  glu    p[s] = W[e] x[s],  h[s][i] = p[2i] / (1 + exp(-p[2i])) * p[2i + 1]; p kept for the
         backward pass where save says so (16: in the operands' type)
  bwd    dh[s] = Wd[e]^T dy[s] and, from the kept p, dp (the gradient by p) and h again
  act8   rows kept in 8 bits (e4m3, a power-of-two scale per 32) and read back into slot order
  ffn8   the two together with everything kept in 8 bits: gather, keep x, glu keeping p,
         then bwd from that p and x read back
  norm   r' = alpha r + beta gate n(f),  x = n(r'):  the RMS norms before and after a block with
         its gate and residual scale (n with weights; the one of f only with post)
  normb  the gradients of norm by r, f, the gate and both weights
  mix    out[t] = sum_k w[t][k] y[slot of (t, k)], then the gradients by y and w
"""
import math

import torch

own = False

WORKSPACE_BYTES = 65536
NORM_WORKSPACE_BYTES = (65536, 4864)             # and for every column
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token's eight routed experts while serving: nothing is kept
        dict(name="glu_token", op="glu", dtype="bf16", save=0, E=256, top_k=8, T=1, K=2048, I=512,
             spare=0),
        # few tokens, odd widths, buffers larger than the rows in use
        dict(name="glu_ragged", op="glu", dtype="fp16", save=16, E=32, top_k=4, T=251, K=1000, I=133,
             spare=37),
        # a 2048-token prompt of a tuning step
        dict(name="glu_prompt", op="glu", dtype="bf16", save=16, E=256, top_k=8, T=2048, K=2048,
             I=512, spare=0),
        # the backward pass of a small ragged batch
        dict(name="bwd_ragged", op="bwd", dtype="fp16", E=32, top_k=4, T=251, K=1000, I=264, spare=37),
        # the backward pass of the prompt
        dict(name="bwd_prompt", op="bwd", dtype="bf16", E=256, top_k=8, T=2048, K=2048, I=512, spare=0),
        # the prompt's block inputs kept over the forward pass, read back in slot order
        dict(name="act8_prompt", op="act8", dtype="bf16", E=256, top_k=8, T=2048, K=2048, spare=0),
        # long batches over the toy layer's expert count, all that is kept in 8 bits
        dict(name="ffn8_long", op="ffn8", dtype="bf16", E=32, top_k=4, T=16384, K=2048, I=512, spare=0),
        # a decode step's norms around the block
        dict(name="norm_token", op="norm", dtype="bf16", resid="fp32", post=True, gate=True, T=1, K=2048),
        # the norms of a long batch
        dict(name="norm_long", op="norm", dtype="bf16", resid="fp32", post=True, gate=True, T=16384,
             K=2048),
        # their gradients
        dict(name="normb_long", op="normb", dtype="bf16", resid="fp32", post=True, gate=True, T=16384,
             K=2048),
        # a window of 16 tokens, the wider family geometry's ten experts a token
        dict(name="mix_window", op="mix", dtype="fp16", E=512, top_k=10, T=16, K=2048, spare=0),
        # the prompt's slots weighted into tokens, and the gradients back into slots
        dict(name="mix_prompt", op="mix", dtype="bf16", E=256, top_k=8, T=2048, K=2048, spare=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glu", "glu", "bwd", "bwd", "act8", "ffn8", "norm", "normb", "mix"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op in ("norm", "normb"):
        c["resid"] = rng.choice(["fp32", c["dtype"]])
        c["post"], c["gate"] = rng.choice([False, True]), rng.choice([False, True])
        c["K"] = rng.choice([8 * _log(rng, 8, 1024), _log(rng, 64, 8192)])
        c["T"] = min(_log(rng, 1, 16384), (1 << 25) // c["K"])
        return c
    E = _log(rng, 1, 512)
    c.update(E=E, top_k=rng.randint(1, min(E, 10)), T=_log(rng, 1, 2048),
             spare=rng.choice([0, 0, rng.randint(1, 200)]))
    if op == "mix":
        c["K"] = rng.choice([8 * _log(rng, 8, 512), _log(rng, 64, 4096)])
    elif op in ("act8", "ffn8"):
        c["K"] = 32 * _log(rng, 1, 128)
    else:
        c["K"] = 8 * _log(rng, 2, 512)
    if op == "glu":
        c["save"] = rng.choice([0, 16])
    if op in ("glu", "bwd", "ffn8"):
        step, most = {"glu": (1, 1024), "bwd": (8, 128), "ffn8": (16, 64)}[op]
        c["I"] = step * _log(rng, 1, most)
        # the listed cases' weights and products bound the drawn ones
        if E * c["I"] * c["K"] > 1 << 28:
            c["K"] = max(32, (1 << 28) // (E * c["I"]) // 32 * 32)
        c["T"] = max(1, min(c["T"], (1 << 34) // (c["top_k"] * c["I"] * c["K"])))
    return c


# ------------------------------------------------------------------ inputs
def _routing(c, gen):
    """Tokens routed top_k of E with a mild Zipf skew, in slot order."""
    E, k, T = c["E"], c["top_k"], c["T"]
    rank = torch.randperm(E, generator=gen, device="cuda") + 1
    logits = torch.randn(T, E, generator=gen, device="cuda") - 0.1815 * torch.log(rank.float())
    top = logits.topk(k, dim=1)
    ids, order = top.indices.sort(dim=1)
    ids = ids.reshape(-1)
    perm = torch.sort(ids, stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device="cuda")
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    weights = torch.softmax(top.values, dim=1).gather(1, order)
    return dict(perm=perm.int(), inv=inv.int(), offsets=offsets, weights=weights, cap=int(counts.max()))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, K, I = c["T"], c["K"], c.get("I", 0)
    dt = DT[c["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)

    def zeros(*shape, dtype=dt):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    if c["op"] in ("norm", "normb"):
        rt = DT[c["resid"]]
        st = dict(case=c, f=normal(T, K, scale=0.5), r=normal(T, K, dtype=rt, scale=3.0),
                  w_pre=1 + normal(K, dtype=torch.float32, scale=0.1),
                  w_post=1 + normal(K, dtype=torch.float32, scale=0.1) if c["post"] else None,
                  gate=torch.sigmoid(normal(T, dtype=torch.float32)) if c["gate"] else None,
                  alpha=0.875, beta=1.25, r2=zeros(T, K, dtype=rt), x=zeros(T, K),
                  rstd=zeros(T, 2, dtype=torch.float32))
        if c["op"] == "normb":
            # what the forward pass leaves behind
            st["r2"], st["x"], st["rstd"] = _norm(st)
            st.update(dx=normal(T, K, scale=0.25), dr2=normal(T, K, dtype=rt, scale=0.25), df=zeros(T, K),
                      dr=zeros(T, K, dtype=rt), dgate=zeros(T, dtype=torch.float32),
                      dw_pre=zeros(K, dtype=torch.float32), dw_post=zeros(K, dtype=torch.float32),
                      ws=zeros(NORM_WORKSPACE_BYTES[0] + K * NORM_WORKSPACE_BYTES[1], dtype=torch.uint8))
        return st
    st = dict(case=c, ws=zeros(WORKSPACE_BYTES, dtype=torch.uint8), **_routing(c, gen))
    live = T * c["top_k"]
    rows = live + c["spare"]
    st["rows"] = rows
    if c["op"] in ("glu", "ffn8"):
        st["w"] = normal(c["E"], 2 * I, K, scale=0.02)
        st["h"] = zeros(rows, I)
    if c["op"] in ("bwd", "ffn8"):
        st["dy"] = normal(rows, K, scale=0.1)
        st["wd"] = normal(c["E"], K, I, scale=0.02)
        st["dp"], st["h2"] = zeros(rows, 2 * I), zeros(rows, I)
    if c["op"] == "glu":
        st["x"] = normal(rows, K)
        st["p"] = zeros(rows, 2 * I) if c["save"] else None
    elif c["op"] == "bwd":
        st["p"] = normal(rows, 2 * I, scale=0.9)
    elif c["op"] == "mix":
        st["y"], st["dout"] = normal(rows, K, scale=0.5), normal(T, K, scale=0.1)
        st["out"], st["dy"] = zeros(T, K), zeros(rows, K)
        st["dweights"] = zeros(T, c["top_k"], dtype=torch.float32)
    else:
        st["x"] = normal(T, K)
        st["xq"] = zeros(T, K, dtype=torch.uint8)
        st["xsc"] = zeros(T, K // 32, dtype=torch.uint8)
        st["xs"], st["xs2"] = zeros(rows, K), zeros(rows, K)
    if c["op"] == "ffn8":
        st["pq"] = zeros(rows, 2 * I, dtype=torch.uint8)
        st["psc"] = zeros(rows, 2 * I // 32, dtype=torch.uint8)
    return st


# ------------------------------------------------------------- plain forms
def _spread(a, st):
    """fp32 rows as [E][cap][.], short groups filled with zeros."""
    off = st["offsets"].long()
    idx = off[:-1, None] + torch.arange(st["cap"], device="cuda")
    live = idx < off[1:, None]
    return torch.where(live[..., None], a.float()[idx.clamp(max=a.shape[0] - 1)], 0.0)


def _collect(p, st):
    """The rows of [E][cap][.] in slot order; rows behind the last group are zero."""
    off = st["offsets"]
    r = torch.arange(st["rows"], device="cuda", dtype=torch.int32)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True).clamp(max=off.numel() - 2)
    first = (r - off[e]).clamp(max=st["cap"] - 1)
    return torch.where((r < off[-1])[:, None], p[e, first], 0.0)


def _silu_parts(p):
    g, u = p[..., 0::2], p[..., 1::2]
    s = 1 / (1 + torch.exp(-g))
    return g, u, s


def _pow2(e):
    """2^e in fp32, exactly, for e of -126 to 127."""
    return ((e + 127) << 23).view(torch.float32)


def _act8(x):
    """The values of fp32 rows kept in 8 bits: e4m3 times the smallest power of two that no value of
    a block of 32 exceeds 448 times."""
    b = x.reshape(x.shape[0], -1, 32)
    frac, ex = torch.frexp(b.abs().amax(dim=2, keepdim=True))
    e = (ex - 9 + (frac > 0.875).int()).clamp(min=-126)
    q = (b * _pow2(-e)).to(torch.float8_e4m3fn).float()
    return (q * _pow2(e)).reshape(x.shape)


def _rows_of(x, st):
    """Token rows in slot order, rows behind the last one zero."""
    g = x[st["perm"].long() // st["case"]["top_k"]]
    return torch.cat([g, g.new_zeros(st["rows"] - g.shape[0], g.shape[1])])


def _dp(dh, p):
    g, u, s = _silu_parts(p)
    dg = dh * u * s * (1 + g * (1 - s))
    du = dh * g * s
    return torch.stack([dg, du], dim=-1).reshape(p.shape), g * s * u


def _norm(st):
    c = st["case"]
    f = st["f"].float()
    r0 = torch.rsqrt((f * f).mean(dim=1) + EPS) if c["post"] else torch.ones_like(f[:, 0])
    n = f * r0[:, None]
    if c["post"]:
        n = n * st["w_post"]
    if c["gate"]:
        n = n * st["gate"][:, None]
    r2 = (st["alpha"] * st["r"].float() + st["beta"] * n).to(st["r"].dtype)
    v = r2.float()
    r1 = torch.rsqrt((v * v).mean(dim=1) + EPS)
    return r2, (v * r1[:, None] * st["w_pre"]).to(st["f"].dtype), torch.stack([r0, r1], dim=1)


def _norm_back(st):
    c = st["case"]
    f, v, dx = st["f"].float(), st["r2"].float(), st["dx"].float()
    r0, r1 = st["rstd"][:, :1], st["rstd"][:, 1:]
    gx = dx * st["w_pre"]
    d = st["dr2"].float() + r1 * (gx - v * r1 * r1 * (gx * v).mean(dim=1, keepdim=True))
    w = st["w_post"] if c["post"] else torch.ones_like(st["w_pre"])
    n = f * r0 * w
    dn = st["beta"] * d
    out = dict(dr=(st["alpha"] * d).to(st["r"].dtype), dw_pre=(dx * v * r1).sum(dim=0))
    if c["gate"]:
        out["dgate"] = (dn * n).sum(dim=1)
        dn = dn * st["gate"][:, None]
    if c["post"]:
        out["dw_post"] = (dn * f * r0).sum(dim=0)
        gf = dn * w
        dn = r0 * (gf - f * r0 * r0 * (gf * f).mean(dim=1, keepdim=True))
    out["df"] = dn.to(st["f"].dtype)
    return out


def _plain(st):
    c = st["case"]
    dt = DT[c["dtype"]]
    if c["op"] == "norm":
        return list(_norm(st))
    if c["op"] == "normb":
        return _norm_back(st)
    if c["op"] == "mix":
        k, live = c["top_k"], st["inv"].numel()
        inv = st["inv"].long()
        w = st["weights"].reshape(-1, 1)
        y = st["y"].float()[inv]
        d = st["dout"].float().repeat_interleave(k, dim=0)
        dy = torch.zeros(st["rows"], c["K"], device="cuda")
        dy[inv] = w * d
        out = (w * y).reshape(live // k, k, -1).sum(dim=1)
        return dict(out=out.to(dt), dy=dy.to(dt), dweights=(y * d).sum(dim=1).reshape(-1, k))
    if c["op"] == "act8":
        return _rows_of(_act8(st["x"].float()), st).to(dt)
    if c["op"] in ("glu", "ffn8"):
        x = st["x"] if c["op"] == "glu" else _rows_of(st["x"], st)
        p = torch.bmm(_spread(x, st), st["w"].float().transpose(1, 2))
        p = _collect(p, st)
        g, u, s = _silu_parts(p)
        h = (g * s * u).to(dt)
        if c["op"] == "glu":
            return [h, p.to(dt)] if c["save"] else [h]
        p = _act8(p)
    else:
        p = st["p"].float()
    dh = _collect(torch.bmm(_spread(st["dy"], st), st["wd"].float()), st)
    dp, h2 = _dp(dh, p)
    live = (torch.arange(st["rows"], device="cuda") < st["offsets"][-1])[:, None]
    out = [dp.to(dt), torch.where(live, h2, 0.0).to(dt)]
    if c["op"] == "ffn8":
        out += [h, _rows_of(_act8(st["x"].float()), st).to(dt)]
    return out


# ------------------------------------------------------------------ a pass
def run(state):
    if not own:
        return _plain(state)
    import quantized_moe_expert_fwd_gb300 as q
    st, c = state, state["case"]
    if c["op"] == "norm":
        q.moe_norm_residual(st["r"], st["r2"], f=st["f"], x=st["x"], w_pre=st["w_pre"],
                            w_post=st["w_post"], gate=st["gate"], post_norm=c["post"],
                            alpha=st["alpha"], beta=st["beta"], eps=EPS, rstd=st["rstd"])
        return [st["r2"], st["x"], st["rstd"]]
    if c["op"] == "normb":
        out = {n: st[n] for n, there in (("dr", True), ("dw_pre", True), ("dgate", c["gate"]),
                                         ("dw_post", c["post"]), ("df", True)) if there}
        q.moe_norm_residual_bwd(st["r2"], st["rstd"], st["ws"], dx=st["dx"], dresid_out=st["dr2"],
                                f=st["f"], w_pre=st["w_pre"], w_post=st["w_post"], gate=st["gate"],
                                post_norm=c["post"], alpha=st["alpha"], beta=st["beta"],
                                dresid=st["dr"], df=st["df"], dgate=out.get("dgate"),
                                dw_pre=st["dw_pre"], dw_post=out.get("dw_post"))
        return out
    off, ws = st["offsets"], st["ws"]
    if c["op"] == "mix":
        q.moe_slots_combine(st["y"], st["inv"], st["out"], ws, weights=st["weights"])
        q.moe_slots_spread(st["dout"], st["inv"], ws, dy=st["dy"], weights=st["weights"], y=st["y"],
                           dweights=st["dweights"])
        return dict(out=st["out"], dy=st["dy"], dweights=st["dweights"])
    if c["op"] == "glu":
        q.moe_grouped_swiglu(st["x"], st["w"], off, st["h"], ws, p=st["p"])
        return [st["h"], st["p"]] if c["save"] else [st["h"]]
    if c["op"] == "bwd":
        q.moe_grouped_swiglu_bwd(st["dy"], st["wd"], st["p"], off, st["dp"], ws, h=st["h2"])
        return [st["dp"], st["h2"]]
    q.moe_act8_save(st["x"], st["xq"], st["xsc"])
    if c["op"] == "ffn8":
        q.moe_slots_spread(st["x"], st["inv"], ws, dy=st["xs"])
        q.moe_grouped_swiglu(st["xs"], st["w"], off, st["h"], ws, p=st["pq"], p_scales=st["psc"])
        q.moe_grouped_swiglu_bwd(st["dy"], st["wd"], st["pq"], off, st["dp"], ws, p_scales=st["psc"],
                                 h=st["h2"])
    q.moe_act8_load(st["xq"], st["xsc"], st["xs2"], ws, perm=st["perm"], top_k=c["top_k"])
    return st["xs2"] if c["op"] == "act8" else [st["dp"], st["h2"], st["h"], st["xs2"]]


def work(case):
    c = case
    T, K, I, E = c["T"], c["K"], c.get("I", 0), c.get("E", 1)
    if c["op"] in ("norm", "normb"):
        r = 4 if c["resid"] == "fp32" else 2
        # r, f in, r', x out; back: f, r', dx, dr' in, df, dr out
        return {"bytes": T * K * (2 * r + 4 if c["op"] == "norm" else 3 * r + 6), "flops": 0}
    rows = T * c["top_k"]
    if c["op"] == "mix":
        # y and dout in (y for both passes once), out and dy out
        return {"bytes": (2 * rows + 2 * T) * K * 2, "flops": 4 * rows * K}
    kept = T * K * 2 * (1 + 1 / 32)              # 8 bits and their scales, written and read
    if c["op"] == "act8":
        return {"bytes": T * K * 2 + kept + rows * K * 2, "flops": 0}
    # experts that T tokens of top_k picks touch, on average
    touched = E * (1 - (1 - c["top_k"] / E) ** T)
    glu = touched * 2 * I * K * 2 + rows * I * 2
    bwd = touched * I * K * 2 + rows * (K * 2 + 2 * I * 2 + I * 2)
    if c["op"] == "glu":
        return {"bytes": glu + rows * K * 2 + (rows * 2 * I * 2 if c["save"] else 0),
                "flops": 4 * rows * I * K}
    if c["op"] == "bwd":
        return {"bytes": bwd + rows * 2 * I * 2, "flops": 2 * rows * I * K}
    # tokens in, their rows in slot order out, p kept
    return {"bytes": glu + bwd + T * K * 2 + kept + rows * K * 2 + rows * 4 * I * (1 + 1 / 32),
            "flops": 6 * rows * I * K}


# ----------------------------------------------------------- in 64 bits
def _keep8(x):
    """float64 rows after the 8-bit rounding, from its definition: with m the largest magnitude of
    32 values, the scale is 2^e with 448 2^(e - 1) < m <= 448 2^e (at least 2^-126), and values round
    to nearest even multiples of their binade's eighth, at least 2^-9 of the scale."""
    b = x.reshape(x.shape[0], -1, 32)
    m = b.abs().amax(dim=2, keepdim=True)
    e = torch.ceil(torch.log2(m.clamp(min=1e-300) / 448)).clamp(min=-126)
    e = torch.where(m > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((m <= 448 * torch.exp2(e - 1)) & (e > -126), e - 1, e)
    v = b * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step * torch.exp2(e)).reshape(x.shape)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    dt = DT[c["dtype"]]
    if c["op"] in ("norm", "normb"):
        f, r = st["f"].double(), st["r"].double()
        wpre = st["w_pre"].double()
        wpost = st["w_post"].double() if c["post"] else torch.ones_like(wpre)
        g = st["gate"].double()[:, None] if c["gate"] else torch.ones_like(f[:, :1])
        if c["op"] == "norm":
            s0 = 1 / torch.sqrt(f.square().mean(dim=1, keepdim=True) + EPS)
            s0 = s0 if c["post"] else torch.ones_like(s0)
            r2 = st["alpha"] * r + st["beta"] * g * (f * s0 * wpost)
            v = r2.to(st["r"].dtype).double()     # the norm is of what is stored
            s1 = 1 / torch.sqrt(v.square().mean(dim=1, keepdim=True) + EPS)
            return [r2, v * s1 * wpre, torch.cat([s0, s1], dim=1)]
        v, dx, dr2 = st["r2"].double(), st["dx"].double(), st["dr2"].double()
        s0, s1 = st["rstd"].double().split(1, dim=1)
        h = c["K"]
        d = dr2 + s1 * dx * wpre - v * s1 ** 3 * torch.einsum("th,h,th->t", dx, wpre, v)[:, None] / h
        out = dict(dr=st["alpha"] * d, dw_pre=torch.einsum("th,th,to->h", dx, v, s1))
        if c["gate"]:
            out["dgate"] = st["beta"] * torch.einsum("th,th,to,h->t", d, f, s0, wpost)
        df = st["beta"] * g * d * wpost * s0
        if c["post"]:
            out["dw_post"] = st["beta"] * torch.einsum("to,th,th,to->h", g, d, f, s0)
            df = df - f * s0 ** 2 * (df * f).sum(dim=1, keepdim=True) / h
        out["df"] = df
        return out
    k = c["top_k"]
    off = st["offsets"].tolist()
    live, rows = off[-1], st["rows"]
    if c["op"] == "mix":
        out = torch.zeros(c["T"], c["K"], dtype=torch.float64, device="cuda")
        dy = torch.zeros(rows, c["K"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(c["T"], k, dtype=torch.float64, device="cuda")
        inv, dout = st["inv"].reshape(-1, k).long(), st["dout"].double()
        for j in range(k):
            yj, wj = st["y"][inv[:, j]].double(), st["weights"][:, j:j + 1].double()
            out += wj * yj
            dy[inv[:, j]] = wj * dout
            dw[:, j] = torch.einsum("th,th->t", yj, dout)
        return dict(out=out, dy=dy, dweights=dw)

    def slots(x):
        y = torch.zeros(rows, c["K"], dtype=torch.float64, device="cuda")
        y[:live] = x[(st["perm"] // k).long()]
        return y

    def grouped(a, w, n):
        y = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            if off[e + 1] > off[e]:
                y[off[e]:off[e + 1]] = a[off[e]:off[e + 1]].double() @ w(e)
        return y

    if c["op"] == "act8":
        return slots(_keep8(st["x"].double()))
    I, out = c["I"], []
    if c["op"] in ("glu", "ffn8"):
        x = st["x"] if c["op"] == "glu" else slots(st["x"].double())
        p = grouped(x, lambda e: st["w"][e].double().T, 2 * I)
        h = p[:, 1::2] * p[:, 0::2] * torch.sigmoid(p[:, 0::2])
        if c["op"] == "glu":
            return [h, p] if c["save"] else [h]
        p, out = _keep8(p), [h, slots(_keep8(st["x"].double()))]
    else:
        p = st["p"].double()
    dh = grouped(st["dy"], lambda e: st["wd"][e].double(), I)
    g, u = p[:, 0::2], p[:, 1::2]
    sg = torch.sigmoid(g)
    dp = torch.zeros(rows, 2 * I, dtype=torch.float64, device="cuda")
    dp[:, 0::2] = dh * u * (sg + g * sg * torch.sigmoid(-g))
    dp[:, 1::2] = dh * g * sg
    h2 = u * g * sg
    h2[live:] = 0
    return [dp, h2] + out
