"""Cases of the operators around the block-scaled GEMMs: the norms and the gated
residual between blocks, the expert-grouped products, and the router with its
gather and combine.

`own` false: run() computes the plain torch form in FP32; true: the library's
entry points.  Sizes: 4096 / 14336 / 28672 are the repository's 8B MLP; the
others are generic mixture-of-experts shapes (64 or 128 experts, ragged widths).
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}


def listed():
    return [
        # norm ------------------------------------------------------------------
        # one decoded token between two blocks: pure latency
        dict(name="norm_token", op="norm", dir="fwd", rows=1, cols=4096, res="bf16", gate="none", post=True),
        # a training batch, residual in FP32, learned per-channel gate on the block's output
        dict(name="norm_train_fwd", op="norm", dir="fwd", rows=16384, cols=4096, res="f32", gate="channel", post=True),
        # its gradient with a BF16 residual and a ragged number of rows
        dict(name="norm_train_bwd", op="norm", dir="bwd", rows=8191, cols=4096, res="bf16", gate="channel", post=True),
        # router ------------------------------------------------------------------
        # a decode batch of 16 sequences over 64 experts
        dict(name="route_decode", op="route", dir="fwd", tokens=16, experts=64, k=4, align=1, scoring="softmax",
             normalize=True, dtype="bf16"),
        # a training batch over 128 experts, masked padding tokens, forward and backward
        dict(name="route_train", op="route", dir="both", tokens=16381, experts=128, k=8, align=32, scoring="sigmoid",
             normalize=True, dtype="f32"),
        # tokens to the experts' rows and back ------------------------------------
        # gather of a ragged prompt batch into expert order, groups padded for quantization
        dict(name="gather_prompt", op="gather", tokens=4093, experts=64, k=4, align=16, cols=2048),
        # weighted sum of the experts' rows and its gradient
        dict(name="combine_train", op="combine", tokens=8192, experts=8, k=2, align=32, cols=4096),
        # grouped products ----------------------------------------------------------
        # one token through two of eight experts' gate/up weights
        dict(name="grouped_token_nvfp4", op="grouped", fmt="nvfp4", experts=8, rows=2, n=28672, kdim=4096, align=1),
        # a decode batch over many small experts, a width that is no multiple of 512
        dict(name="grouped_decode_mxfp8", op="grouped", fmt="mxfp8", experts=64, rows=256, n=2048, kdim=1408, align=1),
        # the forward product of a training batch
        dict(name="grouped_train_nvfp4", op="grouped", fmt="nvfp4", experts=8, rows=16384, n=28672, kdim=4096, align=32),
        # weight gradients: small ragged experts; the training batch
        dict(name="wgrad_ragged_mxfp4", op="wgrad", fmt="mxfp4", experts=32, rows=4000, m=2048, n=1408, align=32),
        dict(name="wgrad_train_nvfp4", op="wgrad", fmt="nvfp4", experts=8, rows=16384, m=14336, n=4096, align=16),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["norm", "norm", "route", "gather", "combine", "grouped", "grouped", "wgrad"])
    if op == "norm":
        d = rng.choice(["fwd", "bwd"])
        cols = rng.choice([4096, 2048, _log_int(rng, 64, 8192), _log_int(rng, 64, 8192, 8)])
        rows = _log_int(rng, 1, 16384 * 4096 // max(cols, 4096))
        return dict(op=op, dir=d, rows=rows, cols=cols, res=rng.choice(["bf16", "f32"]),
                    gate=rng.choice(["none", "channel", "row", "full"]), post=rng.random() < 0.7)
    if op == "route":
        e = rng.choice([8, 16, 60, 64, 128, 160, 256])
        return dict(op=op, dir=rng.choice(["fwd", "both"]), tokens=_log_int(rng, 1, 16384), experts=e,
                    k=rng.randint(1, 8), align=rng.choice([1, 16, 32]), scoring=rng.choice(["softmax", "sigmoid"]),
                    normalize=rng.random() < 0.6, dtype=rng.choice(["bf16", "f32"]))
    if op in ("gather", "combine"):
        return dict(op=op, tokens=_log_int(rng, 1, 8192), experts=rng.choice([8, 16, 64, 128]), k=rng.choice([1, 2, 4, 6]),
                    align=rng.choice([1, 16, 32]), cols=rng.choice([2048, 4096, _log_int(rng, 128, 4096), 1408]))
    fmt = rng.choice(["nvfp4", "mxfp4", "mxfp8"])
    e = rng.choice([4, 8, 16, 32, 64])
    if op == "grouped":
        return dict(op=op, fmt=fmt, experts=e, rows=_log_int(rng, 1, 8192), n=_log_int(rng, 256, 4096, 4),
                    kdim=rng.choice([1024, 2048, 4096, _log_int(rng, 256, 4096, 32)]), align=rng.choice([1, 16, 32]))
    return dict(op=op, fmt=fmt, experts=e, rows=_log_int(rng, 64, 8192), m=_log_int(rng, 256, 4096, 32),
                n=_log_int(rng, 256, 2048, 32), align=rng.choice([16, 32]) if fmt == "nvfp4" else 32)


# ---------------------------------------------------------------- sizes of a case

def _buffer_rows(assigned, experts, align):
    """Rows of the expert-ordered buffers: every group padded to align, and 512-row
    multiples where the rows become a quantized reduction dimension."""
    if align == 1:
        return assigned
    rows = assigned + min(experts, assigned) * (align - 1)
    return -(-rows // 512) * 512


def _groups(c):
    """Rows per expert of a grouped case: uneven, some experts empty when rows are few."""
    r = np.random.RandomState(c["experts"] * 1009 + c["rows"])
    p = np.exp(0.5 * r.randn(c["experts"]))
    n = r.multinomial(c["rows"], p / p.sum())
    ends = np.cumsum(-(-n // c["align"]) * c["align"])
    return [int(v) for v in n], [0] + [int(v) for v in ends]


def _bits(fmt):
    return (8 if fmt == "mxfp8" else 4) + 8 / BLOCK[fmt]


def work(c):
    op = c["op"]
    if op == "norm":
        n, s = c["rows"] * c["cols"], 4 if c["res"] == "f32" else 2
        gate = {"none": 0, "channel": 4 * c["cols"], "row": 4 * c["rows"], "full": 2 * n}[c["gate"]]
        if c["dir"] == "fwd":
            return {"bytes": n * (2 * s + 4) + gate + 8 * c["cols"] + 8 * c["rows"], "flops": 12 * n}
        return {"bytes": n * (3 * s + 6) + 2 * gate + 16 * c["cols"] + 8 * c["rows"], "flops": 26 * n}
    if op == "route":
        t, e, k = c["tokens"], c["experts"], c["k"]
        s = 4 if c["dtype"] == "f32" else 2
        b = t * e * s + 12 * t * k + 4 * e + 4 * _buffer_rows(t * k, e, c["align"])
        if c["dir"] == "both":
            b += 2 * t * e * s + 8 * t * k
        return {"bytes": b, "flops": t * e * (2 + k)}
    if op in ("gather", "combine"):
        t, h, k = c["tokens"], c["cols"], c["k"]
        rows = _buffer_rows(t * k, c["experts"], c["align"])
        if op == "gather":
            return {"bytes": 2 * h * (t + rows) + 4 * rows, "flops": 0}
        return {"bytes": 2 * h * (2 * t + t * k + rows) + 12 * t * k + 4 * rows, "flops": 5 * t * k * h}
    n, off = _groups(c)
    p = _buffer_rows(c["rows"], c["experts"], c["align"])
    if op == "grouped":
        hit = sum(1 for v in n if v)
        return {"bytes": int(_bits(c["fmt"]) / 8 * c["kdim"] * (c["rows"] + hit * c["n"])) + 2 * p * c["n"],
                "flops": 2 * c["rows"] * c["n"] * c["kdim"]}
    return {"bytes": int(_bits(c["fmt"]) / 8 * c["rows"] * (c["m"] + c["n"])) + 2 * c["experts"] * c["m"] * c["n"],
            "flops": 2 * c["rows"] * c["m"] * c["n"]}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _randn(g, shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _operand(g, shape, fmt, std):
    """Codes and scales of a normal tensor of the given shape as its quantizer leaves
    them: the elements' codes relative to their block's amax, and the block scales."""
    rows, k = shape
    blk = BLOCK[fmt]
    byte = torch.empty((rows, k // (1 if fmt == "mxfp8" else 2)), dtype=torch.uint8, device=DEV)
    byte.random_(0, 256, generator=g)
    q = np.arange(256)
    if fmt == "mxfp8":
        # E4M3 codes: a sign and a magnitude spread over the normal range below 448
        lut = (q & 0x80) | np.clip(0x7E - ((q & 0x7F) ** 2) // 320, 0, 0x7E)
    else:
        # both nibbles through the code frequencies of normal data scaled to a block amax of 6
        mag = np.array([0, 1, 2, 2, 3, 4, 5, 6])
        nib = np.concatenate([mag, mag | 8])
        nib[7] = 7
        lut = nib[q & 15] | (nib[q >> 4] << 4)
    codes = torch.from_numpy(lut.astype(np.uint8)).to(DEV)[byte.int()] if rows * k <= 1 << 26 else _lut_rows(byte, lut)
    s = torch.randint(0, 256, (rows, k // blk), generator=g, device=DEV, dtype=torch.uint8)
    if fmt == "nvfp4":
        scales = (0x66 + (s >> 4)).to(torch.uint8)           # E4M3 112 .. 416 under the per-tensor scale
    else:
        top = int(round(math.log2(std))) + 127 - (7 if fmt == "mxfp8" else 1)
        scales = (top - (s < 40).to(torch.uint8) + (s > 200).to(torch.uint8)).to(torch.uint8)
    return codes, scales


def _lut_rows(byte, lut):
    t = torch.from_numpy(lut.astype(np.uint8)).to(DEV)
    flat = byte.view(-1)
    step = 1 << 26
    return torch.cat([t[flat[i:i + step].int()] for i in range(0, flat.numel(), step)]).view(byte.shape)


def _moe_layout(c, g):
    """A routing of the case's tokens: what moe_route returns, from uneven random experts."""
    t, e, k, al = c["tokens"], c["experts"], c["k"], c["align"]
    logits = torch.randn((t, e), generator=g, device=DEV) + 0.5 * torch.randn((1, e), generator=g, device=DEV)
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(torch.gather(logits, 1, ids), 1)
    off, row_of, src = _plan(ids, torch.ones_like(ids, dtype=torch.bool), e, al, _buffer_rows(t * k, e, al))
    return w, off, row_of, src


def prepare(c, seed):
    g = _gen(seed)
    op = c["op"]
    st = dict(case=c)
    if op == "norm":
        r, d = c["rows"], c["cols"]
        t = torch.float32 if c["res"] == "f32" else torch.bfloat16
        st.update(x=_randn(g, (r, d), 1.0, t), o=_randn(g, (r, d), 0.5), w_pre=1 + 0.2 * _randn(g, (d,), 1.0, torch.float32),
                  w_post=1 + 0.2 * _randn(g, (d,), 1.0, torch.float32) if c["post"] else None, gate=None, alpha=0.875)
        if c["gate"] == "channel":
            st["gate"] = _randn(g, (d,), 0.5, torch.float32)
        elif c["gate"] == "row":
            st["gate"] = _randn(g, (r, 1), 0.5, torch.float32)
        elif c["gate"] == "full":
            st["gate"] = torch.sigmoid(_randn(g, (r, d), 1.0, torch.float32)).to(torch.bfloat16)
        if c["dir"] == "bwd":
            f = _norm_fwd(st, torch.float32)
            st.update(r=f[0].to(t), rstd_pre=f[2], rstd_post=f[3], d_r=_randn(g, (r, d), 0.01, t), d_h=_randn(g, (r, d), 0.01))
        return st
    if op == "route":
        t, e = c["tokens"], c["experts"]
        lg = torch.randn((t, e), generator=g, device=DEV) * 2
        pad = torch.rand((t, 1), generator=g, device=DEV) < 0.01
        off = torch.rand((t, e), generator=g, device=DEV) < 0.05
        if t > 64:                       # padding tokens and experts that a token may not use
            lg = lg.masked_fill(pad | off, float("-inf"))
        st.update(logits=lg.to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16),
                  bias=0.1 * torch.randn((e,), generator=g, device=DEV), scale=1.5)
        if c["dir"] == "both":
            st["d_w"] = torch.randn((t, c["k"]), generator=g, device=DEV)
        return st
    if op in ("gather", "combine"):
        w, off, row_of, src = _moe_layout(c, g)
        t, h = c["tokens"], c["cols"]
        st.update(weights=w, offsets=off, row_of=row_of, src=src)
        if op == "gather":
            st.update(x=_randn(g, (t, h)))
        else:
            st.update(y=_randn(g, (src.numel(), h)), d_out=_randn(g, (t, h), 0.01))
        return st
    n, off = _groups(c)
    p = _buffer_rows(c["rows"], c["experts"], c["align"])
    st.update(sizes=n, ends=off, offsets=torch.tensor(off, dtype=torch.int32, device=DEV), a_amax=None, b_amax=None)
    fmt = c["fmt"]
    if op == "grouped":
        st["a"] = _operand(g, (p, c["kdim"]), fmt, 1.0)
        bc, bs = _operand(g, (c["experts"] * c["n"], c["kdim"]), fmt, 0.03)
        st["b"] = (bc.view(c["experts"], c["n"], -1), bs.view(c["experts"], c["n"], -1))
        if fmt == "nvfp4":
            st["a_amax"] = 4 + torch.rand(1, generator=g, device=DEV)
            st["b_amax"] = 0.1 + 0.05 * torch.rand(c["experts"], generator=g, device=DEV)
    else:
        st["a"] = _operand(g, (c["m"], p), fmt, 0.01)
        st["b"] = _operand(g, (c["n"], p), fmt, 1.0)
        if fmt == "nvfp4":
            st["a_amax"] = 0.05 + 0.01 * torch.rand(1, generator=g, device=DEV)
            st["b_amax"] = 4 + torch.rand(1, generator=g, device=DEV)
    return st


# ---------------------------------------------------------------- plain forms (FP32)

def _norm_fwd(s, dt):
    """r, h, rstd_pre, rstd_post in dt, unrounded."""
    x, o = s["x"].to(dt), s["o"].to(dt)
    rp = None
    if s["w_post"] is not None:
        rp = torch.rsqrt((o * o).mean(1) + 1e-6)
        o = o * rp[:, None] * s["w_post"].to(dt)
    r = s["alpha"] * x + (o if s["gate"] is None else s["gate"].to(dt) * o)
    rr = torch.rsqrt((r * r).mean(1) + 1e-6)
    return r, r * rr[:, None] * s["w_pre"].to(dt), rr, rp


def _plain_norm(s):
    if s["case"]["dir"] == "fwd":
        r, h, rr, rp = _norm_fwd(s, torch.float32)
        h = h.to(torch.bfloat16)
        return dict(r=r.to(s["x"].dtype), h=h, rstd_pre=rr, rstd_post=rp, amax=h.abs().max().float().reshape(1))
    dh, w = s["d_h"].float(), s["w_pre"]
    rn = s["r"].float() * s["rstd_pre"][:, None]
    a = dh * w
    G = s["d_r"].float() + s["rstd_pre"][:, None] * (a - rn * (a * rn).mean(1, keepdim=True))
    o = s["o"].float()
    on = o if s["w_post"] is None else o * s["rstd_post"][:, None]
    n = on if s["w_post"] is None else on * s["w_post"]
    gn = G if s["gate"] is None else G * s["gate"].float()
    out = dict(d_x=(s["alpha"] * G).to(s["r"].dtype), d_w_pre=(dh * rn).sum(0), d_w_post=None, d_gate=None)
    if s["w_post"] is None:
        out["d_o"] = gn.to(torch.bfloat16)
    else:
        b = gn * s["w_post"]
        out["d_o"] = (s["rstd_post"][:, None] * (b - on * (b * on).mean(1, keepdim=True))).to(torch.bfloat16)
        out["d_w_post"] = (gn * on).sum(0)
    kind = s["case"]["gate"]
    if kind == "channel":
        out["d_gate"] = (G * n).sum(0)
    elif kind == "row":
        out["d_gate"] = (G * n).sum(1, keepdim=True)
    elif kind == "full":
        out["d_gate"] = (G * n).to(torch.bfloat16)
    return out


def _plan(ids, ok, e, align, rows):
    """offsets, row_of, src of the chosen experts (stable in token and slot order)."""
    t, k = ids.shape
    flat = torch.where(ok, ids, e).reshape(-1)
    cnt = (flat[None, :] == torch.arange(e, device=DEV)[:, None]).sum(1)
    start = torch.cumsum(cnt, 0) - cnt
    pad = (cnt + align - 1) // align * align
    ends = torch.cumsum(pad, 0)
    off = torch.cat([torch.zeros_like(ends[:1]), ends])
    order = torch.sort(flat, stable=True).indices
    se = flat[order]
    live = se < e
    at = torch.clamp(se, max=e - 1)
    row = torch.where(live, off[at] + torch.arange(t * k, device=DEV) - start[at], -1)
    row_of = torch.empty_like(row)
    row_of[order] = row
    src = torch.full((rows + 1,), -1, dtype=torch.int64, device=DEV)
    src[torch.where(live, row, rows)] = torch.where(live, order, -1)
    return off.int(), row_of.view(t, k).int(), src[:rows].int()


def _plain_route(s):
    c, k = s["case"], s["case"]["k"]
    lg = s["logits"].float()
    sc = lg + s["bias"]
    top = torch.sort(sc, dim=1, descending=True, stable=True)
    ids = top.indices[:, :k]
    ok = top.values[:, :k] > float("-inf")
    sel = torch.gather(lg, 1, ids)
    live = lambda v: torch.where(ok, v, torch.zeros_like(v))
    if c["scoring"] == "sigmoid":
        q = torch.sigmoid(sel)
        if c["normalize"]:
            z = -torch.nn.functional.softplus(-sel)
            z = torch.exp(z - torch.where(ok, z, float("-inf")).amax(1, keepdim=True))
            p = live(z) / live(z).sum(1, keepdim=True)
        else:
            p = q
    else:
        m = lg.amax(1, keepdim=True)
        full = torch.exp(lg - m)
        if c["normalize"]:
            z = torch.exp(sel - torch.where(ok, sel, float("-inf")).amax(1, keepdim=True))
            p = live(z) / live(z).sum(1, keepdim=True)
        else:
            full = full / full.sum(1, keepdim=True)
            p = torch.gather(full, 1, ids)
    p = live(p)
    rows = _buffer_rows(c["tokens"] * k, c["experts"], c["align"])
    off, row_of, src = _plan(ids, ok, c["experts"], c["align"], rows)
    out = dict(experts=torch.where(ok, ids, -1).int(), weights=s["scale"] * p, offsets=off, row_of=row_of, src=src)
    if c["dir"] == "both":
        dp = live(s["scale"] * s["d_w"])
        if c["scoring"] == "softmax" and not c["normalize"]:
            full = torch.where(ok.any(1, keepdim=True), full, torch.zeros_like(full))
            d = full * (torch.zeros_like(lg).scatter(1, ids, dp) - (dp * p).sum(1, keepdim=True))
        else:
            ds = p * (dp - (dp * p).sum(1, keepdim=True)) if c["normalize"] else dp * p
            if c["scoring"] == "sigmoid":
                ds = ds * torch.sigmoid(-sel)
            d = torch.zeros_like(lg).scatter(1, ids, live(ds))
        out["d_logits"] = d.to(s["logits"].dtype)
    return out


def _plain_gather(s):
    src = s["src"].long()
    x = s["x"][torch.clamp(src, min=0) // s["case"]["k"]]
    return torch.where((src >= 0)[:, None], x, torch.zeros_like(x))


def _plain_combine(s):
    w, row_of, src, k = s["weights"], s["row_of"].long(), s["src"].long(), s["case"]["k"]
    yf = s["y"].float()
    out = (w[:, :, None] * yf[row_of]).sum(1).to(torch.bfloat16)
    do = s["d_out"].float()
    a = torch.clamp(src, min=0)
    dy = torch.where((src >= 0)[:, None], w.reshape(-1)[a][:, None] * do[a // k], 0.0).to(torch.bfloat16)
    dw = (do[:, None, :] * yf[row_of]).sum(2)
    return dict(out=out, d_y=dy, d_weights=dw)


def _dequant(codes, scales, fmt):
    """FP32 values of codes and block scales, without the per-tensor scale."""
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
        v = torch.stack([e2m1[(codes & 15).int()], e2m1[(codes >> 4).int()]], -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.exp2(scales.float() - 127)
    return (v.unflatten(-1, (scales.shape[-1], BLOCK[fmt])) * s[..., None]).flatten(-2)


def _alpha(s, dt=torch.float32):
    """Product of the two per-tensor decode scales (one per expert for the grouped rows)."""
    if s["a_amax"] is None:
        return torch.ones(s["case"]["experts"], device=DEV, dtype=dt)
    return ((s["a_amax"].to(dt) / 2688) * (s["b_amax"].to(dt) / 2688)).expand(s["case"]["experts"])


def _plain_grouped(s):
    c, off, al = s["case"], s["ends"], _alpha(s)
    a = _dequant(*s["a"], c["fmt"])
    parts = [(a[b:e] @ _dequant(s["b"][0][i], s["b"][1][i], c["fmt"]).t() * al[i]).to(torch.bfloat16)
             for i, (b, e) in enumerate(zip(off, off[1:])) if e > b]
    tail = torch.zeros((a.shape[0] - off[-1], c["n"]), dtype=torch.bfloat16, device=DEV)
    return torch.cat(parts + [tail])


def _plain_wgrad(s):
    c, off, al = s["case"], s["ends"], _alpha(s)
    a, b = _dequant(*s["a"], c["fmt"]), _dequant(*s["b"], c["fmt"])
    return torch.stack([(a[:, p:q] @ b[:, p:q].t() * al[i]).to(torch.bfloat16)
                        for i, (p, q) in enumerate(zip(off, off[1:]))])


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import fp8_quantized_gemm_amd as bsq
    c = s["case"]
    op = c["op"]
    if op == "norm":
        if c["dir"] == "fwd":
            f = bsq.block_norm(s["x"], o=s["o"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"], alpha=s["alpha"],
                               eps=1e-6, amax=True)
            return {k: f[k] for k in ("r", "h", "rstd_pre", "rstd_post", "amax")}
        f = bsq.block_norm_backward(s["r"], o=s["o"], d_r=s["d_r"], d_h=s["d_h"], w_pre=s["w_pre"], w_post=s["w_post"],
                                    gate=s["gate"], rstd_pre=s["rstd_pre"], rstd_post=s["rstd_post"], alpha=s["alpha"])
        return {k: f[k] for k in ("d_x", "d_w_pre", "d_w_post", "d_gate", "d_o")}
    if op == "route":
        f = bsq.moe_route(s["logits"], c["k"], bias=s["bias"], scoring=c["scoring"], normalize=c["normalize"],
                          scale=s["scale"], align=c["align"])
        out = {k: f[k] for k in ("experts", "weights", "offsets", "row_of", "src")}
        if c["dir"] == "both":
            out["d_logits"] = bsq.moe_route_backward(s["logits"], f["experts"], s["d_w"], scoring=c["scoring"],
                                                     normalize=c["normalize"], scale=s["scale"])
        return out
    if op == "gather":
        return bsq.moe_gather(s["x"], s["src"], c["k"])
    if op == "combine":
        dy, dw = bsq.moe_combine_backward(s["d_out"], s["y"], s["src"], s["row_of"], s["weights"])
        return dict(out=bsq.moe_combine(s["y"], s["row_of"], s["weights"]), d_y=dy, d_weights=dw)
    if op == "grouped":
        return bsq.bs_gemm_grouped(c["fmt"], *s["a"], *s["b"], s["offsets"], a_amax=s["a_amax"], b_amax=s["b_amax"])
    return bsq.bs_gemm_grouped_wgrad(c["fmt"], *s["a"], *s["b"], s["offsets"], a_amax=s["a_amax"], b_amax=s["b_amax"])


def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "route": _plain_route, "gather": _plain_gather, "combine": _plain_combine,
            "grouped": _plain_grouped, "wgrad": _plain_wgrad}[s["case"]["op"]](s)


# ---------------------------------------------------------------- definitions in 64 bits

def _values64(codes, scales, fmt):
    """FP64 values from the formats' bit fields."""
    def minifloat(c, ebits, mbits, bias):
        e, m = (c >> mbits) & ((1 << ebits) - 1), c & ((1 << mbits) - 1)
        lead = (e > 0).double()
        mag = torch.ldexp(lead + m.double() / (1 << mbits), torch.clamp(e, min=1) - bias)
        return torch.where((c >> (ebits + mbits)) & 1 == 1, -mag, mag)
    c = codes.int()
    if fmt == "mxfp8":
        v = minifloat(c, 4, 3, 7)
    else:
        v = torch.empty((*c.shape[:-1], c.shape[-1] * 2), dtype=torch.float64, device=DEV)
        v[..., 0::2] = minifloat(c & 15, 2, 1, 1)
        v[..., 1::2] = minifloat(c >> 4, 2, 1, 1)
    s = minifloat(scales.int(), 4, 3, 7) if fmt == "nvfp4" else torch.ldexp(torch.ones((), device=DEV, dtype=torch.float64),
                                                                            scales.int() - 127)
    return v * torch.repeat_interleave(s, BLOCK[fmt], dim=-1)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    D = torch.float64
    if op == "norm":
        x, o, wq = s["x"].to(D), s["o"].to(D), s["w_pre"].to(D)
        g = 1.0 if s["gate"] is None else s["gate"].to(D)
        wp = None if s["w_post"] is None else s["w_post"].to(D)
        if c["dir"] == "fwd":
            rp = None if wp is None else 1 / torch.sqrt(o.square().sum(1) / c["cols"] + 1e-6)
            n = o if wp is None else o * wp * rp[:, None]
            r = s["alpha"] * x + g * n
            rr = 1 / torch.sqrt(r.square().sum(1) / c["cols"] + 1e-6)
            h = r * wq * rr[:, None]
            return dict(r=r, h=h, rstd_pre=rr, rstd_post=rp, amax=None)
        # y = u * rs * w with the row's rs = (mean u^2 + eps)^-1/2 given: the adjoint of its Jacobian
        def back(dy, u, rs, w):
            v = dy * w
            return rs[:, None] * v - (rs ** 3)[:, None] * u * (v * u).sum(1, keepdim=True) / c["cols"]
        r, dh = s["r"].to(D), s["d_h"].to(D)
        rr = s["rstd_pre"].to(D)
        G = s["d_r"].to(D) + back(dh, r, rr, wq)
        out = dict(d_x=s["alpha"] * G, d_w_pre=torch.einsum("rc,rc,r->c", dh, r, rr), d_w_post=None, d_gate=None)
        Gg = G * g
        if wp is None:
            n, out["d_o"] = o, Gg
        else:
            rp = s["rstd_post"].to(D)
            n, out["d_o"] = o * rp[:, None] * wp, back(Gg, o, rp, wp)
            out["d_w_post"] = torch.einsum("rc,rc,r->c", Gg, o, rp)
        if c["gate"] != "none":
            out["d_gate"] = {"channel": lambda v: v.sum(0), "row": lambda v: v.sum(1, keepdim=True),
                             "full": lambda v: v}[c["gate"]](G * n)
        return out
    if op == "route":
        lg32 = s["logits"].float()
        key = lg32 + s["bias"]                                  # the selection score is an FP32 sum
        lg, k, e, t = lg32.to(D), c["k"], c["experts"], c["tokens"]
        left, chosen = key.clone(), []
        for _ in range(min(k, e)):                              # repeated first maximum
            best = left.amax(1, keepdim=True)
            i = torch.where(left == best, torch.arange(e, device=DEV), e).amin(1, keepdim=True)
            chosen.append(torch.where(best > float("-inf"), i, -1))
            left = left.scatter(1, i, float("-inf"))
        ids = torch.cat(chosen, 1)
        hot = torch.zeros((t, e + 1), dtype=D, device=DEV).scatter(1, torch.where(ids >= 0, ids, e), 1.0)[:, :e]
        sig = 1 / (1 + torch.exp(-lg))
        if c["scoring"] == "sigmoid":
            z = sig * hot
            p = z / z.sum(1, keepdim=True).clamp_min(1e-300) if c["normalize"] else z
        else:
            z = torch.exp(lg - lg.amax(1, keepdim=True).clamp_min(-1e30))
            full = z / z.sum(1, keepdim=True).clamp_min(1e-300)
            z = z * hot
            p = z / z.sum(1, keepdim=True).clamp_min(1e-300) if c["normalize"] else full * hot
        at = torch.clamp(ids, min=0)
        w = torch.where(ids >= 0, s["scale"] * torch.gather(p, 1, at), 0.0)
        out = dict(experts=None, weights=w, offsets=None, row_of=None, src=None)
        if c["dir"] == "both":
            gsel = s["scale"] * torch.where(ids >= 0, s["d_w"].to(D), 0.0)
            gd = torch.zeros((t, e + 1), dtype=D, device=DEV).scatter(1, torch.where(ids >= 0, ids, e), gsel)[:, :e]
            mean = (gd * p).sum(1, keepdim=True)
            if c["scoring"] == "softmax":
                q = p if c["normalize"] else full * (hot.sum(1, keepdim=True) > 0)
                d = q * (gd - mean)
            elif c["normalize"]:
                d = p * (gd - mean) * (1 - sig)
            else:
                d = gd * sig * (1 - sig)
            out["d_logits"] = d
        return out
    if op == "gather":
        src = s["src"].long()
        out = torch.zeros((src.numel(), c["cols"]), dtype=D, device=DEV)
        rows = torch.nonzero(src >= 0)[:, 0]
        out[rows] = s["x"].to(D)[torch.div(src[rows], c["k"], rounding_mode="floor")]
        return out
    if op == "combine":
        t, k = s["weights"].shape
        w, y, do = s["weights"].to(D), s["y"].to(D), s["d_out"].to(D)
        at = s["row_of"].long()
        out, dy, dw = torch.zeros_like(do), torch.zeros_like(y), torch.empty((t, k), dtype=D, device=DEV)
        for j in range(k):
            yj = y[at[:, j]]
            out += w[:, j:j + 1] * yj
            dw[:, j] = torch.einsum("th,th->t", do, yj)
            dy[at[:, j]] = w[:, j:j + 1] * do
        return dict(out=out, d_y=dy, d_weights=dw)
    # grouped products: group by group in FP64
    off, fmt = s["ends"], c["fmt"]
    al = _alpha(s, D)
    if op == "grouped":
        out = torch.zeros((s["a"][0].shape[0], c["n"]), dtype=D, device=DEV)
        for i in range(c["experts"]):
            b, e = off[i], off[i + 1]
            if e > b:
                out[b:e] = al[i] * torch.matmul(_values64(s["a"][0][b:e], s["a"][1][b:e], fmt),
                                                _values64(s["b"][0][i], s["b"][1][i], fmt).t())
        return out
    a, b = _values64(*s["a"], fmt), _values64(*s["b"], fmt)
    out = torch.zeros((c["experts"], c["m"], c["n"]), dtype=D, device=DEV)
    for i in range(c["experts"]):
        if off[i + 1] > off[i]:
            out[i] = al[i] * torch.matmul(a[:, off[i]:off[i + 1]], b[:, off[i]:off[i + 1]].t())
    return out


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(8)]:
        print(case, work(case))
