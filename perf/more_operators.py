"""Cases of the 8-bit integer products with a scale for each token and channel, with
their quantizers, and of the orthogonalised weight updates.

`own` false: run() computes the plain torch form in FP32; true: the library's
entry points.  Sizes: 4096 / 14336 / 28672 are the repository's 8B MLP; the
others are generic expert and odd shapes.
"""

import math
import random

import torch

own = False

DEV = "cuda"
FLT_MAX = torch.finfo(torch.float32).max
COEFS = (3.4445, -4.7750, 2.0315)
STEPS, EPS, MU, LR, DECAY = 5, 1e-7, 0.95, 1e-3, 0.1


def listed():
    return [
        # BF16 activations through 8-bit weights (quantized within the call) -----------
        # one decoded token through the gate/up weights: a stream of the weights
        dict(name="linear_token", op="linear", rows=1, n=28672, kdim=4096, bias=False),
        # a decode batch of odd size on a small layer with a bias: latency
        dict(name="linear_decode", op="linear", rows=37, n=2048, kdim=1408, bias=True),
        # a ragged prompt through the down weights
        dict(name="linear_prompt", op="linear", rows=4093, n=4096, kdim=14336, bias=False),
        # products of quantized operands ------------------------------------------------
        # the forward gate/up product of a training batch
        dict(name="gemm_fprop", op="gemm", m=16384, n=28672, kdim=4096),
        # a weight gradient: the reduction runs over a batch's tokens
        dict(name="gemm_wgrad", op="gemm", m=4096, n=14336, kdim=8192),
        # quantizers ----------------------------------------------------------------------
        # a decode batch's activations, rows only
        dict(name="quant_rows", op="quant", rows=257, cols=14336, col=False),
        # a training batch's activations, rows (FPROP) and columns (WGRAD)
        dict(name="quant_both", op="quant", rows=16384, cols=4096, col=True),
        # orthogonalisation ---------------------------------------------------------------
        # one small odd matrix: launches
        dict(name="ortho_small", op="ortho", experts=0, rows=200, cols=136, dtype="f32"),
        # a stack of expert weights' gradients
        dict(name="ortho_experts", op="ortho", experts=16, rows=1408, cols=2048, dtype="bf16"),
        # weight updates ------------------------------------------------------------------
        # a stack of small experts, odd sizes
        dict(name="update_experts", op="update", experts=8, rows=520, cols=1000, nesterov=True),
        # a square projection
        dict(name="update_square", op="update", experts=0, rows=2048, cols=2048, nesterov=False),
        # the 8B MLP's down weights
        dict(name="update_down", op="update", experts=0, rows=4096, cols=14336, nesterov=True),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["linear", "linear", "gemm", "quant", "ortho", "update"])
    kdim = lambda: rng.choice([1024, 2048, 4096, _log_int(rng, 256, 8192, 32), _log_int(rng, 256, 8192, 16), _log_int(rng, 250, 4099)])
    if op == "linear":
        return dict(op=op, rows=_log_int(rng, 1, 4096), n=_log_int(rng, 256, 14336), kdim=kdim(), bias=rng.random() < 0.5)
    if op == "gemm":
        return dict(op=op, m=_log_int(rng, 64, 8192), n=_log_int(rng, 256, 14336), kdim=kdim())
    if op == "quant":
        cols = _log_int(rng, 64, 16384, 16)
        rows = _log_int(rng, 1, 16384 * 4096 // max(cols, 4096))
        col = rng.random() < 0.5
        return dict(op=op, rows=max(16, rows // 16 * 16) if col else rows, cols=cols, col=col)
    e = rng.choice([0, 0, 2, 8, 20])
    r, c = _log_int(rng, 48, 4096), _log_int(rng, 48, 4096)
    if e:
        r, c = min(r, 2048), min(c, 2048)
    if op == "ortho":
        return dict(op=op, experts=e, rows=r, cols=c, dtype=rng.choice(["bf16", "f32"]))
    return dict(op=op, experts=e, rows=r, cols=c, nesterov=rng.random() < 0.5)


def work(c):
    op = c["op"]
    if op in ("linear", "gemm"):
        m, n, k = c.get("rows", c.get("m")), c["n"], c["kdim"]
        a = 2 * m * k if op == "linear" else m * k + 4 * m
        return {"bytes": a + n * k + 4 * n + 2 * m * n + (4 * n if c.get("bias") else 0), "flops": 2 * m * n * k}
    if op == "quant":
        n = c["rows"] * c["cols"]
        return {"bytes": 3 * n + 4 * c["rows"] + (n + 4 * c["cols"] if c["col"] else 0), "flops": 4 * n}
    e, r, d = max(1, c["experts"]), c["rows"], c["cols"]
    s, n = min(r, d), max(r, d)
    # A = X X^T and its square are symmetric: half of each is work
    flops = e * STEPS * (s * s * n + s * s * s + 2 * s * s * n)
    el = e * r * d
    if op == "ortho":
        return {"bytes": el * (4 if c["dtype"] == "f32" else 2) + 2 * el, "flops": flops}
    return {"bytes": el * (2 + 8 + 8 + 2), "flops": flops}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _randn(g, shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _activations(g, shape):
    """Normal values of which one in a thousand is fifty times as large, on rows of
    different sizes; every 61st row (a padding token) is zero."""
    x = torch.randn(shape, generator=g, device=DEV)
    x = torch.where(torch.rand(shape, generator=g, device=DEV) < 1e-3, 50 * x, x)
    x *= torch.exp(0.5 * torch.randn((shape[0], 1), generator=g, device=DEV))
    x[60::61] = 0
    return x.to(torch.bfloat16)


def _gradient(g, e, r, c, dtype):
    """Gradients of weight matrices as batches leave them: a few strong directions of
    falling size over a broad floor, channels of different sizes."""
    shape = (max(1, e), r, c)
    k = max(1, min(r, c) // 16)
    u = torch.randn((shape[0], r, k), generator=g, device=DEV)
    v = torch.randn((shape[0], k, c), generator=g, device=DEV)
    x = torch.matmul(u * (4.0 / torch.arange(1, k + 1, device=DEV).sqrt()), v) / math.sqrt(k)
    x += torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp(0.3 * torch.randn((shape[0], 1, c), generator=g, device=DEV)) * 1e-4
    return (x if e else x[0]).to(dtype)


def prepare(c, seed):
    g = _gen(seed)
    op = c["op"]
    s = dict(case=c)
    if op == "linear":
        w = _randn(g, (c["n"], c["kdim"]), 0.02)
        s.update(x=_activations(g, (c["rows"], c["kdim"])), w=_quantize(w), bias=None)
        if c["bias"]:
            s["bias"] = _randn(g, (c["n"],), 0.1, torch.float32)
    elif op == "gemm":
        s.update(a=_quantize(_activations(g, (c["m"], c["kdim"]))), b=_quantize(_randn(g, (c["n"], c["kdim"]), 0.02)))
    elif op == "quant":
        s["x"] = _activations(g, (c["rows"], c["cols"]))
    elif op == "ortho":
        s["x"] = _gradient(g, c["experts"], c["rows"], c["cols"], torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
    else:
        grad = _gradient(g, c["experts"], c["rows"], c["cols"], torch.bfloat16)
        before = _gradient(g, c["experts"], c["rows"], c["cols"], torch.float32)
        s.update(grad=grad, momentum=5 * before, w=0.02 * torch.randn(grad.shape, generator=g, device=DEV))
        s["scale"] = 0.2 * math.sqrt(max(c["rows"], c["cols"]))
    return s


# ---------------------------------------------------------------- plain forms (FP32)

def _quantize(x, dim=1):
    """int8 codes and FP32 scales [rows] of the rows (dim 1) or columns (dim 0, codes transposed)."""
    f = x.float()
    amax = f.abs().amax(dim, keepdim=True)
    enc = torch.where(amax == 0, torch.ones_like(amax), (127.0 / amax).clamp(max=FLT_MAX))
    codes = torch.round(f * enc).clamp(-127, 127).to(torch.int8)
    return (codes if dim else codes.t().contiguous()), (1.0 / enc).reshape(-1)


def _product(a, sa, b, sb, bias=None):
    y = (a.float() @ b.float().t()) * (sa[:, None] * sb[None, :])
    return (y if bias is None else y + bias).to(torch.bfloat16)


def _newton_schulz(x):
    """FP32 orthogonalisation of x [..., R, C], FP32."""
    x = x.float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    a, b, c = COEFS
    for _ in range(STEPS):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.mT if tall else x


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "linear":
        return _product(*_quantize(s["x"]), *s["w"], s["bias"])
    if op == "gemm":
        return _product(*s["a"], *s["b"])
    if op == "quant":
        codes, scales = _quantize(s["x"])
        out = dict(row_codes=codes, row_scales=scales)
        if c["col"]:
            out["col_codes"], out["col_scales"] = _quantize(s["x"], 0)
        return out
    if op == "ortho":
        return _newton_schulz(s["x"]).to(torch.bfloat16)
    m, w, gr = s["momentum"], s["w"], s["grad"].float()
    m.mul_(MU).add_(gr)
    o = _newton_schulz(gr + MU * m if c["nesterov"] else m)
    w.mul_(1 - LR * DECAY).sub_(o, alpha=LR * s["scale"])
    return dict(w=w, momentum=m, w_bf16=w.to(torch.bfloat16))


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import fp8_quantized_gemm_amd as bsq
    c = s["case"]
    op = c["op"]
    if op == "linear":
        return bsq.int8_linear(s["x"], *s["w"], bias=s["bias"])
    if op == "gemm":
        return bsq.int8_gemm(*s["a"], *s["b"])
    if op == "quant":
        if c["col"]:
            q = bsq.int8_quantize_transpose(s["x"])
            return {k: q[k] for k in ("row_codes", "row_scales", "col_codes", "col_scales")}
        codes, scales = bsq.int8_quantize(s["x"])
        return dict(row_codes=codes, row_scales=scales)
    if op == "ortho":
        return bsq.orthogonalize(s["x"], steps=STEPS, coefs=COEFS, eps=EPS)
    u = bsq.muon_update(s["w"], s["momentum"], s["grad"], LR, mu=MU, nesterov=c["nesterov"], weight_decay=DECAY,
                        scale=s["scale"], steps=STEPS, coefs=COEFS, eps=EPS)
    return dict(w=s["w"], momentum=s["momentum"], w_bf16=u["w_bf16"])       # the amax is that of w_bf16


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------- definitions in 64 bits

def _scales64(x, dim):
    """(encode, decode) scales of an 8-bit row or column, FP32 numbers by definition:
    each is the exact quotient rounded once."""
    amax = x.double().abs().amax(dim, keepdim=True)
    enc = torch.where(amax == 0, 1.0, 127.0 / torch.where(amax == 0, 1.0, amax)).clamp(max=FLT_MAX).float().double()
    return enc, (1.0 / enc).float().double()


def _codes64(x, enc):
    """RNE of the FP32 product of x and the encode scale."""
    return torch.clamp(torch.round((x.double() * enc).float().double()), -127, 127)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op in ("linear", "gemm"):
        if op == "linear":
            enc, dec = _scales64(s["x"], 1)
            a, sa = _codes64(s["x"], enc), dec.reshape(-1)
            b, sb = s["w"]
        else:
            (a, sa), (b, sb) = s["a"], s["b"]
        bd, sbd = b.double(), sb.double()
        out = []
        for i in range(0, a.shape[0], 4096):
            y = torch.matmul(a[i:i + 4096].double(), bd.t())
            out.append(y * sa[i:i + 4096, None].double() * sbd)
        y = torch.cat(out)
        return y if s.get("bias") is None else y + s["bias"].double()
    if op == "quant":
        out = dict(row_codes=None, row_scales=_scales64(s["x"], 1)[1].reshape(-1))
        if c["col"]:
            out.update(col_codes=None, col_scales=_scales64(s["x"], 0)[1].reshape(-1))
        return out

    def polar(x):
        """The Newton-Schulz polynomial of x, matrix by matrix, through its singular values
        on the smaller side: x -> h(x x^T) x, h applied to the powers of one Gram matrix."""
        parts = []
        for y in (x if x.dim() == 3 else x[None]):
            t = y if y.shape[0] <= y.shape[1] else y.t().contiguous()
            t = t / (torch.linalg.vector_norm(t) + EPS)
            eye = torch.eye(t.shape[0], dtype=torch.float64, device=DEV)
            for _ in range(STEPS):
                gram = torch.matmul(t, t.t())
                t = torch.matmul(COEFS[0] * eye + torch.matmul(gram, COEFS[1] * eye + COEFS[2] * gram), t)
            parts.append(t if y.shape[0] <= y.shape[1] else t.t())
        return torch.stack(parts) if x.dim() == 3 else parts[0]

    if op == "ortho":
        return polar(s["x"].double())
    g64 = s["grad"].double()
    m = MU * s["momentum"].double() + g64
    w = (1 - LR * DECAY) * s["w"].double() - LR * s["scale"] * polar(MU * m + g64 if c["nesterov"] else m)
    return dict(w=w, momentum=m, w_bf16=w)


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(8)]:
        print(case, work(case))
