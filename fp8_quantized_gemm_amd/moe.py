"""One mixture-of-experts MLP block's NVFP4 training step, driven through the C ABI.

The expert counterpart of mlp.MLPLayer: the same recipe (NVFP4 pretraining post:
the data-flow paragraph after Figure 1 and the recipe's ingredients) with the
tokens sorted by expert and the products grouped.  Every step is a libbsq call on
the current stream; the router's logits are the caller's (a product of the model's
own, usually kept in higher precision).

  open      r = alpha * x + gate * norm(o) * w_post;  h = norm(r) * w_pre
              (block_norm: closes the block before, opens this one)
  forward   route the logits; gather h into expert rows (groups padded to 32)
            q(xp): rows RNE, columns RNE + RHT
            q(W_gu), q(W_down) per expert: 16x16 tiles, under the amax the last
              update of the stacked master weight produced
            Y_gu = xp . W_gu[e]^T (grouped);  H = SwiGLU(Y_gu) with its amaxes
            q(H);  Y_down = H . W_down[e]^T (grouped)
            y = combine of the experts' rows with the routing weights
  backward  combine backward: dY_down and the weights' gradient; route backward
            q(dY_down): rows SR, columns SR + RHT
            dH = dY_down . W_down[e];  dW_down[e] = dY_down^T . H (grouped over rows)
            dY_gu = SwiGLU backward;  q(dY_gu)
            dxp = dY_gu . W_gu[e];  dW_gu[e] = dY_gu^T . xp
            dh = combine of dxp without weights
  close     block_norm backward: dx, do and the norm's and gate's gradients
  update    W <- W - lr * dW on the FP32 masters (stacked over the experts), or with
              optimizer "muon" the orthogonalised update of an FP32 momentum, each
              expert's gate, up and down projection a matrix of its own

y is the next block_norm's o.  Groups are padded to 32 rows of zeros and the
buffers to a multiple of 512 rows, so the column-quantized operands' 16-row blocks
and RHT chunks never cross a group.
"""

import torch

from . import (_check, _on_device, _ptr, _stream, block_norm, block_norm_backward, bs_gemm_grouped,
               bs_gemm_grouped_wgrad, lib, master_weight_update, moe_combine, moe_combine_backward,
               moe_gather, moe_route, moe_route_backward, muon_update, quantize_transpose,
               quantize_transpose_amax, swiglu, swiglu_backward)
from .mlp import muon_options

ALIGN = 32


class MoELayer:
    """w_gu: FP32 masters [E, 2F, hidden] (gate rows first); w_down: [E, hidden, F]; both
    copied.  norm: dict of block_norm's w_pre, w_post, gate, alpha, eps (w_pre
    required).  scoring, normalize, scale, bias, score_bias: moe_route's.  hidden %
    16 == 0, F % 16 == 0.  optimizer: "sgd", or "muon" with muon a dict of muon_update's
    options (its defaults otherwise) and lr its lr."""

    def __init__(self, w_gu, w_down, k, norm, scoring="softmax", normalize=True, scale=1.0, bias=None,
                 rht=True, rht_signs=0, sr_seed=0, lr=1e-4, score_bias=None, optimizer="sgd", muon=None):
        if not (w_gu.is_cuda and w_down.is_cuda and w_gu.device == w_down.device):
            raise ValueError("the master weights must be CUDA tensors on one device")
        E, F2, Hd = w_gu.shape
        F = F2 // 2
        if tuple(w_down.shape) != (E, Hd, F) or F2 != 2 * F or Hd % 16 or F % 16:
            raise ValueError("w_gu must be [E, 2F, hidden] and w_down [E, hidden, F], F and hidden multiples of 16")
        if norm.get("w_pre") is None:
            raise ValueError("norm needs w_pre: the block's input is normalised")
        if optimizer not in ("sgd", "muon") or (muon is not None and optimizer != "muon"):
            raise ValueError("optimizer must be 'sgd', or 'muon' (which alone takes muon)")
        self.optimizer, self.muon = optimizer, muon_options(muon)
        self.dev, self.E, self.F, self.Hd, self.k = w_gu.device, E, F, Hd, int(k)
        self.norm, self.bias, self.score_bias = dict(norm), bias, score_bias
        self.routing = dict(scoring=scoring, normalize=normalize, scale=scale)
        self.rht, self.signs, self.seed, self.lr, self.it = bool(rht), int(rht_signs), int(sr_seed), float(lr), 0
        self.w32 = {"W_gu": w_gu.detach().float().contiguous().clone(),
                    "W_down": w_down.detach().float().contiguous().clone()}
        u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=self.dev)
        self.wbf, self.wamax, self.wq, self.grad = {}, {}, {}, {}
        for n, w in self.w32.items():
            _, R, C = w.shape
            self.wbf[n] = torch.empty(w.shape, dtype=torch.bfloat16, device=self.dev)
            self.wq[n] = dict(rc=u8(E, R, C // 2), rs=u8(E, R, C // 16), cc=u8(E, C, R // 2), cs=u8(E, C, R // 16))
            # the BF16 working copies and their amaxes: an update with a zero gradient
            self.grad[n] = torch.zeros(w.shape, dtype=torch.bfloat16, device=self.dev)
            self._update(n, 0.0)
        if optimizer == "muon":
            self.momentum = {n: torch.zeros_like(w) for n, w in self.w32.items()}

    def _update_muon(self, n):
        w = self.w32[n]
        shape = (2 * self.E, self.F, self.Hd) if n == "W_gu" else w.shape    # gate and up rows apart
        v = lambda t: t.view(shape)
        u = muon_update(v(w), v(self.momentum[n]), v(self.grad[n]), self.lr, w_bf16=v(self.wbf[n]), **self.muon)
        self.wamax[n] = u["amax"]

    @_on_device
    def _update(self, n, lr):
        u = master_weight_update(self.w32[n], self.grad[n], lr, w_bf16=self.wbf[n])
        self.wamax[n] = u["amax"]

    def _quantize_weight(self, n):
        q, w, am = self.wq[n], self.wbf[n], _ptr(self.wamax[n])
        _, R, C = w.shape
        for e in range(self.E):
            st = lib().quantize_transpose_amax(_ptr(w[e]), R, C, 16, 0, 0, 0, 0, 0, am, am, _ptr(q["rc"][e]),
                                               _ptr(q["rs"][e]), _ptr(q["cc"][e]), _ptr(q["cs"][e]),
                                               _stream(self.dev))
            _check("quantize_transpose_amax " + n, st)

    def _quantize(self, x, rnd, offset, amax=None):
        kw = dict(rnd=rnd, seed=self.seed, offset=offset, rht_col=self.rht, rht_signs=self.signs)
        if amax is None:
            return quantize_transpose(x, **kw)
        q = quantize_transpose_amax(x, *amax, **kw)
        return dict(q, row_amax=amax[0], col_amax=amax[1])

    def _product(self, q, n, side):
        w = self.wq[n]
        return bs_gemm_grouped("nvfp4", q["row_codes"], q["row_scales"], w[side + "c"], w[side + "s"],
                               self.route["offsets"], q["row_amax"], self.wamax[n])

    def _wgrad(self, qa, qb, n):
        bs_gemm_grouped_wgrad("nvfp4", qa["col_codes"], qa["col_scales"], qb["col_codes"], qb["col_scales"],
                              self.route["offsets"], qa["col_amax"], qb["col_amax"], out=self.grad[n])

    @_on_device
    def open(self, x, o=None):
        """(r, h): the residual after the block before (its output o), and this
        block's normalised input."""
        n = self.norm
        kw = dict(alpha=n.get("alpha", 1.0), w_post=n.get("w_post"), gate=n.get("gate")) if o is not None else {}
        f = block_norm(x, o, w_pre=n["w_pre"], eps=n.get("eps", 1e-6), **kw)
        self.saved = dict(f, r=f["r"] if o is not None else x, o=o, kw=kw)
        return self.saved["r"], f["h"]

    @_on_device
    def forward(self, h, logits):
        """y [T, hidden] (bfloat16) of h [T, hidden] and the router's logits [T, E]."""
        self.logits = logits
        self.route = moe_route(logits, self.k, bias=self.bias, score_bias=self.score_bias, align=ALIGN, **self.routing)
        xp = moe_gather(h, self.route["src"], self.k)
        self.qx = self._quantize(xp, "rne", 0)
        self._quantize_weight("W_gu")
        self.y_gu = self._product(self.qx, "W_gu", "r")
        s = swiglu(self.y_gu, rht_col=self.rht, rht_signs=self.signs)
        self.qh = self._quantize(s["h"], "rne", 0, (s["amax_row"], s["amax_col"]))
        self._quantize_weight("W_down")
        self.y_down = self._product(self.qh, "W_down", "r")
        return moe_combine(self.y_down, self.route["row_of"], self.route["weights"])

    @_on_device
    def backward(self, d_y):
        """(d_h, d_logits); the experts' weight gradients are left in grad."""
        r, off = self.route, 2 * self.it
        d_down, d_w = moe_combine_backward(d_y, self.y_down, r["src"], r["row_of"], r["weights"])
        d_logits = moe_route_backward(self.logits, r["experts"], d_w, **self.routing)
        self.qd = self._quantize(d_down, "sr", off)
        d_act = self._product(self.qd, "W_down", "c")
        self._wgrad(self.qd, self.qh, "W_down")
        s = swiglu_backward(self.y_gu, d_act, rht_col=self.rht, rht_signs=self.signs)
        self.qg = self._quantize(s["d_y_gu"], "sr", off + 1, (s["amax_row"], s["amax_col"]))
        d_xp = self._product(self.qg, "W_gu", "c")
        self._wgrad(self.qg, self.qx, "W_gu")
        return moe_combine(d_xp, r["row_of"]), d_logits

    @_on_device
    def close(self, d_r, d_h):
        """block_norm_backward's gradients from those of open's r and h."""
        s = self.saved
        return block_norm_backward(s["r"], o=s["o"], d_r=d_r, d_h=d_h, w_pre=self.norm["w_pre"],
                                   rstd_pre=s["rstd_pre"], rstd_post=s["rstd_post"], **s["kw"])

    @_on_device
    def update(self):
        for n in self.w32:
            if self.optimizer == "muon":
                self._update_muon(n)
            else:
                self._update(n, self.lr)
        self.it += 1
