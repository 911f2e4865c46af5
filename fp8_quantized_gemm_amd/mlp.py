"""One transformer-MLP layer's NVFP4 (or 8-bit integer) training step, driven through the C ABI.

Every step is a libbsq call on the current stream; this module only holds the
preallocated buffers and the launch order.  Data flow (NVFP4 pretraining post:
the data-flow paragraph after Figure 1 and the recipe's ingredients; the
SwiGLU MLP of the Llama models in "Performance results"):

  forward   q(X): rows RNE, columns RNE + RHT (amax pass + encode)
            q(W_gu), q(W_down): 16x16 tiles, under the amax the last update
              of the master weight produced (encode only); a weight orientation
              whose FP16 copy stays cache-resident is expanded once
              (nvfp4_expand) and its GEMMs take it pre-expanded
            Y_gu = X . W_gu^T;  H = SwiGLU(Y_gu), emitting H's amaxes
            q(H): rows RNE, columns RNE + RHT (encode only)
            Y_down = H . W_down^T
  backward  q(dY_down): rows SR, columns SR + RHT (amax pass + encode)
            dH = dY_down . W_down;  dW_down = dY_down^T . H
            dY_gu = SwiGLU backward (Y_gu, dH), emitting dY_gu's amaxes
            q(dY_gu): rows SR, columns SR + RHT (encode only)
            dX = dY_gu . W_gu;  dW_gu = dY_gu^T . X
  update    W <- W - lr * dW on the FP32 masters, writing the BF16 copies
            and their amaxes for the next step

Stochastic rounding uses counter word `offset` = 2 * step (dY_down) and
2 * step + 1 (dY_gu), so successive steps draw fresh bits.

fmt "int8" runs the same products on 8-bit integers: every operand is quantized once
along its rows and once along its columns (int8_quantize_transpose, one scale for each,
round to nearest even, no transform), and int8_gemm takes the side whose rows run along
the product's K.

optimizer "muon" takes, in place of W - lr * dW, the orthogonalised update
(muon_update) of an FP32 momentum kept for each weight: the gate and the up rows of W_gu
as two matrices, W_down as one.
"""

import ctypes

import torch

from . import NEWTON_SCHULZ, _coef_key, _coefs, _on_device, _size, bx_pays, lib as _lib, status_string

NV, RNE, SR = 0, 0, 1


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def muon_options(given):
    """muon_update's options with its defaults for those not given."""
    o = dict(mu=0.95, nesterov=True, weight_decay=0.0, scale=None, steps=5, coefs=NEWTON_SCHULZ, eps=1e-7)
    bad = set(given or {}) - set(o)
    if bad:
        raise ValueError(f"muon takes {', '.join(sorted(o))}, not {', '.join(sorted(bad))}")
    o.update(given or {})
    _coefs(int(o["steps"]), _coef_key(o["coefs"]))
    return o


class MLPLayer:
    """Buffers and launch sequence of one MLP layer (gate/up fused, SwiGLU).

    w_gu: FP32 master [2F, hidden]; w_down: FP32 master [hidden, F] (both
    copied).  tokens % 16 == 0, hidden % 16 == 0, F % 16 == 0.
    fmt: "nvfp4", or "int8" (rht, rht_signs and sr_seed are NVFP4's; tokens, hidden and 2F
    below 2^17).  optimizer: "sgd", or "muon" with muon a dict of muon_update's mu, nesterov,
    weight_decay, scale, steps, coefs, eps (its defaults otherwise) and lr its lr."""

    def __init__(self, w_gu, w_down, tokens, rht=True, rht_signs=0, sr_seed=0, lr=1e-4, fmt="nvfp4",
                 optimizer="sgd", muon=None):
        if not (w_gu.is_cuda and w_down.is_cuda and w_gu.device == w_down.device):
            raise ValueError("the master weights must be CUDA tensors on one device")
        if fmt not in ("nvfp4", "int8"):
            raise ValueError(f"fmt must be 'nvfp4' or 'int8', not {fmt!r}")
        if optimizer not in ("sgd", "muon") or (muon is not None and optimizer != "muon"):
            raise ValueError("optimizer must be 'sgd', or 'muon' (which alone takes muon)")
        dev = w_gu.device
        self.lib = _lib()
        self.dev = dev
        F2, Hd = w_gu.shape
        F = F2 // 2
        assert w_down.shape == (Hd, F) and F2 == 2 * F
        T = tokens
        self.T, self.Hd, self.F = T, Hd, F
        self.rht, self.signs, self.seed, self.lr = (1 if rht else 0), int(rht_signs) & 0xFFFF, int(sr_seed), float(lr)
        self.it = 0
        self.fmt, self.optimizer = fmt, optimizer
        if fmt == "int8" and (max(T, Hd, F2) >= 1 << 17 or T % 16 or Hd % 16 or F % 16):
            raise ValueError("int8 needs tokens, hidden and F multiples of 16; tokens, hidden and 2F below 2^17")
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=dev)
        u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=dev)
        f32 = lambda: torch.empty(1, dtype=torch.float32, device=dev)
        self.w32 = {"W_gu": w_gu.detach().float().contiguous().clone(),
                    "W_down": w_down.detach().float().contiguous().clone()}
        self.wbf = {k: bf(*v.shape) for k, v in self.w32.items()}
        self.wamax = {k: f32() for k in self.w32}
        sizes = (("X", (T, Hd)), ("W_gu", (F2, Hd)), ("H", (T, F)), ("W_down", (Hd, F)),
                 ("dY_down", (T, Hd)), ("dY_gu", (T, F2)))
        self.q = {}
        if fmt == "int8":
            i8 = lambda *s: torch.empty(s, dtype=torch.int8, device=dev)
            scales = lambda n: torch.empty(n, dtype=torch.float32, device=dev)
            for name, (R, C) in sizes:
                self.q[name] = dict(rc=i8(R, C), rs=scales(R), cc=i8(C, R), cs=scales(C))
            self.q_ws = u8(max(_size("int8_quantize_transpose_workspace", R, C) for _, (R, C) in sizes))
        else:
            for name, (R, C) in sizes:
                self.q[name] = dict(rc=u8(R, C // 2), rs=u8(R, C // 16), ra=f32(),
                                    cc=u8(C, R // 2), cs=u8(C, R // 16), ca=f32())
            # a weight's 16x16 quantization runs under the amax its last update
            # produced; both orientations share it, and the GEMMs read it from here
            for k in self.w32:
                self.q[k]["ra"] = self.q[k]["ca"] = self.wamax[k]
        self.act = dict(Y_gu=bf(T, F2), H=bf(T, F), Y_down=bf(T, Hd), dH=bf(T, F),
                        dY_gu=bf(T, F2), dX=bf(T, Hd))
        self.grad = {"W_gu": bf(F2, Hd), "W_down": bf(Hd, F)}
        # B operands taken pre-expanded to FP16 (see bx_pays): (tensor, side) -> buffer
        self.xb = {}
        for name, b, side, N, K in (("FPROP_gu", "W_gu", "r", F2, Hd), ("FPROP_down", "W_down", "r", Hd, F),
                                    ("DGRAD_down", "W_down", "c", F, Hd), ("DGRAD_gu", "W_gu", "c", Hd, F2)):
            if fmt == "nvfp4" and bx_pays(N, K):
                self.xb[(b, side)] = torch.empty((N, K), dtype=torch.float16, device=dev)
        self.flops = 2.0 * 3 * (T * F2 * Hd + T * Hd * F)
        # the BF16 working copies and their amaxes: an update with a zero gradient
        for k in self.w32:
            self.grad[k].zero_()
            self._update(k, 0.0)
        if optimizer == "muon":
            self.muon = muon_options(muon)
            self.momentum = {k: torch.zeros_like(w) for k, w in self.w32.items()}
            self.stack = {"W_gu": (2, F, Hd), "W_down": (1, Hd, F)}
            self.muon_coefs = _coefs(int(self.muon["steps"]), _coef_key(self.muon["coefs"]))
            self.muon_ws = u8(max(_size("orthogonalize_workspace", *s) for s in self.stack.values()))

    # -- single launches -------------------------------------------------------------
    def _stream(self):
        return ctypes.c_void_p(torch.cuda.current_stream(self.dev).cuda_stream)

    def _ok(self, what, st):
        if st != 0:
            raise RuntimeError(f"{what}: {status_string(st)}")

    def _quant(self, name, x, rnd, rht, offset):
        b, (R, C) = self.q[name], x.shape
        self._ok("quantize_transpose " + name, self.lib.quantize_transpose(
            _p(x), R, C, NV, 1, rnd, self.seed, offset, rht, self.signs, _p(b["rc"]), _p(b["rs"]),
            _p(b["ra"]), _p(b["cc"]), _p(b["cs"]), _p(b["ca"]), self._stream()))

    def _quant_amax(self, name, x, block_rows, rnd, rht, offset, amax_row, amax_col):
        b, (R, C) = self.q[name], x.shape
        self._ok("quantize_transpose_amax " + name, self.lib.quantize_transpose_amax(
            _p(x), R, C, block_rows, rnd, self.seed, offset, rht, self.signs, _p(amax_row),
            _p(amax_col), _p(b["rc"]), _p(b["rs"]), _p(b["cc"]), _p(b["cs"]), self._stream()))

    def _expand(self, name):
        for (b, side), out in self.xb.items():
            if b == name:
                q, (R, C) = self.q[b], out.shape
                self._ok("nvfp4_expand " + b, self.lib.nvfp4_expand(
                    _p(q[side + "c"]), _p(q[side + "s"]), R, C, _p(out), self._stream()))

    def _gemm(self, what, a, ao, b, bo, c, M, N, K):
        qa, qb = self.q[a], self.q[b]
        if (b, bo) in self.xb:
            self._ok("bs_gemm_nvfp4_bx " + what, self.lib.bs_gemm_nvfp4_bx(
                M, N, K, _p(qa[ao + "c"]), _p(qa[ao + "s"]), _p(qa[ao + "a"]), _p(self.xb[(b, bo)]),
                _p(qb[bo + "a"]), _p(c), N, self._stream()))
            return
        self._ok("bs_gemm " + what, self.lib.bs_gemm(
            NV, M, N, K, _p(qa[ao + "c"]), _p(qa[ao + "s"]), _p(qa[ao + "a"]), _p(qb[bo + "c"]),
            _p(qb[bo + "s"]), _p(qb[bo + "a"]), _p(c), N, self._stream()))

    @_on_device
    def _update(self, name, lr):
        w = self.w32[name]
        self._ok("master_weight_update " + name, self.lib.master_weight_update(
            _p(w), _p(self.grad[name]), w.numel(), ctypes.c_float(lr), _p(self.wbf[name]),
            _p(self.wamax[name]), self._stream()))

    def _quant8(self, name, x):
        b, (R, C) = self.q[name], x.shape
        self._ok("int8_quantize_transpose " + name, self.lib.int8_quantize_transpose(
            _p(x), R, C, _p(b["rc"]), _p(b["rs"]), _p(b["cc"]), _p(b["cs"]), _p(self.q_ws), self.q_ws.numel(),
            self._stream()))

    def _gemm8(self, what, a, ao, b, bo, c, M, N, K):
        qa, qb = self.q[a], self.q[b]
        self._ok("int8_gemm " + what, self.lib.int8_gemm(
            M, N, K, _p(qa[ao + "c"]), _p(qa[ao + "s"]), _p(qb[bo + "c"]), _p(qb[bo + "s"]), None, _p(c), N,
            self._stream()))

    def _update_muon(self, name):
        o, (B, R, C) = self.muon, self.stack[name]
        scale = 0.2 * max(R, C) ** 0.5 if o["scale"] is None else o["scale"]
        self._ok("muon_update " + name, self.lib.muon_update(
            _p(self.w32[name]), _p(self.momentum[name]), _p(self.grad[name]), B, R, C, self.lr, float(o["mu"]),
            1 if o["nesterov"] else 0, float(o["weight_decay"]), float(scale), int(o["steps"]), self.muon_coefs,
            float(o["eps"]), _p(self.wbf[name]), _p(self.wamax[name]), _p(self.muon_ws), self.muon_ws.numel(),
            self._stream()))

    # -- the step --------------------------------------------------------------------
    @_on_device
    def forward(self, x):
        T, Hd, F = self.T, self.Hd, self.F
        if not (x.shape == (T, Hd) and x.dtype == torch.bfloat16 and x.is_contiguous()
                and x.device == self.dev):
            raise ValueError(f"x must be a contiguous bfloat16 [{T}, {Hd}] tensor on {self.dev}")
        if self.fmt == "int8":
            return self._forward_int8(x)
        self._quant("X", x, RNE, self.rht, 0)
        wa = self.wamax["W_gu"]
        self._quant_amax("W_gu", self.wbf["W_gu"], 16, RNE, 0, 0, wa, wa)
        self._expand("W_gu")
        self._gemm("FPROP_gu", "X", "r", "W_gu", "r", self.act["Y_gu"], T, 2 * F, Hd)
        H, qh = self.act["H"], self.q["H"]
        self._ok("swiglu_amax", self.lib.swiglu_amax(
            _p(self.act["Y_gu"]), T, F, self.rht, self.signs, _p(H), _p(qh["ra"]), _p(qh["ca"]),
            self._stream()))
        self._quant_amax("H", H, 1, RNE, self.rht, 0, qh["ra"], qh["ca"])
        wa = self.wamax["W_down"]
        self._quant_amax("W_down", self.wbf["W_down"], 16, RNE, 0, 0, wa, wa)
        self._expand("W_down")
        self._gemm("FPROP_down", "H", "r", "W_down", "r", self.act["Y_down"], T, Hd, F)
        return self.act["Y_down"]

    @_on_device
    def backward(self, dy_down):
        T, Hd, F = self.T, self.Hd, self.F
        if not (dy_down.shape == (T, Hd) and dy_down.dtype == torch.bfloat16 and dy_down.is_contiguous()
                and dy_down.device == self.dev):
            raise ValueError(f"dy_down must be a contiguous bfloat16 [{T}, {Hd}] tensor on {self.dev}")
        if self.fmt == "int8":
            return self._backward_int8(dy_down)
        off = 2 * self.it
        self._quant("dY_down", dy_down, SR, self.rht, off)
        self._gemm("DGRAD_down", "dY_down", "r", "W_down", "c", self.act["dH"], T, F, Hd)
        self._gemm("WGRAD_down", "dY_down", "c", "H", "c", self.grad["W_down"], Hd, F, T)
        dY, qd = self.act["dY_gu"], self.q["dY_gu"]
        self._ok("swiglu_backward_amax", self.lib.swiglu_backward_amax(
            _p(self.act["Y_gu"]), _p(self.act["dH"]), T, F, self.rht, self.signs, _p(dY),
            _p(qd["ra"]), _p(qd["ca"]), self._stream()))
        self._quant_amax("dY_gu", dY, 1, SR, self.rht, off + 1, qd["ra"], qd["ca"])
        self._gemm("DGRAD_gu", "dY_gu", "r", "W_gu", "c", self.act["dX"], T, Hd, 2 * F)
        self._gemm("WGRAD_gu", "dY_gu", "c", "X", "c", self.grad["W_gu"], 2 * F, Hd, T)
        return self.act["dX"]

    def _forward_int8(self, x):
        T, Hd, F, act = self.T, self.Hd, self.F, self.act
        self._quant8("X", x)
        self._quant8("W_gu", self.wbf["W_gu"])
        self._gemm8("FPROP_gu", "X", "r", "W_gu", "r", act["Y_gu"], T, 2 * F, Hd)
        self._ok("swiglu_amax", self.lib.swiglu_amax(_p(act["Y_gu"]), T, F, 0, 0, _p(act["H"]), None, None,
                                                     self._stream()))
        self._quant8("H", act["H"])
        self._quant8("W_down", self.wbf["W_down"])
        self._gemm8("FPROP_down", "H", "r", "W_down", "r", act["Y_down"], T, Hd, F)
        return act["Y_down"]

    def _backward_int8(self, dy_down):
        T, Hd, F, act = self.T, self.Hd, self.F, self.act
        self._quant8("dY_down", dy_down)
        self._gemm8("DGRAD_down", "dY_down", "r", "W_down", "c", act["dH"], T, F, Hd)
        self._gemm8("WGRAD_down", "dY_down", "c", "H", "c", self.grad["W_down"], Hd, F, T)
        self._ok("swiglu_backward_amax", self.lib.swiglu_backward_amax(
            _p(act["Y_gu"]), _p(act["dH"]), T, F, 0, 0, _p(act["dY_gu"]), None, None, self._stream()))
        self._quant8("dY_gu", act["dY_gu"])
        self._gemm8("DGRAD_gu", "dY_gu", "r", "W_gu", "c", act["dX"], T, Hd, 2 * F)
        self._gemm8("WGRAD_gu", "dY_gu", "c", "X", "c", self.grad["W_gu"], 2 * F, Hd, T)
        return act["dX"]

    @_on_device
    def update(self):
        for k in ("W_gu", "W_down"):
            if self.optimizer == "muon":
                self._update_muon(k)
            else:
                self._update(k, self.lr)
        self.it += 1

    def step(self, x, dy_down):
        """Forward, backward and the master-weight update; returns (Y_down, dX)."""
        y = self.forward(x)
        dx = self.backward(dy_down)
        self.update()
        return y, dx
