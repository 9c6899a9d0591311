"""Device-resident layer: weights, descriptor and workspace for repeated
moe_forward calls (memory management only; the math is in the kernels)."""
from __future__ import annotations

import threading
from typing import Optional

import torch

from .binding import (MOE_BF16, MOE_F32, MOE_FP8_E4M3, MOE_LAYOUT_FRAG16,
                      MOE_LAYOUT_ROW_MAJOR, _empty, alloc_few_workspace, alloc_workspace,
                      make_desc, moe_add_rms_norm, moe_add_rms_norm_quant_fp8, moe_forward,
                      moe_forward_few, moe_forward_signaled, moe_gemm_fp8, moe_gemm_mxfp4,
                      moe_pack_weights, moe_quant_fp8, moe_quant_mxfp4, moe_route,
                      moe_silu_mul_quant_fp8, moe_silu_mul_quant_mxfp4)

_ACT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_W = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.uint8: MOE_FP8_E4M3}


class DeviceLayer:
    """Holds one layer's router / expert weights on the GPU.

    router [E, H], w13 [E+ns, 2I, H], w2 [E+ns, H, I] (uint8 = fp8 e4m3fn codes
    with fp32 block scales s13 [E+ns, 2I/128, H/128], s2 [E+ns, H/128, I/128]).
    packed=True re-lays the expert weights out once with moe_pack_weights and
    keeps only that copy (bf16 / fp8 weights).  block_m: the descriptor's
    segment padding (0 = library default).
    """

    def __init__(self, router, w13, w2, topk: int, n_shared: int = 0,
                 s13: Optional[torch.Tensor] = None, s2: Optional[torch.Tensor] = None,
                 device="cuda", packed: bool = False, block_m: int = 0):
        self.router = router.to(device).contiguous()
        self.w13 = w13.to(device).contiguous()
        self.w2 = w2.to(device).contiguous()
        self.s13 = None if s13 is None else s13.to(device, torch.float32).contiguous()
        self.s2 = None if s2 is None else s2.to(device, torch.float32).contiguous()
        self.E, self.H = self.router.shape
        self.n_shared = n_shared
        self.I = self.w13.shape[1] // 2
        self.topk = topk
        self.act = _ACT[self.router.dtype]
        self.wd = _W[self.w13.dtype]
        self._check_scales()
        self.device = device
        self.block_m = block_m
        self._ws = {}
        self._few_ws, self._few_lock = {}, threading.Lock()
        self.layout = MOE_LAYOUT_ROW_MAJOR
        if packed:
            self.w13, self.w2 = moe_pack_weights(self.desc(1), self.w13, self.w2)
            self.layout = MOE_LAYOUT_FRAG16

    # Copies and pickles: the workspaces of forward_few belong to this process's
    # streams, and a lock is not copied.
    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k not in ("_few_ws", "_few_lock")}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._few_ws, self._few_lock = {}, threading.Lock()

    def _check_scales(self):
        if self.wd != MOE_FP8_E4M3:
            return
        ne, I, H = self.E + self.n_shared, self.I, self.H
        for s, name, shape, said in (
                (self.s13, "s13", (ne, 2 * I // 128, H // 128), "[E+ns, 2I/128, H/128]"),
                (self.s2, "s2", (ne, H // 128, I // 128), "[E+ns, H/128, I/128]")):
            if s is None or s.shape != shape or s.dtype != torch.float32 or \
                    not s.is_contiguous() or s.device != self.w13.device:
                raise ValueError(f"fp8 weights need {name} {said}, contiguous fp32 on "
                                 f"{self.w13.device}")

    def desc(self, T: int):
        self._check_scales()
        return make_desc(T, self.H, self.E, self.I, self.n_shared, self.act, self.wd,
                         self.s13, self.s2, block_m=self.block_m, w_layout=self.layout)

    def workspace(self, T: int) -> torch.Tensor:
        if T not in self._ws:
            self._ws[T] = alloc_workspace(self.desc(T), self.topk, self.device)
        return self._ws[T]

    def forward(self, x, valid=None, out=None, workspace=None, stream=None):
        """The layer for x [T, H] (forward_few is faster for a few rows).
        Returns out."""
        T = x.shape[0]
        if out is None:
            out = torch.empty_like(x)
        ws = workspace if workspace is not None else self.workspace(T)
        moe_forward(self.desc(T), x, valid, self.router, self.w13, self.w2, self.topk,
                    out, ws, stream)
        return out

    def few_workspace(self, T: int, stream=None) -> torch.Tensor:
        """Workspace of forward_few, one per row count and stream (calls on one
        stream follow each other); a new one while a graph is captured, so that
        graphs do not share it with each other or with eager calls."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.few_workspace(T)
        device = self.router.get_device()
        if device != torch._C._cuda_getDevice():
            # (whether a capture is on is asked of the current device's stream)
            with torch.cuda.device(device):
                return self.few_workspace(T)
        if torch.cuda.is_current_stream_capturing():
            return alloc_few_workspace(self.desc(T), self.topk, self.router.device)
        key = T, torch._C._cuda_getCurrentRawStream(device)
        ws = self._few_ws.get(key)
        if ws is None:
            ws = self._few_ws[key] = alloc_few_workspace(self.desc(T), self.topk,
                                                         self.router.device)
        return ws

    def forward_few(self, x, valid=None, out=None, workspace=None, stream=None):
        """forward for at most FEW_MAX_ROWS token rows (one or a few sequences
        decoding) of a layer with bf16 activations, in two or three launches; other
        roundings than forward's, so not its bits.  Returns out."""
        T = x.size(0)
        if out is None:
            out = _empty((T, self.H), x.dtype, x.device, stream)
        # threads that call on one stream share its workspace: a call's launches
        # stay together
        with self._few_lock:
            ws = workspace if workspace is not None else self.few_workspace(T, stream)
            moe_forward_few(self.desc(T), x, valid, self.router, self.w13, self.w2, self.topk, out,
                            ws, stream)
        return out

    def block_signals(self, T: int) -> torch.Tensor:
        """Completion counters for forward_signaled: int32 [E+ns, ceil(T/64)]."""
        return torch.empty((self.E + self.n_shared, (T + 63) // 64), dtype=torch.int32,
                           device=self.device)

    def forward_signaled(self, x, valid=None, out=None, workspace=None, block_signal=None,
                         stream=None, consumer_stream=None):
        """forward with per-(expert, 64-row block) completion counters and the
        combine waiting on them on consumer_stream.  Returns (out, block_signal)."""
        T = x.shape[0]
        if out is None:
            out = torch.empty_like(x)
        ws = workspace if workspace is not None else self.workspace(T)
        sig = block_signal if block_signal is not None else self.block_signals(T)
        moe_forward_signaled(self.desc(T), x, valid, self.router, self.w13, self.w2, self.topk,
                             out, ws, sig, stream, consumer_stream)
        return out, sig

    def route(self, x, valid=None, logits=False, stream=None):
        T = x.shape[0]
        ids = torch.empty((T, self.topk), dtype=torch.int32, device=x.device)
        w = torch.empty((T, self.topk), dtype=torch.float32, device=x.device)
        lg = torch.empty((T, self.E), dtype=torch.float32, device=x.device) if logits else None
        moe_route(self.desc(T), x, valid, self.router, self.topk, ids, w, lg,
                  self.workspace(T), stream)
        return ids, w, lg


class DenseFP8:
    """The FFN of a dense block in the experts' fp8 format, tokens quantised
    too: out = W2 (SiLU(W_gate x) * (W_up x)) in fp8 products with block scales.

    w13 [2I, H] (gate rows, then up rows) and w2 [H, I]: uint8 e4m3fn codes,
    with fp32 block scales s13 [ceil(2I/128), ceil(H/128)], s2 [ceil(H/128),
    ceil(I/128)].  H and I multiples of 16.  gate_up: the type of the gate/up
    product between the kernels, torch.bfloat16 (its rounding, 2^-8, is little
    beside that of the codes made of it, 2^-4) or torch.float32.
    """

    gate_up = torch.bfloat16   # of layers that were saved without it

    def __init__(self, w13, w2, s13, s2, device="cuda", gate_up=torch.bfloat16):
        if gate_up not in _ACT:
            raise ValueError(f"gate_up {gate_up}: torch.float32 or torch.bfloat16 expected")
        self.gate_up = gate_up
        self.w13 = w13.to(device).contiguous()
        self.w2 = w2.to(device).contiguous()
        self.s13 = s13.to(device, torch.float32).contiguous()
        self.s2 = s2.to(device, torch.float32).contiguous()
        self.I, self.H = self.w13.shape[0] // 2, self.w13.shape[1]
        blocks = lambda n: (n + 127) // 128  # noqa: E731
        if tuple(self.w13.shape) != (2 * self.I, self.H) or tuple(self.w2.shape) != (self.H, self.I):
            raise ValueError("dense weights are w13 [2I, H] and w2 [H, I]")
        if tuple(self.s13.shape) != (blocks(2 * self.I), blocks(self.H)) or \
                tuple(self.s2.shape) != (blocks(self.H), blocks(self.I)):
            raise ValueError("s13 is [ceil(2I/128), ceil(H/128)], s2 [ceil(H/128), ceil(I/128)]")

    def forward(self, x, out=None, stream=None):
        """x [T, H] bf16 or fp32 -> out [T, H], bf16 unless `out` is fp32."""
        xq, xs = moe_quant_fp8(x, stream=stream)
        return self._of_codes(xq, xs, out, stream)

    def forward_normed(self, x, residual, weight, eps=1e-6, out=None, residual_out=None,
                       stream=None):
        """forward of moe_add_rms_norm's rows, whose codes leave the norm at once.
        Returns (out, residual_out); without a residual (None) the latter is None."""
        xq, xs, kept = moe_add_rms_norm_quant_fp8(x, residual, weight, eps,
                                                  residual_out=residual_out, stream=stream)
        return self._of_codes(xq, xs, out, stream), kept

    def _of_codes(self, xq, xs, out, stream):
        gu = moe_gemm_fp8(xq, xs, self.w13, self.s13, out_dtype=self.gate_up, stream=stream)
        hq, hs = moe_silu_mul_quant_fp8(gu, stream=stream)
        return moe_gemm_fp8(hq, hs, self.w2, self.s2, out=out, stream=stream)


class DenseFP4:
    """DenseFP8's block in 4 bits: e2m1 codes, two to a byte, in blocks of 32 under
    a power of two (e8m0), weights and tokens.

    w13 [2I, H/2] (gate rows, then up rows) and w2 [H, I/2]: uint8, the first of
    two codes in the low half; scale codes s13 [2I, H/32], s2 [H, I/32], uint8 or
    float8_e8m0fnu.  H and I multiples of 32.  gate_up: as DenseFP8's; normed: the
    type of forward_normed's rows between the norm and their codes (fp32: one
    rounding less, twice the bytes).
    """

    def __init__(self, w13, w2, s13, s2, device="cuda", gate_up=torch.bfloat16, normed=torch.bfloat16):
        for name, dtype in (("gate_up", gate_up), ("normed", normed)):
            if dtype not in _ACT:
                raise ValueError(f"{name} {dtype}: torch.float32 or torch.bfloat16 expected")
        self.gate_up, self.normed = gate_up, normed
        self.w13 = w13.to(device).contiguous()
        self.w2 = w2.to(device).contiguous()
        for name, t in (("w13", w13), ("w2", w2), ("s13", s13), ("s2", s2)):
            if t.dtype != torch.uint8 and (name[0] == "w" or t.dtype != torch.float8_e8m0fnu):
                raise ValueError(f"{name}: {t.dtype}, expected torch.uint8")
        # (as bytes: torch does not pickle all of its 8-bit types)
        self.s13 = s13.to(device).contiguous().view(torch.uint8)
        self.s2 = s2.to(device).contiguous().view(torch.uint8)
        self.I, self.H = self.w13.shape[0] // 2, 2 * self.w13.shape[1]
        if self.H % 32 or self.I % 32 or tuple(self.w13.shape) != (2 * self.I, self.H // 2) or \
                tuple(self.w2.shape) != (self.H, self.I // 2):
            raise ValueError("dense weights are w13 [2I, H/2] and w2 [H, I/2], H and I multiples of 32")
        if tuple(self.s13.shape) != (2 * self.I, self.H // 32) or \
                tuple(self.s2.shape) != (self.H, self.I // 32):
            raise ValueError("s13 is [2I, H/32], s2 [H, I/32]")

    @classmethod
    def quantised(cls, w13, w2, device="cuda", gate_up=torch.bfloat16, normed=torch.bfloat16):
        """Of weights w13 [2I, H], w2 [H, I] in bf16 or fp32 (moe_quant_mxfp4)."""
        c13, s13 = moe_quant_mxfp4(w13.to(device))
        c2, s2 = moe_quant_mxfp4(w2.to(device))
        return cls(c13, c2, s13, s2, device, gate_up, normed)

    def forward(self, x, out=None, stream=None):
        """x [T, H] bf16 or fp32 -> out [T, H], bf16 unless `out` is fp32."""
        xq, xs = moe_quant_mxfp4(x, stream=stream)
        gu = moe_gemm_mxfp4(xq, xs, self.w13, self.s13, out_dtype=self.gate_up, stream=stream)
        hq, hs = moe_silu_mul_quant_mxfp4(gu, stream=stream)
        return moe_gemm_mxfp4(hq, hs, self.w2, self.s2, out=out, stream=stream)

    def forward_normed(self, x, residual, weight, eps=1e-6, out=None, residual_out=None,
                       stream=None):
        """forward of moe_add_rms_norm's rows (in the type `normed`).  Returns (out,
        residual_out); without a residual (None) the latter is None."""
        rows, kept = moe_add_rms_norm(x, residual, weight, eps, residual_out=residual_out,
                                      out_dtype=self.normed, stream=stream)
        return self.forward(rows, out, stream), kept
