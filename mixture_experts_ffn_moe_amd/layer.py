"""Tensor-level convenience over the C ABI: allocate a layer call's output and
workspace with torch and expose the workspace's intermediates as views."""
from __future__ import annotations

import torch

from ._lib import (MOE_BF16, moe_forward, moe_forward_q4, moe_forward_shared,
                   moe_get_shared_workspace_layout, moe_get_workspace_layout, moe_lora_workspace_size,
                   moe_shared_backward_workspace_size, moe_shared_ffn_backward, moe_shared_ffn_lora,
                   moe_shared_ffn_train, moe_shared_workspace_size, moe_workspace_size, y_nbytes)


def _dtype(shape) -> torch.dtype:
    return torch.bfloat16 if shape.dtype == MOE_BF16 else torch.float32


def workspace_views(shape, ws: torch.Tensor) -> dict:
    """Views of the intermediates moe_forward (or moe_forward_q4) leaves in workspace `ws` (uint8).  The small-token
    path writes no y: its view then holds what was there before."""
    L = moe_get_workspace_layout(shape)
    T, E, k, H = shape.T, shape.E, shape.k, shape.H
    R = T * k
    I = shape.micro_count * shape.Im
    dt = _dtype(shape)
    es = 2 if dt == torch.bfloat16 else 4

    def view(name, n, elem, dtype, dims):
        off = L[name]
        return ws[off:off + n * elem].view(dtype).view(*dims)

    return {
        "logits": view("logits", T * E, 4, torch.float32, (T, E)),
        "ids": view("topk_ids", R, 4, torch.int32, (T, k)),
        "w": view("topk_w", R, 4, torch.float32, (T, k)),
        "counts": view("counts", E, 4, torch.int32, (E,)),
        "offsets": view("offsets", E + 1, 4, torch.int32, (E + 1,)),
        "perm": view("perm", R, 4, torch.int32, (R,)),
        "inv": view("inv", R, 4, torch.int32, (R,)),
        "h": view("h", R * I, es, dt, (R, I)),
        # raw bytes: block-scaled half in the bf16 layers, fp32 in the fp32 layer
        "y": ws[L["y"]:L["y"] + y_nbytes(shape, R)],
    }


class MoELayerBuffers:
    """Output and workspace of one layer shape, allocated once with torch.
    With shared_Im the workspace also holds the shared expert's regions and
    forward_shared runs the layer with its shared expert; with lora (make_lora)
    as well, forward_shared_lora runs it with every token's own adapter."""

    def __init__(self, shape, device="cuda", shared_Im=None, lora=None):
        self.shape = shape
        self.shared_Im = shared_Im
        self.lora = lora
        if lora is not None:
            if shared_Im is None:
                raise ValueError("adapters are the shared expert's: shared_Im is required")
            n = moe_lora_workspace_size(shape, shared_Im, lora)
            if n == 0:
                raise ValueError("adapters outside the library's envelope")
            self.lora_workspace = torch.empty(n, dtype=torch.uint8, device=device)
        n = moe_workspace_size(shape) if shared_Im is None else moe_shared_workspace_size(shape, shared_Im)
        if n == 0:
            raise ValueError("shape (or shared_Im) outside the library's envelope")
        self.workspace = torch.empty(n, dtype=torch.uint8, device=device)
        self.out = torch.empty(shape.T, shape.H, dtype=_dtype(shape), device=device)

    def forward(self, x, wg, bias, w1, w2, stream=None) -> torch.Tensor:
        moe_forward(self.shape, x, wg, bias, w1, w2, self.out, self.workspace, stream)
        return self.out

    def forward_q4(self, q4, x, wg, bias, w1_codes, w1_scales, w2_codes, w2_scales, stream=None) -> torch.Tensor:
        """The layer over 4-bit expert weights (make_q4, moe_q4_quantize_w13, moe_q4_quantize_down)."""
        moe_forward_q4(self.shape, q4, x, wg, bias, w1_codes, w1_scales, w2_codes, w2_scales, self.out,
                       self.workspace, stream)
        return self.out

    def forward_shared(self, x, wg, bias, w1, w2, w1s, w2s, stream=None) -> torch.Tensor:
        if self.shared_Im is None:
            raise ValueError("buffers were allocated without shared_Im")
        moe_forward_shared(self.shape, self.shared_Im, x, wg, bias, w1, w2, w1s, w2s, self.out,
                           self.workspace, stream)
        return self.out

    def forward_shared_lora(self, x, wg, bias, w1, w2, w1s, w2s, a1, b1, a2, b2, scale, adapter_ids,
                            stream=None) -> torch.Tensor:
        """The layer with its shared expert and the tokens' adapters on it: the routed output is rounded to the
        layer's type, the shared expert's added to it."""
        if self.lora is None:
            raise ValueError("buffers were allocated without lora")
        moe_forward(self.shape, x, wg, bias, w1, w2, self.out, self.workspace, stream)
        moe_shared_ffn_lora(self.shape, self.shared_Im, self.lora, x, w1s, w2s, a1, b1, a2, b2, scale, adapter_ids,
                            self.out, self._hs(), self.out, self.lora_workspace, stream)
        return self.out

    def _hs(self) -> torch.Tensor:
        at = moe_get_shared_workspace_layout(self.shape, self.shared_Im)["hs"]
        n = self.shape.T * self.shared_Im * self.out.element_size()
        return self.workspace[at:at + n].view(self.out.dtype).view(self.shape.T, self.shared_Im)

    def views(self) -> dict:
        v = workspace_views(self.shape, self.workspace)
        if self.shared_Im is not None:
            Ls = moe_get_shared_workspace_layout(self.shape, self.shared_Im)
            dt = _dtype(self.shape)
            es = 2 if dt == torch.bfloat16 else 4
            T, H, Is = self.shape.T, self.shape.H, self.shared_Im
            v["hs"] = self.workspace[Ls["hs"]:Ls["hs"] + T * Is * es].view(dt).view(T, Is)
            v["ys"] = self.workspace[Ls["ys"]:Ls["ys"] + y_nbytes(self.shape, T)]
        return v


class SharedTrainBuffers:
    """What a training step of the shared expert keeps: output, the values its backward pass reads, workspace and
    gradients.  p is the dropout of the hidden values; rng (int64 [2] on the GPU: seed, offset) has to hold the same
    values in forward and backward, and others in the next step."""

    def __init__(self, shape, Is, p=0.0, device="cuda"):
        n = moe_shared_backward_workspace_size(shape, Is)
        if n == 0:
            raise ValueError("shape or Is outside the library's envelope")
        self.shape, self.Is, self.p = shape, Is, p
        T, H, dt = shape.T, shape.H, _dtype(shape)
        e = lambda *dims, dtype=dt: torch.empty(*dims, dtype=dtype, device=device)  # noqa: E731
        self.gu, self.hs, self.out = e(T, 2 * Is, dtype=torch.float32), e(T, Is), e(T, H)
        self.d_x, self.d_w1s, self.d_w2s = e(T, H), e(2 * Is, H), e(H, Is)
        self.workspace = e(n, dtype=torch.uint8)

    def forward(self, x, w1s, w2s, residual=None, rng=None, stream=None) -> torch.Tensor:
        moe_shared_ffn_train(self.shape, self.Is, self.p, rng, x, w1s, w2s, residual, self.gu, self.hs, self.out, stream)
        return self.out

    def backward(self, x, w1s, w2s, d_out, rng=None, stream=None):
        """(d_x, d_w1s, d_w2s); the residual's gradient is d_out."""
        moe_shared_ffn_backward(self.shape, self.Is, self.p, rng, x, w1s, w2s, self.gu, self.hs, d_out, self.d_x,
                                self.d_w1s, self.d_w2s, self.workspace, stream)
        return self.d_x, self.d_w1s, self.d_w2s
