"""Buffer management around the C ABI for one problem shape.

`LayerRunner` allocates (through PyTorch) the plan arrays, workspaces, the
saved context and the outputs for a fixed shape once, then runs
moe_plan / moe_ffn_fwd / moe_ffn_bwd on them.  All arithmetic happens in the
library's kernels.

What only some calls need is made at the first of them, with that call's stream
current: a zero-fill comes before the kernels that use the buffer, and the allocator
gives no memory that another stream still has work for.
"""

import torch

from . import (MOE_BF16, MOE_FP32, Shape, alloc_plan, bias_struct, check_device_error, ffn_bwd,
               ffn_few, ffn_fwd, few_workspace, grad_clip, grad_clip_workspace, grad_table,
               moe_grad_clip_workspace_size, moe_saved_size, mx_alloc, mx_quantize, mx_struct,
               plan, route, workspace)

_TORCH_DTYPE = {MOE_BF16: torch.bfloat16, MOE_FP32: torch.float32}


class LayerRunner:
    def __init__(self, T, H, I, E, k, act, dtype=MOE_BF16, clamp_limit=7.0, alpha=1.702,
                 device="cuda", training=True, backward=True, gate_up_layout=0, out_fp32=False):
        """out_fp32: y and dx in fp32 instead of the storage dtype."""
        self.shape = Shape(T, H, I, E, k, act, dtype, clamp_limit, alpha, gate_up_layout, out_fp32)
        self.device = device
        self.tdtype = _TORCH_DTYPE[dtype]
        odt = torch.float32 if out_fp32 else self.tdtype
        self.plan_t, self.plan_s = alloc_plan(self.shape, device)
        self.ws_plan = workspace(self.shape, 0, device)
        self.ws_fwd = workspace(self.shape, 1, device)
        self.ws_bwd = workspace(self.shape, 2, device) if backward else None
        self.saved = (torch.empty(moe_saved_size(self.shape), dtype=torch.uint8, device=device)
                      if training else None)
        self.y = torch.empty((T, H), dtype=odt, device=device)
        self.gave_bias = False
        self.ws_clip, self.ws_clips = None, []
        if backward:
            self.dx = torch.empty((T, H), dtype=odt, device=device)
            self.d_topk_w = torch.empty((T, k), dtype=torch.float32, device=device)
            self.dw_gate_up = torch.empty((E, H, 2 * I), dtype=torch.float32, device=device)
            self.dw_down = torch.empty((E, I, H), dtype=torch.float32, device=device)

    def plan(self, topk_idx, stream=None):
        plan(self.shape, topk_idx, self.plan_s, self.ws_plan, stream)

    def route(self, logits, topk_idx, topk_w, stream=None):
        """Fill topk_idx [T,k] int32 and topk_w [T,k] fp32 from fp32 logits
        [T,E] and build the plan of the chosen ids."""
        route(self.shape, logits, topk_idx, topk_w, self.plan_s, self.ws_plan, stream)

    def forward(self, x, topk_idx, topk_w, w_gate_up, w_down, use_plan=True, stream=None,
                b_gate_up=None, b_down=None, inference=False):
        """y = layer(x).  With use_plan the plan must have been built by plan();
        otherwise the forward builds its own inside the workspace.  b_gate_up
        [E,2I] / b_down [E,H] (storage dtype) are the optional per-expert biases.
        inference=True saves no context for the backward (as a runner built
        with training=False)."""
        ffn_fwd(self.shape, x, topk_idx, topk_w, w_gate_up, w_down, self.y, self.ws_fwd,
                self.plan_s if use_plan else None, None if inference else self.saved, stream,
                bias_struct(b_gate_up, b_down))
        return self.y

    def quantize(self, w_gate_up, w_down, stream=None):
        """Keep both weights in microscaled 4-bit for few(): (codes, scales) of
        w_gate_up and of w_down.  Call it again when the weights change: the same
        tensors then hold the new ones, for captured graphs too."""
        if getattr(self, "mx_t", None) is None:
            E, H, I = self.shape.E, self.shape.H, self.shape.I
            with torch.cuda.stream(stream):
                self.mx_t = mx_alloc(E, H, 2 * I, self.device) + mx_alloc(E, I, H, self.device)
        mx_quantize(w_gate_up, *self.mx_t[:2], stream=stream)
        mx_quantize(w_down, *self.mx_t[2:], stream=stream)
        self.mx_s = mx_struct(*self.mx_t)
        return self.mx_t

    def few(self, x, topk_idx, topk_w, w_gate_up=None, w_down=None, x_scale=None, stream=None,
            b_gate_up=None, b_down=None):
        """y = layer(x) for at most 128 tokens, without a plan or a saved context.
        Without weights, on the 4-bit ones that quantize() keeps.  x may be e4m3
        codes with x_scale, as rms_norm_fwd gives them."""
        if getattr(self, "ws_few", None) is None:
            with torch.cuda.stream(stream):
                self.ws_few = few_workspace(self.shape, self.device)
        mx = None
        if w_gate_up is None and w_down is None:
            mx = getattr(self, "mx_s", None)
            if mx is None:
                raise ValueError("few: no weights given, and quantize() has not been called")
        ffn_few(self.shape, x, topk_idx, topk_w, w_gate_up, w_down, self.y, self.ws_few, stream,
                bias_struct(b_gate_up, b_down), x_scale, mx)
        return self.y

    def backward(self, dy, x, topk_idx, topk_w, w_gate_up, w_down, stream=None, recompute=False,
                 b_gate_up=None, b_down=None):
        """Gradients of <dy, y>: (dx, d_topk_w, dw_gate_up, dw_down), and with
        biases also (db_gate_up, db_down).  The biases must be those given to
        the forward.  With recompute the saved context is not used: the
        backward recomputes it in a larger workspace (allocated on first use)."""
        with_bias = b_gate_up is not None or b_down is not None
        self.gave_bias = with_bias      # what clip_grads takes
        bias = None
        if with_bias:
            if getattr(self, "db_gate_up", None) is None:
                E, H, I = self.shape.E, self.shape.H, self.shape.I
                with torch.cuda.stream(stream):
                    self.db_gate_up = torch.empty((E, 2 * I), dtype=torch.float32, device=self.device)
                    self.db_down = torch.empty((E, H), dtype=torch.float32, device=self.device)
            bias = bias_struct(b_gate_up, b_down, self.db_gate_up, self.db_down)
        if recompute:
            if getattr(self, "ws_bwd_recompute", None) is None:
                with torch.cuda.stream(stream):
                    self.ws_bwd_recompute = workspace(self.shape, 3, self.device)
            ws, saved = self.ws_bwd_recompute, None
        else:
            ws, saved = self.ws_bwd, self.saved
        ffn_bwd(self.shape, dy, x, topk_idx, topk_w, w_gate_up, w_down, self.plan_s, saved,
                self.dx, self.d_topk_w, self.dw_gate_up, self.dw_down, ws, stream, bias)
        out = (self.dx, self.d_topk_w, self.dw_gate_up, self.dw_down)
        return out + (self.db_gate_up, self.db_down) if with_bias else out

    def clip_grads(self, max_norm, extra=(), stream=None):
        """Scale the last backward's weight gradients (and bias gradients, where it
        gave them), with those of `extra` (tensors), so that their global norm is at
        most max_norm, in place.  Returns (norm before, factor) as a tensor [2]."""
        grads = [self.dw_gate_up, self.dw_down]
        if self.gave_bias:
            grads += [self.db_gate_up, self.db_down]
        table = grad_table(grads + list(extra))
        if self.ws_clip is None or self.ws_clip.numel() < moe_grad_clip_workspace_size(table, table.count):
            with torch.cuda.stream(stream):
                if self.ws_clip is None:
                    self.clip_norm = torch.empty(2, dtype=torch.float32, device=self.device)
                self.ws_clip = grad_clip_workspace(table, self.device)
            # those of shorter lists stay for the graphs that may have been captured with them
            self.ws_clips.append(self.ws_clip)
        grad_clip(table, max_norm, self.clip_norm, self.ws_clip, stream)
        return self.clip_norm

    def check(self, stream=None):
        for ws in (self.ws_plan, self.ws_fwd, self.ws_bwd, getattr(self, "ws_bwd_recompute", None),
                   getattr(self, "ws_few", None)):
            if ws is not None:
                check_device_error(ws, stream)
