"""A recurrent language-model block on the sequence operators: a prompt, then one
token at a time, and a training step of its recurrent part.

    residual + RMS norm -> 8 bits -> 8-bit product to (x, r, i)
    x -> causal depthwise convolution, SiLU -> gated linear recurrence with r, i
    -> 8 bits -> 8-bit product back to the residual's width

Run on a GPU:  python examples/recurrent_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import depthwise_convolution_forward_gb300 as gc  # noqa: E402

DT, CODE = torch.bfloat16, gc.DTYPE_CODES["bf16"]


class RecurrentBlock:
    """Weights, and the state that a sequence carries: K - 1 rows for the
    convolution in the data type, one fp32 row for the recurrence."""

    def __init__(self, width: int, inner: int, taps: int = 4, decay: float = 8.0, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.width, self.inner, self.taps, self.decay, self.device = width, inner, taps, decay, device

        def normal(*shape, std):
            return (torch.randn(shape, generator=g, device=device) * std).to(DT)

        self.norm = torch.ones(width, dtype=DT, device=device)
        self.conv_w, self.conv_b = normal(inner, taps, std=taps ** -0.5), normal(inner, std=0.1)
        slowest = torch.rand(inner, generator=g, device=device) * 0.099 + 0.9
        self.lam = torch.log(torch.expm1(-torch.log(slowest) / decay))
        self.w_in = self._to_8_bits(normal(3 * inner, width, std=width ** -0.5))
        self.w_out = self._to_8_bits(normal(width, inner, std=inner ** -0.5))

    def _to_8_bits(self, w):
        q, s = torch.empty(w.shape, dtype=torch.int8, device=self.device), torch.empty(w.shape[0], device=self.device)
        gc.gconv_quantize_rows_q8(w, q, s, gc.make_norm_problem(*w.shape), CODE, torch.cuda.current_stream())
        return q, s

    def empty_state(self, batch: int):
        return (torch.zeros(batch, self.taps - 1, self.inner, dtype=DT, device=self.device),
                torch.zeros(batch, self.inner, device=self.device))

    def __call__(self, x, residual, state, lens=None):
        """x, residual [B, T, width] -> (output, new residual), both [B, T, width];
        `state` moves on in place.  lens: tokens in each row of a padded batch."""
        B, T, W = x.shape
        x, residual = x.contiguous(), residual.contiguous()  # the records below say that they are packed
        D, rows, st = self.inner, B * T, torch.cuda.current_stream()
        conv_state, h = state
        new = lambda *s, dtype=DT: torch.empty(s, dtype=dtype, device=self.device)  # noqa: E731

        res, q, s = new(B, T, W), new(rows, W, dtype=torch.int8), new(rows, dtype=torch.float32)
        gc.gconv_rms_norm_q8(x, residual, self.norm, res, None, q, s, gc.make_norm_problem(rows, W), CODE, st)
        wide = new(B, T, 3 * D)
        gc.gconv_matmul_q8(q, s, *self.w_in, None, wide, gc.make_matmul_q8_problem(rows, 3 * D, W), CODE, st)
        cols = (T * 3 * D, 3 * D)  # x, r and i are column slices of the product
        conv = new(B, T, D)
        gc.gconv_causal_conv1d_fwd(wide, self.conv_w, self.conv_b, conv_state, lens, conv, conv_state,
                                   gc.make_conv1d_problem(B, T, D, self.taps, gc.ACT_SILU, x_stride=cols), CODE, st)
        y = new(B, T, D)
        gc.gconv_gated_scan_fwd(conv, wide[..., D:2 * D], wide[..., 2 * D:], self.lam, h, lens, y, h, None,
                                gc.make_scan_problem(B, T, D, self.decay, r_stride=cols, i_stride=cols), CODE, st)
        yq, ys = new(rows, D, dtype=torch.int8), new(rows, dtype=torch.float32)
        gc.gconv_quantize_rows_q8(y, yq, ys, gc.make_norm_problem(rows, D), CODE, st)
        out = new(B, T, W)
        gc.gconv_matmul_q8(yq, ys, *self.w_out, None, out, gc.make_matmul_q8_problem(rows, W, D), CODE, st)
        return out, res


class RecurrentPart(torch.autograd.Function):
    """The convolution and the recurrence with their gradients, for training.  x, r and
    i may have any strides, as column slices of one product have."""

    @staticmethod
    def forward(ctx, x, r, i, w, b, lam, decay):
        B, T, D = x.shape
        x, r, i, w, b, lam = (t.contiguous() for t in (x, r, i, w, b, lam))  # the records say that they are packed
        st = torch.cuda.current_stream()
        cp = gc.make_conv1d_problem(B, T, D, w.shape[1], gc.ACT_SILU)
        sp = gc.make_scan_problem(B, T, D, decay)
        u, y = torch.empty_like(x), torch.empty_like(x)
        saved = torch.empty(gc.gconv_gated_scan_saved_size(sp, CODE), dtype=torch.uint8, device=x.device)
        gc.gconv_causal_conv1d_fwd(x, w, b, None, None, u, None, cp, CODE, st)
        gc.gconv_gated_scan_fwd(u, r, i, lam, None, None, y, None, saved, sp, CODE, st)
        ctx.save_for_backward(x, r, i, w, b, lam, u, saved)
        ctx.problems = cp, sp
        return y

    @staticmethod
    def backward(ctx, dy):
        x, r, i, w, b, lam, u, saved = ctx.saved_tensors
        cp, sp = ctx.problems
        st = torch.cuda.current_stream()
        du, dr, di, dlam = torch.empty_like(u), torch.empty_like(r), torch.empty_like(i), torch.empty_like(lam)
        ws = torch.empty(max(gc.gconv_gated_scan_bwd_workspace_size(sp, CODE),
                             gc.gconv_causal_conv1d_bwd_workspace_size(cp, CODE)), dtype=torch.uint8, device=x.device)
        gc.gconv_gated_scan_bwd(dy.contiguous(), None, u, r, i, lam, None, saved, du, dr, di, dlam, None, sp, CODE, ws, 0, st)
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        gc.gconv_causal_conv1d_bwd(du, None, x, w, b, None, None, dx, dw, db, None, cp, CODE, ws, 0, st)
        return dx, dr, di, dw, db, dlam, None


def prompt_then_tokens(batch=3, prompt=40, tokens=8, width=256, inner=384):
    """(outputs of the whole sequence at once, outputs of the prompt and then one
    token at a time, the two final states)."""
    block = RecurrentBlock(width, inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    T = prompt + tokens
    x = torch.randn(batch, T, width, generator=g, device="cuda").to(DT)
    res = torch.randn(batch, T, width, generator=g, device="cuda").to(DT)
    whole_state, state = block.empty_state(batch), block.empty_state(batch)
    whole, _ = block(x, res, whole_state)
    parts = [block(x[:, :prompt].contiguous(), res[:, :prompt].contiguous(), state)[0]]
    for t in range(prompt, T):
        parts.append(block(x[:, t:t + 1].contiguous(), res[:, t:t + 1].contiguous(), state)[0])
    return whole, torch.cat(parts, 1), whole_state, state


def training_step(batch=2, length=96, inner=128):
    """Loss and gradients of the recurrent part for a squared error."""
    g = torch.Generator(device="cuda").manual_seed(2)
    block = RecurrentBlock(64, inner)
    leaf = lambda t: t.detach().clone().requires_grad_(True)  # noqa: E731
    x, r, i, goal = (torch.randn(batch, length, inner, generator=g, device="cuda").to(DT) for _ in range(4))
    leaves = [leaf(t) for t in (x, r, i, block.conv_w, block.conv_b, block.lam)]
    loss = (RecurrentPart.apply(*leaves, block.decay).float() - goal.float()).square().sum()
    loss.backward()
    return loss.detach(), leaves, goal, block.decay


if __name__ == "__main__":
    whole, parts, s0, s1 = prompt_then_tokens()
    print("prompt and tokens against the whole sequence: largest difference %.3g of %.3g" %
          ((whole - parts).abs().max(), whole.abs().max()))
    loss, leaves, _, _ = training_step()
    print("training step: loss %.4g, gradient norms %s" %
          (loss, ", ".join("%.4g" % t.grad.float().norm() for t in leaves)))
