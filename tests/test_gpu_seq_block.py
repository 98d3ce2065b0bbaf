"""The sequence operators together, as examples/recurrent_block.py uses them: a
prompt followed by single tokens against the whole sequence, the block against
its formulas in 64 bits, and a training step against differentiation."""
import os
import sys

import pytest
import torch

from gpu_util import require_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_prompt_then_tokens():
    """A bf16 rounding (2^-9 of a value) may fall differently where fp32 sums run in
    another order, and an 8-bit one (2^-8 of a row's largest) after it: each is
    rare, so the outputs differ by far less than one such step, 2^-7, in the norm."""
    import recurrent_block as rb

    whole, parts, s0, s1 = rb.prompt_then_tokens()
    assert rel(parts, whole) < 2.0 ** -7
    assert rel(s1[1], s0[1]) < 2.0 ** -7 and rel(s1[0], s0[0]) < 2.0 ** -7


def plain_part(x, r, i, w, b, lam, decay):
    """The recurrent part in differentiable 64-bit torch."""
    K, T = w.shape[1], x.shape[1]
    ext = torch.nn.functional.pad(x, (0, 0, K - 1, 0))
    u = torch.nn.functional.silu(b + sum(ext[:, j:j + T] * w[:, j] for j in range(K)))
    la = -decay * torch.nn.functional.softplus(lam) * torch.sigmoid(r)
    put = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i) * u
    h, hs = torch.zeros_like(put[:, 0]), []
    for t in range(T):
        h = torch.exp(la[:, t]) * h + put[:, t]
        hs.append(h)
    return torch.stack(hs, 1)


def test_training_step():
    """Gradients of the whole part: each passes at most four bf16 roundings (u, its
    gradient, y's error and the result), 2^-9 each, so 2^-7 in the norm."""
    import recurrent_block as rb

    loss, leaves, goal, decay = rb.training_step()
    ref = [t.detach().double().requires_grad_(True) for t in leaves]
    want = (plain_part(*ref, decay) - goal.double()).square().sum()
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) <= 2.0 ** -7 * want
    for got, exact in zip(leaves, ref):
        assert rel(got.grad, exact.grad) < 2.0 ** -7


def test_block_against_its_formulas():
    """The block in 64 bits with 8-bit weights and rows at the same places.  A
    quantised row is off by at most half a step, 2^-8 of its largest value (under
    4 norms a row of this width: 2^-6 of the norm at most, 2^-8 typical); two such
    rows and bf16's roundings: 2^-5 in the norm."""
    import recurrent_block as rb

    block = rb.RecurrentBlock(256, 384)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, res = (torch.randn(2, 33, 256, generator=g, device="cuda").to(rb.DT) for _ in range(2))
    out, new = block(x, res, block.empty_state(2))
    h = (x.float() + res.float()).to(rb.DT)
    assert torch.equal(new, h)
    d = h.double()
    v = d / (d.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    w_in = block.w_in[0].double() * block.w_in[1].double()[:, None]
    w_out = block.w_out[0].double() * block.w_out[1].double()[:, None]
    a, r, i = (v @ w_in.t()).split(384, -1)
    y = plain_part(a, r, i, block.conv_w.double(), block.conv_b.double(), block.lam.double(), block.decay)
    assert rel(out, y @ w_out.t()) < 2.0 ** -5


def test_training_on_column_slices():
    """The recurrent part takes x, r and i as the product leaves them, column slices
    of one wide tensor, and any other strides: the same results as from copies."""
    import recurrent_block as rb

    g = torch.Generator(device="cuda").manual_seed(4)
    B, T, D = 2, 50, 128
    block = rb.RecurrentBlock(64, D)
    wide = torch.randn(B, T, 3 * D, generator=g, device="cuda").to(rb.DT)
    goal = torch.randn(B, T, D, generator=g, device="cuda").to(rb.DT)
    time_major = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in wide.split(D, -1)]

    def step(x, r, i, w):
        leaves = [t.detach().requires_grad_(True) for t in (x, r, i, w, block.conv_b, block.lam)]
        y = rb.RecurrentPart.apply(*leaves, block.decay)
        (y.float() - goal.float()).square().sum().backward()
        return [y.detach()] + [t.grad for t in leaves]

    want = step(*(t.contiguous() for t in wide.split(D, -1)), block.conv_w)
    for parts in (wide.split(D, -1), time_major):
        for w in (block.conv_w, block.conv_w.t().contiguous().t()):
            for a, b in zip(step(*parts, w), want):
                assert torch.equal(a, b)


def test_block_takes_inputs_of_any_strides():
    import recurrent_block as rb

    block = rb.RecurrentBlock(256, 384)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, res = (torch.randn(2, 9, 512, generator=g, device="cuda").to(rb.DT)[..., 100:356] for _ in range(2))
    out, new = block(x, res, block.empty_state(2))
    want, want_new = block(x.contiguous(), res.contiguous(), block.empty_state(2))
    assert torch.equal(out, want) and torch.equal(new, want_new)
