"""The gradient of the whole layer, router included, by the README's recipe:
moe_backward, and the three products of dlogits that are the caller's."""
import os
import re

import pytest
import torch

import grouped_expert_gemm_router_b200 as moe
from test_gpu_backward import D, Layer, layer_f64

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _recipe():
    text = open(README).read()
    return re.search(r"```\n(import grouped_expert_gemm_router_b200 as moe\nshape = .*?moe_backward.*?)```", text, re.S).group(1)


@pytest.mark.parametrize("case", [(96, 256, 256, 8, 2, None, "uniform"), (301, 384, 256, 8, 3, None, "skew")])
def test_training_recipe_gives_the_gradient_of_the_layer(case):
    """The example's lines as they stand, against the float64 gradient of the
    whole layer.  The experts' share of dx goes through the 8-bit checkpoint
    (below 0.1 in norm); the router's share and its weights' and bias'
    gradients do not (dlogits below 2e-2 in norm, and the products are linear
    in it: a norm of x^T d is at most the norm of x times that error, so these
    two are compared with the products of the float64 dlogits through that
    bound)."""
    L = Layer("recipe", case=case)
    T, H, F, E, k = L.T, L.H, L.F, L.E, L.k
    wr = torch.randn(H, E, generator=L.gen, device="cuda") / H ** 0.5
    v = dict(T=T, H=H, F=F, E=E, k=k, x=L.x, wr=wr, wg=L.w_gate, wu=L.w_up, wd=L.w_down, dout=L.randn(T, H))
    exec(_recipe(), v)
    torch.cuda.synchronize()
    b = v["b"]
    assert moe.moe_read_status(b["ws"]) == 0
    ps = [t.to(D).requires_grad_() for t in (L.x, wr, L.w_gate, L.w_up, L.w_down)]
    out, logits = layer_f64(*ps, b["topk_idx"].long())
    logits.retain_grad()
    (out * v["dout"].to(D)).sum().backward()
    d, x = logits.grad, ps[0].detach()
    err = (b["dlogits"].to(D) - d).norm()
    assert err <= 2e-2 * d.norm()

    def near(got, ref, tol):
        assert got.shape == ref.shape and (got.to(D) - ref).norm() <= tol, ((got.to(D) - ref).norm(), tol)

    near(v["dw_router"], ps[1].grad, torch.linalg.matrix_norm(x, 2) * err * (1 + 1e-3))
    near(v["dbias"], d.sum(0), T ** 0.5 * err * (1 + 1e-3))
    share = d @ ps[1].detach().T
    near(v["dx"], ps[0].grad, 0.1 * (ps[0].grad - share).norm() + 2e-2 * share.norm()
         + torch.linalg.matrix_norm(ps[1].detach(), 2) * err + 2.0 ** -8 * ps[0].grad.norm())
    # without the router's share it would not be the gradient
    assert (b["dx"].to(D) - ps[0].grad).norm() > 0.2 * ps[0].grad.norm()


def test_forward_activations_kept_for_the_down_weights():
    """moe_grouped_down_wgrad on the forward pass's h in place of the codes':
    within the roundings of h, dy and dw_down itself (each at most 2^-8 in
    norm, and h's silu as much again)."""
    L = Layer("kept", case=(300, 256, 384, 8, 2, None, "uniform"))
    wr = torch.randn(L.H, L.E, generator=L.gen, device="cuda") / L.H ** 0.5
    dout = L.randn(L.T, L.H)
    b = moe.alloc_buffers(L.shape)
    b.update(x=L.x, w_router=wr, bias=None, w_gate=L.w_gate, w_up=L.w_up, w_down=L.w_down,
             **moe.alloc_checkpoint(L.shape))
    moe.moe_forward_checkpoint(L.shape, b, b["ws"])
    dy, dw, kept = torch.empty_like(b["y"]), torch.empty_like(b["topk_w"]), torch.empty_like(L.w_down)
    moe.moe_combine_backward(L.shape, dout, b["y"], b["dest_row"], b["topk_w"], None, dy, dw)
    moe.moe_grouped_down_wgrad(L.shape, b["h"], dy, kept, b["ws"])
    b.update(moe.alloc_backward_buffers(L.shape), dout=dout)
    moe.moe_backward(L.shape, b, b["ws"])
    assert moe.moe_read_status(b["ws"]) == 0
    ps = [t.to(D).requires_grad_() for t in (L.x, wr, L.w_gate, L.w_up, L.w_down)]
    out, _ = layer_f64(*ps, b["topk_idx"].long())
    (out * dout.to(D)).sum().backward()
    ref = ps[4].grad
    assert (kept.to(D) - ref).norm() <= 4 * 2.0 ** -8 * ref.norm()
    assert (b["dw_down"].to(D) - ref).norm() <= 0.1 * ref.norm()


def test_forward_silu_far_below_zero():
    """silu(g) = g/2 + g/2 tanh(g/2) with the hardware's tanh (2^-11 of its
    value): at most |g| 2^-12, an fp32 rounding and the bf16 one.  x picks one
    row of the weights, so g and u are exact."""
    H, F = 128, 4096
    g = torch.linspace(-20, 20, F, device="cuda").bfloat16()
    s = moe.make_shape(1, H, F, 1, 1)
    x, wg, wu = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in ((1, H), (1, H, F), (1, H, F)))
    x[0, 3], wg[0, 3], wu[0, 3] = 1, g, 1
    ws = torch.empty((moe.moe_workspace_bytes(s) + 255) // 256 * 256, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(s, ws)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    moe.moe_dispatch(s, i32((1, 1)), i32(1), i32(2), i32(1), i32(1), ws)
    h, h_ck, ck = torch.empty_like(wg[0, :1]), torch.empty_like(wg[0, :1]), moe.alloc_checkpoint(s)
    moe.moe_grouped_swiglu(s, x, wg, wu, h, ws)
    moe.moe_grouped_swiglu_checkpoint(s, x, wg, wu, h_ck, ck["g_q"], ck["u_q"], ck["scale"], ws)
    assert torch.equal(h, h_ck)
    z = g.to(D)
    ref = z * torch.sigmoid(z)
    e = z.abs() * 2.0 ** -12 + z.abs() * 2.0 ** -24
    assert ((h[0].to(D) - ref).abs() <= e + 2.0 ** -8 * (ref.abs() + e)).all()
