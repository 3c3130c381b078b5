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
