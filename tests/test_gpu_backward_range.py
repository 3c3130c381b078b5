"""The down gradient far from zero: gate and up values over the whole range of
the checkpoint's scales, against the formula in float64.

The sigmoid is computed as 1 / (1 + e^-g) in fp32.  Below, with the fast
exponential's bound (2 + 1.16 |g| ulp) and the fast division's (2 ulp):
  - g >= 18: e^-g < 2^-25, so the sum is 1 and its reciprocal too: silu(g) = g
    and the derivative is 1, where the formula differs by less than g e^-g
    < 2^-21;
  - -87 <= g < 18: the sigmoid is off by (16 + 2 |g|) 2^-23 of itself at most,
    the derivative by that of its terms s (1 + |g|);
  - g < -87: e^-g is above 2^125, and the division may return 0 from 2^126 on:
    the sigmoid is off by 2^-125 at most.
A product may fall below the normal numbers: 2^-149 of each factor's step, and
the bf16 result half a step of 2^-133."""
import pytest
import torch

import grouped_expert_gemm_router_b200 as moe
from test_gpu_backward import D, HALF, Layer, acc

pytestmark = pytest.mark.gpu
BF16_MAX = float(torch.finfo(torch.bfloat16).max)

RANGES = {
    # scale bytes of g, of u (a byte b stands for 2^(b - 127), codes reach 448)
    "moderate": ((118, 119, 120, 121, 122), (110, 119, 127)),
    "far": ((121, 122, 123, 124, 126, 128, 140), (100, 119, 127)),
    "least": ((1, 2, 20, 60), (1, 2, 60, 119)),
    "huge_gate": ((160, 200, 240, 246), (1, 60, 100, 119)),
    # dh u alone would overflow; with the sigmoid's derivative it is finite, or zero
    "huge_up": ((120, 121, 122, 123, 124, 130), (230, 244, 246)),
}


@pytest.mark.parametrize("name", list(RANGES))
@pytest.mark.parametrize("H", [128, 3584])  # 128- and 256-feature units
def test_down_backward_far_from_zero(name, H):
    L = Layer(name, seed=3, case=(300, H, 512, 3, 2, None, "uniform"))
    dy = L.rows(L.P, L.H)
    ck = {}
    for n in ("g_q", "u_q"):
        mag = torch.randint(0, 127, (L.P, L.F), generator=L.gen, device="cuda", dtype=torch.uint8)  # every finite code
        sign = torch.randint(0, 2, (L.P, L.F), generator=L.gen, device="cuda", dtype=torch.uint8)
        ck[n] = mag | sign << 7
    pick = [torch.tensor(b, dtype=torch.uint8, device="cuda")[
        torch.randint(0, len(b), (L.P, L.F // 32), generator=L.gen, device="cuda")] for b in RANGES[name]]
    scale = torch.stack(pick, -1).contiguous()
    dg, du, h = (L.poison(L.P, L.F) for _ in range(3))
    moe.moe_grouped_down_backward(L.shape, dy, L.w_down, ck["g_q"], ck["u_q"], scale, dg, du, h, L.ws)
    assert L.status() == 0
    g_all, u_all = (moe.checkpoint_values(ck[n], scale, i).to(D) for i, n in enumerate(("g_q", "u_q")))
    assert torch.isfinite(g_all).all() and torch.isfinite(u_all).all()

    def check(got, ref, tol, what):
        tol = tol + HALF * ref.abs() + 2.0 ** -134
        got = got.to(D)
        fits = ref.abs() + tol < BF16_MAX  # beyond: the bf16 result may be an infinity of the same sign
        assert torch.isfinite(got[fits]).all(), "%s: %d values not finite" % (what, (~torch.isfinite(got[fits])).sum())
        worst = ((got - ref).abs() / tol)[fits].max()
        assert worst <= 1, "%s: %g of the tolerance" % (what, worst)
        assert not torch.isnan(got).any() and (got[~fits].sign() == ref[~fits].sign()).all(), what

    for e, i in enumerate(L.row_of):
        a, w = dy[i].to(D), L.w_down[e].to(D)
        dh, e_dh = a @ w.T, acc(H) * (a.abs() @ w.T.abs())
        g, u = g_all[i], u_all[i]
        s = torch.sigmoid(g)
        f = s * (1 + g * (1 - s))
        rel = (16 + 2 * g.abs().clamp(max=87)) * 2.0 ** -23
        high, low = g >= 18, g < -87
        e_s = torch.where(high, 2.0 ** -24 * s, rel * s + low * 2.0 ** -125)
        e_f = torch.where(high, torch.full_like(g, 2.0 ** -20), rel * s * (1 + g.abs()) + low * 2.0 ** -125 * (1 + g.abs()))
        e_silu = e_s * g.abs() + 2.0 ** -23 * (g * s).abs() + 2.0 ** -149
        up = 1 + HALF
        d = dh.abs() + e_dh
        check(dg[i], dh * u * f, up * (e_dh * (u * f).abs() + d * (u.abs() * e_f + 2.0 ** -22 * (u * f).abs() + 2.0 ** -149)),
              "dg")
        check(du[i], dh * g * s, up * (e_dh * (g * s).abs() + d * (e_silu + 2.0 ** -23 * (g * s).abs())), "du")
        check(h[i], g * s * u, up * (u.abs() * e_silu + 2.0 ** -23 * (g * s * u).abs()), "h")


def _byte_of(f):
    """Where feature f's code sits in a row."""
    return f // 32 * 32 + 4 * (f % 8) + f % 32 // 8


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("name,case", [("ragged", (700, 256, 384, 4, 2, None, "uniform")),
                                       ("few_rows", (40, 128, 128, 4, 4, None, "uniform")),
                                       ("capacity", (200, 256, 256, 16, 4, 24, "skew"))])
def test_checkpoint_of_one_non_finite_feature_in_a_block(name, case, value):
    """One column of an expert's gate weights makes one feature of its rows
    non-finite, one of its up weights another: those features' codes are NaN;
    the scales, the other 31 codes of each block and h are those of the same
    layer with these columns zero, bit for bit (a zero does not count for the
    largest magnitude)."""
    L = Layer(name, case=case)
    e, fg, fu = L.E // 2, 37, 70
    assert L.row_of[e].numel() > 0
    L.w_gate[e, :, fg] = 0
    L.w_up[e, :, fu] = 0

    def run():
        ck, h = moe.alloc_checkpoint(L.shape), L.poison(L.P, L.F)
        for t in ck.values():
            t.fill_(0xAB)
        moe.moe_grouped_swiglu_checkpoint(L.shape, L.x_perm, L.w_gate, L.w_up, h, ck["g_q"], ck["u_q"], ck["scale"],
                                          L.ws)
        assert L.status() == 0
        return ck, h.view(torch.int16)

    ref, h_ref = run()
    L.w_gate[e, 5, fg] = value
    L.w_up[e, 9, fu] = value
    got, h = run()
    rows = L.row_of[e]
    assert torch.equal(got["scale"], ref["scale"])
    for q, f in (("g_q", fg), ("u_q", fu)):
        assert ((got[q][rows, _byte_of(f)] & 0x7F) == 0x7F).all(), q
        same = torch.ones(L.F, dtype=torch.bool, device="cuda")
        same[_byte_of(f)] = False
        assert torch.equal(got[q][:, same], ref[q][:, same]), q
        others = torch.ones(L.P, dtype=torch.bool, device="cuda")
        others[rows] = False
        assert torch.equal(got[q][others], ref[q][others]), q
    same = torch.ones(L.F, dtype=torch.bool, device="cuda")
    same[[fg, fu]] = False
    assert torch.equal(h[:, same], h_ref[:, same])
