"""The training entry points on the GPU, each against its formula in float64.

Tolerances, from the arithmetic (never from a run):
  - a result rounded once to bf16 is off by at most 2^-8 of its value;
  - a tensor-core reduction of K products is off by at most
    ACC(K) * sum |a b|, ACC(K) = (K/16 + 2) 2^-22: K/16 accumulations, each
    losing less than 2^-22 of the running magnitude;
  - an fp32 sum of n terms on the CUDA cores by at most n 2^-23 of the sum of
    magnitudes;
  - an e4m3 code is off by at most 2^-4 of the value, or half the smallest
    step, 2^-10 of the scale.
Every buffer starts as NaN, so a read of a row nobody wrote shows, and rows
nobody should write are checked to be untouched."""
import numpy as np
import pytest
import torch

import grouped_expert_gemm_router_b200 as moe

pytestmark = pytest.mark.gpu
D = torch.float64
HALF = 2.0 ** -8


def acc(K):
    return (K / 16 + 2) * 2.0 ** -22


# T, H, F, E, k, C (None: uncapped), routing
CASES = {
    "one_token": (1, 128, 128, 1, 1, None, "uniform"),
    "tiny": (64, 128, 256, 8, 2, None, "uniform"),
    # several row tiles per expert, 384 = an odd number of 128-blocks (output tiles across gate and up)
    "two_tiles": (700, 256, 384, 4, 2, None, "uniform"),
    "skew_H384": (301, 384, 256, 8, 3, None, "skew"),
    "one_expert": (300, 128, 256, 1, 1, None, "uniform"),
    "all_experts": (40, 128, 128, 4, 4, None, "uniform"),
    # all tokens on the same two of sixteen experts: fourteen without rows
    "empty_experts": (130, 256, 128, 16, 2, None, "first"),
    "capacity": (200, 256, 256, 16, 4, 24, "skew"),
    "capacity_unused": (50, 128, 256, 4, 2, 64, "uniform"),
    "capacity_zero": (90, 128, 128, 4, 2, 0, "skew"),
    "experts_256_k9": (96, 128, 128, 256, 9, None, "uniform"),
    "experts_256_k256": (5, 128, 128, 256, 256, None, "uniform"),
    "long_rows": (4, 4096, 128, 3, 3, None, "uniform"),
    # enough tokens for one warp each, and for four; an odd last block
    "many_tokens": (4001, 384, 128, 4, 2, None, "uniform"),
    "many_tokens_H1152": (901, 1152, 128, 8, 4, None, "skew"),
    "capacity_long": (1500, 128, 256, 3, 2, 700, "skew"),
    # long reductions: 256-feature units (here of full and of ragged row tiles, and an odd last feature block)
    "wide_units": (700, 3584, 384, 2, 1, None, "uniform"),
    "wide_units_capacity": (400, 3712, 640, 2, 1, 130, "uniform"),
    "wide_unit_one_block": (300, 3584, 128, 1, 1, None, "uniform"),
    # more row tiles than are made equally high
    "eleven_tiles": (2600, 128, 256, 1, 1, None, "uniform"),
}


class Layer:
    """One layer's tensors on the device, its dispatch, and poisoned buffers."""

    def __init__(self, name, seed=0, case=None):
        T, H, F, E, k, C, routing = case or CASES[name]
        self.T, self.H, self.F, self.E, self.k, self.C = T, H, F, E, k, C
        g = torch.Generator(device="cuda").manual_seed(1000 + seed)
        self.gen = g
        self.shape = moe.make_shape(T, H, F, E, k, C=C or 0, capacity=C is not None)
        self.P = moe.moe_permuted_rows(self.shape)
        lg = torch.randn(T, E, generator=g, device="cuda")
        if routing == "skew":
            lg -= 1.5 * torch.arange(1, E + 1, device="cuda").float().log()
        if routing == "first":
            lg[:, k:] = -float("inf")
        top, idx = lg.topk(k, 1)
        self.idx = idx.int().contiguous()
        self.w = torch.softmax(top, 1).contiguous()
        self.x = self.randn(T, H)
        self.w_gate, self.w_up, self.w_down = (self.randn(*n, std=1.0 / n[1] ** 0.5)
                                               for n in ((E, H, F), (E, H, F), (E, F, H)))
        self.ws = torch.empty((moe.moe_workspace_bytes(self.shape) + 255) // 256 * 256, dtype=torch.uint8,
                              device="cuda")
        moe.moe_workspace_init(self.shape, self.ws)
        self.counts, self.offsets = self.i32(E), self.i32(E + 1)
        self.src, self.dest = self.i32(self.P), self.i32(T * k)
        moe.moe_dispatch(self.shape, self.idx, self.counts, self.offsets, self.src, self.dest, self.ws)
        torch.cuda.synchronize()
        d = self.dest.long()
        flat = self.idx.reshape(-1).long()
        assert torch.equal(torch.bincount(flat, minlength=E).int(), self.counts)
        assert d.unique().numel() == T * k and int(d.min()) >= 0 and int(d.max()) < self.P
        tok = torch.arange(T * k, device="cuda") // k
        self.row_of = [d[flat == e] for e in range(E)]  # permuted rows of each expert
        self.filled = torch.zeros(self.P, dtype=torch.bool, device="cuda")
        self.filled[d] = True
        self.x_perm = self.poison(self.P, H)
        self.x_perm[d] = self.x[tok]

    def randn(self, *n, std=1.0):
        return torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=self.gen)

    def i32(self, n):
        return torch.full((n,), -7, dtype=torch.int32, device="cuda")

    def poison(self, *n):
        return torch.full(n, float("nan"), dtype=torch.bfloat16, device="cuda")

    def rows(self, *n, std=1.0):
        """A permuted buffer with random filled rows and NaN elsewhere."""
        v = self.randn(*n, std=std)
        v[~self.filled] = float("nan")
        return v

    def checkpoint(self, seed_std=1.0):
        """A checkpoint with random codes (as a forward pass would leave), 0xFF where no row is."""
        q = {}
        for n in ("g_q", "u_q"):
            v = (torch.randn(self.P, self.F, generator=self.gen, device="cuda") * 60).to(torch.float8_e4m3fn)
            q[n] = v.view(torch.uint8).clone()
            q[n][~self.filled] = 0xFF
        q["scale"] = torch.randint(119, 124, (self.P, self.F // 32, 2), generator=self.gen, device="cuda",
                                   dtype=torch.uint8)
        q["scale"][~self.filled] = 0xFF
        return q

    def status(self):
        return moe.moe_read_status(self.ws)

    def untouched(self, *bufs):
        for b in bufs:
            assert torch.isnan(b[~self.filled]).all(), "an unfilled row was written"


def close(got, ref, tol, what):
    """|got - ref| <= tol, element by element, everything finite."""
    got = got.to(D)
    assert torch.isfinite(got).all(), "%s: not finite" % what
    bad = (got - ref).abs() - tol
    assert bad.max() <= 0, "%s: off by %g more than allowed (of %g) at %d" % (
        what, bad.max(), ref.abs().max(), int(bad.argmax()))


@pytest.mark.parametrize("name", list(CASES))
def test_dispatch_is_the_index_part_of_permute(name):
    L = Layer(name)
    ws = torch.empty_like(L.ws)
    moe.moe_workspace_init(L.shape, ws)
    c, o, s, d, xp = L.i32(L.E), L.i32(L.E + 1), L.i32(L.P), L.i32(L.T * L.k), L.poison(L.P, L.H)
    moe.moe_permute(L.shape, L.x, L.idx, c, o, s, d, xp, ws)
    for a, b in ((c, L.counts), (o, L.offsets), (s, L.src), (d, L.dest)):
        assert torch.equal(a, b)
    lay = moe.moe_workspace_layout(L.shape)
    n = 16 * int(ws[lay.num_tiles:lay.num_tiles + 4].view(torch.int32))
    assert torch.equal(ws[lay.tile_map:lay.tile_map + n], L.ws[lay.tile_map:lay.tile_map + n])


@pytest.mark.parametrize("name", list(CASES))
def test_combine_backward(name):
    L = Layer(name)
    y, dout = L.rows(L.P, L.H), L.randn(L.T, L.H)
    dy, dw = L.poison(L.P, L.H), torch.full((L.T, L.k), float("nan"), device="cuda")
    dl = torch.full((L.T, L.E), float("nan"), device="cuda")
    moe.moe_combine_backward(L.shape, dout, y, L.dest, L.w, L.idx, dy, dw, dl)
    d = L.dest.long().view(L.T, L.k)
    w, do = L.w.to(D), dout.to(D)
    ref_dy = w[:, :, None] * do[:, None, :]
    # one fp32 product, one rounding
    close(dy[d], ref_dy, (HALF + 2.0 ** -23) * ref_dy.abs(), "dy")
    L.untouched(dy)
    prod = y[d].to(D) * do[:, None, :]
    ref_dw = prod.sum(-1)
    e_dw = L.H * 2.0 ** -23 * prod.abs().sum(-1)
    close(dw, ref_dw, e_dw, "dtopk_w")
    mean = (w * ref_dw).sum(1, keepdim=True)
    e_mean = (w * e_dw).sum(1, keepdim=True) + (L.k + 2) * 2.0 ** -23 * (w * ref_dw.abs()).sum(1, keepdim=True)
    ref = torch.zeros(L.T, L.E, dtype=D, device="cuda").scatter_(1, L.idx.long(), w * (ref_dw - mean))
    tol = torch.zeros_like(ref).scatter_(
        1, L.idx.long(), w * (e_dw + e_mean + 2.0 ** -22 * (ref_dw.abs() + mean.abs())) + 1e-45)
    close(dl, ref, tol, "dlogits")  # exactly zero off the selected experts
    # without dlogits: the other two, the same bits
    dy2, dw2 = L.poison(L.P, L.H), torch.empty_like(dw)
    moe.moe_combine_backward(L.shape, dout, y, L.dest, L.w, None, dy2, dw2)
    assert torch.equal(dy2[d], dy[d]) and torch.equal(dw2, dw)


@pytest.mark.parametrize("name", list(CASES))
def test_gather_backward(name):
    L = Layer(name)
    dxp, dx = L.rows(L.P, L.H), L.poison(L.T, L.H)
    moe.moe_gather_backward(L.shape, dxp, L.dest, dx)
    v = dxp[L.dest.long().view(L.T, L.k)].to(D)
    ref = v.sum(1)
    close(dx, ref, HALF * ref.abs() + (1 + HALF) * L.k * 2.0 ** -23 * v.abs().sum(1), "dx")


def _checkpoint_ref(L):
    """g, u of the filled rows in float64, with the sums of magnitudes."""
    out = []
    for w in (L.w_gate, L.w_up):
        v, m = (torch.zeros(L.P, L.F, dtype=D, device="cuda") for _ in range(2))
        for e, i in enumerate(L.row_of):
            v[i] = L.x_perm[i].to(D) @ w[e].to(D)
            m[i] = L.x_perm[i].to(D).abs() @ w[e].to(D).abs()
        out.append((v, m))
    return out


def _new_checkpoint(L):
    ck = moe.alloc_checkpoint(L.shape)
    for t in ck.values():
        t.fill_(0xAB)
    return ck


@pytest.mark.parametrize("name", list(CASES))
def test_swiglu_checkpoint(name):
    L = Layer(name)
    h0, h, ck = L.poison(L.P, L.F), L.poison(L.P, L.F), _new_checkpoint(L)
    moe.moe_grouped_swiglu(L.shape, L.x_perm, L.w_gate, L.w_up, h0, L.ws)
    moe.moe_grouped_swiglu_checkpoint(L.shape, L.x_perm, L.w_gate, L.w_up, h, ck["g_q"], ck["u_q"], ck["scale"], L.ws)
    assert torch.equal(h.view(torch.int16), h0.view(torch.int16)), "h must be moe_grouped_swiglu's"
    for t in ck.values():
        assert (t[~L.filled] == 0xAB).all(), "codes of an unfilled row were written"
    for which, (n, (v, m)) in enumerate(zip(("g_q", "u_q"), _checkpoint_ref(L))):
        f = L.filled
        err = acc(L.H) * m[f]
        s = 2.0 ** (ck["scale"][f][..., which].to(D) - 127)
        amax = v[f].view(-1, L.F // 32, 32).abs().amax(-1)
        e = err.view(-1, L.F // 32, 32).amax(-1)
        assert (amax - e <= 256 * s).all() and (amax + e > 128 * s).all(), "scale of %s" % n
        got = moe.checkpoint_values(ck[n], ck["scale"], which)[f]
        close(got, v[f], (2.0 ** -4 * v[f].abs() + 2.0 ** -10 * s.repeat_interleave(32, 1)) + (1 + 2.0 ** -4) * err, n)
    assert L.status() == 0


def test_checkpoint_of_zero_tiny_huge_and_non_finite_rows():
    """Rows of zeros (scale byte 1, zero codes), below and near the ends of
    the scale's range, and rows that hold infinities: their codes are NaN and
    no other row changes."""
    L = Layer("two_tiles")
    h, ck0, ck = L.poison(L.P, L.F), _new_checkpoint(L), _new_checkpoint(L)

    def run(c):
        moe.moe_grouped_swiglu_checkpoint(L.shape, L.x_perm, L.w_gate, L.w_up, h, c["g_q"], c["u_q"], c["scale"], L.ws)

    run(ck0)
    zero, tiny, huge, inf, nan = 3, 40, 300, 500, 1000
    L.x_perm[zero] = 0
    L.x_perm[tiny] = 2.0 ** -126
    L.x_perm[huge] *= 2.0 ** 120
    L.x_perm[inf, 5] = float("inf")
    L.x_perm[nan, 7] = float("nan")
    run(ck)
    same = torch.ones(L.P, dtype=torch.bool, device="cuda")
    same[[zero, tiny, huge, inf, nan]] = False
    for n in ck:
        assert torch.equal(ck[n][same], ck0[n][same]), n
    for which, n in enumerate(("g_q", "u_q")):
        assert (ck[n][zero] & 0x7F).max() == 0 and (ck["scale"][zero, :, which] == 1).all()
        for r in (inf, nan):
            assert ((ck[n][r] & 0x7F) == 0x7F).all() and (ck["scale"][r, :, which] == 1).all()
        v, m = _checkpoint_ref(L)[which]
        got = moe.checkpoint_values(ck[n], ck["scale"], which).to(D)
        # the tiny row's values (about 2^-126) are far below 2^-118, where the
        # scale stops at 2^-126: 2^-4 of the value from the codes' three
        # mantissa bits, or half their smallest step, 2^-10 2^-126; the fp32
        # sums lose up to a subnormal step, 2^-149, per accumulated product
        assert (ck["scale"][tiny, :, which] == 1).all()
        close(got[tiny], v[tiny], (2.0 ** -4 * v[tiny].abs() + 2.0 ** -136) + 2 * L.H * 2.0 ** -149
              + 2 * acc(L.H) * m[tiny], "tiny")
        s = 2.0 ** (ck["scale"][huge, :, which].to(D) - 127).repeat_interleave(32)
        close(got[huge], v[huge], 2.0 ** -4 * v[huge].abs() + 2.0 ** -10 * s + 2 * acc(L.H) * m[huge], "huge")


@pytest.mark.parametrize("name", list(CASES))
def test_down_backward(name):
    L = Layer(name)
    dy, ck = L.rows(L.P, L.H), L.checkpoint()
    dg, du, h = (L.poison(L.P, L.F) for _ in range(3))
    moe.moe_grouped_down_backward(L.shape, dy, L.w_down, ck["g_q"], ck["u_q"], ck["scale"], dg, du, h, L.ws)
    L.untouched(dg, du, h)
    g, u = (moe.checkpoint_values(ck[n], ck["scale"], i).to(D) for i, n in enumerate(("g_q", "u_q")))
    for e, i in enumerate(L.row_of):
        if not i.numel():
            continue
        a, w = dy[i].to(D), L.w_down[e].to(D)
        dh, err = a @ w.T, acc(L.H) * (a.abs() @ w.T.abs())
        gg, uu = g[i], u[i]
        s = torch.sigmoid(gg)
        # the sigmoid, the products and the sum 1 + g (1 - s): a dozen fp32
        # roundings of terms of at most (1 + |g|) s, with the fast exponential
        # (2 + |1.45 g| ulp) and division (2 ulp)
        rel = (16 + 2 * gg.abs()) * 2.0 ** -23
        fg = s * (1 + gg * (1 - s))
        big = s * (1 + gg.abs()) * uu.abs()
        ref = dh * uu * fg
        close(dg[i], ref, HALF * ref.abs() + (1 + HALF) * (err * (uu * fg).abs() + rel * dh.abs() * big), "dg")
        ref = dh * gg * s
        close(du[i], ref, HALF * ref.abs() + (1 + HALF) * ((err + rel * dh.abs()) * (gg * s).abs()), "du")
        ref = gg * s * uu
        close(h[i], ref, (HALF + 2 * rel) * ref.abs(), "h")
    assert L.status() == 0


@pytest.mark.parametrize("name", list(CASES))
def test_swiglu_backward(name):
    L = Layer(name)
    dg, du, dxp = L.rows(L.P, L.F), L.rows(L.P, L.F), L.poison(L.P, L.H)
    moe.moe_grouped_swiglu_backward(L.shape, dg, du, L.w_gate, L.w_up, dxp, L.ws)
    L.untouched(dxp)
    for e, i in enumerate(L.row_of):
        if not i.numel():
            continue
        a, b, wg, wu = dg[i].to(D), du[i].to(D), L.w_gate[e].to(D).T, L.w_up[e].to(D).T
        ref = a @ wg + b @ wu
        close(dxp[i], ref, HALF * ref.abs() + (1 + HALF) * acc(2 * L.F) * (a.abs() @ wg.abs() + b.abs() @ wu.abs()),
              "dx_perm")
    assert L.status() == 0


@pytest.mark.parametrize("name", list(CASES))
def test_wgrad(name):
    L = Layer(name)
    dg, du, h, dy = (L.rows(L.P, n) for n in (L.F, L.F, L.F, L.H))
    dwg, dwu, dwd = L.poison(L.E, L.H, L.F), L.poison(L.E, L.H, L.F), L.poison(L.E, L.F, L.H)
    moe.moe_grouped_swiglu_wgrad(L.shape, L.x_perm, dg, du, dwg, dwu, L.ws)
    moe.moe_grouped_down_wgrad(L.shape, h, dy, dwd, L.ws)
    for e, i in enumerate(L.row_of):
        for got, a, b, what in ((dwg, L.x_perm, dg, "dw_gate"), (dwu, L.x_perm, du, "dw_up"), (dwd, h, dy, "dw_down")):
            a, b = a[i].to(D), b[i].to(D)
            ref = a.T @ b  # zeros for an expert without rows
            close(got[e], ref, HALF * ref.abs() + (1 + HALF) * acc(i.numel()) * (a.abs().T @ b.abs()),
                  "%s[%d], %d rows" % (what, e, i.numel()))
    assert L.status() == 0


# ------------------------------------------------------------- all together --

def layer_f64(x, wr, wg, wu, wd, idx):
    """The layer in float64 with the routing's experts fixed: out, and the
    logits (for their gradient)."""
    logits = x @ wr
    w = torch.softmax(logits.gather(1, idx), 1)
    out = torch.zeros_like(x)
    for j in range(idx.shape[1]):
        g = torch.einsum("th,thf->tf", x, wg[idx[:, j]])
        u = torch.einsum("th,thf->tf", x, wu[idx[:, j]])
        h = g * torch.sigmoid(g) * u
        out = out + w[:, j:j + 1] * torch.einsum("tf,tfh->th", h, wd[idx[:, j]])
    return out, logits


def _forward_backward(L, wr, dout, stream=None, rebuild=False):
    b = moe.alloc_buffers(L.shape)
    b.update(x=L.x, w_router=wr, bias=None, w_gate=L.w_gate, w_up=L.w_up, w_down=L.w_down)
    b.update(moe.alloc_checkpoint(L.shape))
    moe.moe_forward_checkpoint(L.shape, b, b["ws"], stream)
    b["fwd_h"] = b["h"]
    b.update(moe.alloc_backward_buffers(L.shape))
    b["dout"] = dout
    moe.moe_backward(L.shape, b, b["ws"], stream, rebuild_dispatch=rebuild)
    return b


RESULTS = ("dx", "dtopk_w", "dlogits", "dw_gate", "dw_up", "dw_down")


@pytest.mark.parametrize("name", ["tiny", "skew_H384", "capacity"])
def test_layer_gradient(name):
    """Forward and backward through the public entry points against the
    float64 gradient of the whole layer (and that against differences).  The
    checkpoint holds g and u to 2^-4 each, and dg, du, h are smooth functions
    of both with relative slopes up to about 1.3 (g silu'/silu for moderate g)
    plus dg's own zero crossing, so in norm the gradients that go through it
    are within 2 * 1.3 * 2^-4 / sqrt(3) (uniform rounding errors) < 0.1;
    dtopk_w and dlogits do not go through it: bf16 roundings of h and y,
    with tanh.approx in silu, below 2e-2."""
    L = Layer(name)
    wr = torch.randn(L.H, L.E, generator=L.gen, device="cuda") / L.H ** 0.5
    dout = L.randn(L.T, L.H)
    b = _forward_backward(L, wr, dout)
    torch.cuda.synchronize()
    assert moe.moe_read_status(b["ws"]) == 0
    # the forward outputs are moe_forward's
    f = moe.alloc_buffers(L.shape)
    f.update(x=L.x, w_router=wr, bias=None, w_gate=L.w_gate, w_up=L.w_up, w_down=L.w_down)
    moe.moe_forward(L.shape, f, f["ws"])
    assert torch.equal(f["out"], b["out"]) and torch.equal(f["dest_row"], b["dest_row"])
    idx = b["topk_idx"].long()
    ps = [t.to(D).requires_grad_() for t in (L.x, wr, L.w_gate, L.w_up, L.w_down)]
    out, logits = layer_f64(*ps, idx)
    logits.retain_grad()
    (out * dout.to(D)).sum().backward()
    dx_experts = ps[0].grad - logits.grad @ ps[1].detach().T  # the router's share is the caller's

    def rel(a, r):
        return float((a.to(D) - r).norm() / r.norm())

    assert rel(b["dlogits"], logits.grad) < 2e-2
    for n, r in (("dx", dx_experts), ("dw_gate", ps[2].grad), ("dw_up", ps[3].grad), ("dw_down", ps[4].grad)):
        assert rel(b[n], r) < 0.1, (n, rel(b[n], r))
    # the float64 gradient against central differences along the kernels' own gradient
    with torch.no_grad():
        for i, g in ((0, dx_experts), (2, b["dw_gate"].to(D)), (3, b["dw_up"].to(D)), (4, b["dw_down"].to(D))):
            v = g / g.norm()
            eps = 1e-4
            up, dn = (layer_f64(*[p + s * eps * v if j == i else p for j, p in enumerate(ps)], idx)[0]
                      for s in (1, -1))
            diff = float(((up - dn) * dout.to(D)).sum() / (2 * eps))
            assert abs(diff - float((ps[i].grad * v).sum())) <= 1e-5 * abs(diff) + 1e-6


@pytest.mark.parametrize("name", ["two_tiles", "capacity", "empty_experts", "many_tokens", "wide_units"])
def test_backward_is_its_steps_and_repeats(name):
    """moe_backward gives the single steps' results bit for bit, twice over;
    with dx, dlogits or weight gradients not wanted the others are the same;
    with the workspace used by another batch in between, rebuild_dispatch
    gives the same again."""
    L = Layer(name)
    wr = torch.randn(L.H, L.E, generator=L.gen, device="cuda") / L.H ** 0.5
    dout = L.randn(L.T, L.H)
    b = _forward_backward(L, wr, dout)
    ref = {n: b[n].clone() for n in RESULTS}
    s, ws = L.shape, b["ws"]
    c = moe.alloc_backward_buffers(s)
    moe.moe_combine_backward(s, dout, b["y"], b["dest_row"], b["topk_w"], b["topk_idx"], c["dy"], c["dtopk_w"],
                             c["dlogits"])
    moe.moe_grouped_down_backward(s, c["dy"], L.w_down, b["g_q"], b["u_q"], b["scale"], c["dg"], c["du"], c["h"], ws)
    moe.moe_grouped_down_wgrad(s, c["h"], c["dy"], c["dw_down"], ws)
    moe.moe_grouped_swiglu_wgrad(s, b["x_perm"], c["dg"], c["du"], c["dw_gate"], c["dw_up"], ws)
    moe.moe_grouped_swiglu_backward(s, c["dg"], c["du"], L.w_gate, L.w_up, c["dx_perm"], ws)
    moe.moe_gather_backward(s, c["dx_perm"], b["dest_row"], c["dx"])
    for n in RESULTS:
        assert torch.equal(c[n], ref[n]), n
    for skip in (("dx",), ("dlogits",), ("dw_down",), ("dw_gate", "dw_up")):
        d = dict(b, **{n: torch.zeros_like(b[n]) for n in RESULTS})
        d.update({n: None for n in skip})
        moe.moe_backward(s, d, ws)
        for n in RESULTS:
            if n not in skip:
                assert torch.equal(d[n], ref[n]), (skip, n)
    # another batch through the same workspace
    idx2 = torch.zeros_like(b["topk_idx"]) + torch.arange(L.k, dtype=torch.int32, device="cuda")
    moe.moe_dispatch(s, idx2, L.i32(L.E), L.i32(L.E + 1), L.i32(L.P), L.i32(L.T * L.k), ws)
    d = dict(b, **{n: torch.zeros_like(b[n]) for n in RESULTS})
    moe.moe_backward(s, d, ws, rebuild_dispatch=True)
    for n in RESULTS:
        assert torch.equal(d[n], ref[n]), n
    assert moe.moe_read_status(ws) == 0


@pytest.mark.parametrize("name", ["two_tiles", "capacity", "many_tokens"])
def test_forward_checkpoint_in_every_form_of_the_layer(name):
    """The combine inside the down GEMM and logits given by the caller: out
    and the gradients of the plain form, bit for bit."""
    L = Layer(name)
    wr = torch.randn(L.H, L.E, generator=L.gen, device="cuda") / L.H ** 0.5
    dout = L.randn(L.T, L.H)
    ref = _forward_backward(L, wr, dout)
    s = L.shape
    for flags in (moe.MOE_FLAG_FUSED_COMBINE, moe.MOE_FLAG_LOGITS_IN):
        L.shape = moe.make_shape(s.T, s.H, s.F, s.E, s.k, C=s.C, flags=s.flags | flags)
        b = moe.alloc_buffers(L.shape)
        b["logits"].copy_(ref["logits"])
        b.update(x=L.x, w_router=wr, bias=None, w_gate=L.w_gate, w_up=L.w_up, w_down=L.w_down)
        b.update(moe.alloc_checkpoint(L.shape))
        moe.moe_forward_checkpoint(L.shape, b, b["ws"])
        out = b["out"].clone()
        b.update(moe.alloc_backward_buffers(L.shape))
        b["dout"] = dout
        moe.moe_backward(L.shape, b, b["ws"])
        assert torch.equal(out, ref["out"])
        for n in RESULTS:
            assert torch.equal(b[n], ref[n]), n
        assert moe.moe_read_status(b["ws"]) == 0


def test_backward_captured_and_replayed_on_new_inputs():
    """One captured forward + backward serves other inputs written into the
    same buffers, while an eager pass of another layer runs on its own stream
    and workspace."""
    L = Layer("skew_H384")
    wr = torch.randn(L.H, L.E, generator=L.gen, device="cuda") / L.H ** 0.5
    dout = L.randn(L.T, L.H)
    b = moe.alloc_buffers(L.shape)
    b.update(x=L.x.clone(), w_router=wr, bias=None, w_gate=L.w_gate, w_up=L.w_up, w_down=L.w_down)
    b.update(moe.alloc_checkpoint(L.shape))
    h = b["h"]
    b.update(moe.alloc_backward_buffers(L.shape))
    b["h"] = h  # the recomputed activations may take the forward buffer
    b["dout"] = dout.clone()

    def step(stream):
        moe.moe_forward_checkpoint(L.shape, b, b["ws"], stream)
        moe.moe_backward(L.shape, b, b["ws"], stream)

    step(None)
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=cap):
        step(cap)
    other = Layer("capacity", seed=5)
    wr2 = torch.randn(other.H, other.E, generator=other.gen, device="cuda") / other.H ** 0.5
    dout2 = other.randn(other.T, other.H)
    side = torch.cuda.Stream()
    for seed in (1, 2):
        b["x"].normal_(0.0, 1.0, generator=L.gen)
        b["dout"].normal_(0.0, 1.0, generator=L.gen)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            o = _forward_backward(other, wr2, dout2, side)
        graph.replay()
        torch.cuda.synchronize()
        L.x = b["x"]
        e = _forward_backward(L, wr, b["dout"])
        o2 = _forward_backward(other, wr2, dout2)
        torch.cuda.synchronize()
        for n in RESULTS + ("out",):
            assert torch.equal(b[n], e[n]), n
            assert torch.equal(o[n], o2[n]), n
    assert moe.moe_read_status(b["ws"]) == 0


def test_bad_rows_are_skipped():
    """Row and expert indices outside their range (left by an earlier device
    error) are skipped, not followed."""
    L = Layer("tiny")
    y, dout = L.rows(L.P, L.H), L.randn(L.T, L.H)
    bad = L.dest.clone()
    bad[0], bad[3] = -1, L.P
    idx = L.idx.clone()
    idx[2, 0] = L.E
    dy, dw = L.poison(L.P, L.H), torch.full((L.T, L.k), float("nan"), device="cuda")
    dl = torch.full((L.T, L.E), float("nan"), device="cuda")
    moe.moe_combine_backward(L.shape, dout, y, bad, L.w, idx, dy, dw, dl)
    skipped = L.dest[[0, 3]].long()
    assert torch.isnan(dy[skipped]).all() and (dw.view(-1)[[0, 3]] == 0).all()
    assert torch.isfinite(dl).all()
    dxp, dx = L.rows(L.P, L.H), L.poison(L.T, L.H)
    moe.moe_gather_backward(L.shape, dxp, bad, dx)
    d = L.dest.long().view(L.T, L.k)
    assert torch.equal(dx[0], dxp[d[0, 1]]) and torch.equal(dx[1], dxp[d[1, 0]])
