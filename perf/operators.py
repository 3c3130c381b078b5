"""What the training operators of the layer are timed on: the gradient of the
permutation and of the weighted combine, the SwiGLU products with their 8-bit
activation checkpoint, the backward products that use it, and the gradients of
the expert weights.

Each case names one operator (``op``) and one layer: T tokens, hidden size H,
expert FFN size F, E experts, k per token, C capacity slots per expert (0: the
uncapped layout) and alpha, the skew of the routing (an additive router bias
-alpha ln rank); ``weights`` says which weights' gradient "wgrad" computes.  ``run`` with ``own`` false is the operator in elementary
torch operations in fp32, the rows of the experts one after the other.
"""
import math

import numpy as np
import torch

own = False

OPS = ("combine_backward", "gather_backward", "swiglu_checkpoint", "down_backward", "swiglu_backward", "wgrad")


def _case(name, op, T, H, F, E, k, C=0, alpha=0.0, weights=""):
    return dict(name=name, op=op, T=T, H=H, F=F, E=E, k=k, C=C, alpha=alpha, weights=weights)


def listed():
    return [
        # the smallest layer of the benchmark: one launch, latency counts
        _case("combine_backward tiny", "combine_backward", 64, 128, 256, 8, 2),
        # a training batch of many small experts: HBM traffic of k rows per token
        _case("combine_backward prefill", "combine_backward", 8192, 2048, 768, 128, 8),
        # a ragged batch under a Zipfian load
        _case("gather_backward ragged", "gather_backward", 509, 3584, 2560, 64, 8, alpha=2.0),
        # a training batch of few wide experts
        _case("gather_backward wide", "gather_backward", 8192, 4096, 14336, 8, 2),
        # small batch in the capacity layout with overflow rows: expert weights are streamed
        _case("swiglu_checkpoint capacity", "swiglu_checkpoint", 128, 2048, 1408, 64, 6, C=16, alpha=0.25634765625),
        # training batch, skewed routing: tensor cores and the codes' stores
        _case("swiglu_checkpoint prefill", "swiglu_checkpoint", 8192, 2048, 768, 128, 8, alpha=1.0),
        # the smallest layer: latency of one launch
        _case("down_backward tiny", "down_backward", 64, 128, 256, 8, 2),
        # training batch, unbiased routing: product with the codes read and three outputs stored
        _case("down_backward prefill", "down_backward", 8192, 2048, 768, 128, 8),
        # ragged batch under a Zipfian load, experts without rows
        _case("swiglu_backward ragged", "swiglu_backward", 509, 3584, 2560, 64, 8, alpha=2.0),
        # training batch of few wide experts: the largest product
        _case("swiglu_backward wide", "swiglu_backward", 2048, 4096, 14336, 8, 2),
        # training batch, skewed: the reduction over each expert's rows, two weights per expert
        _case("wgrad prefill", "wgrad", 8192, 2048, 768, 128, 8, alpha=1.0, weights="gate_up"),
        # few rows per expert: writing the weight gradients bounds it
        _case("wgrad wide", "wgrad", 512, 4096, 14336, 8, 2, weights="down"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One to 8192 tokens, ragged; hidden and FFN sizes from 128 up in the
    library's steps of 128; 1 to 128 experts; some in the capacity layout;
    no more weight values and no more products than the listed layers."""
    op = rng.choice(OPS)
    while True:
        T = _log_int(rng, 1, 8192)
        H = 128 * _log_int(rng, 1, 32)
        F = 128 * _log_int(rng, 1, 112)
        E = _log_int(rng, 1, 128)
        k = rng.randint(1, min(E, 8))
        if E * H * F <= 8 * 4096 * 14336 and T * k * H * F <= 2 * 2048 * 4096 * 14336 // 2:
            break
    C = rng.choice([0, 0, 0, 8, 16, 40]) if E * 40 < 8192 else 0
    return dict(op=op, T=T, H=H, F=F, E=E, k=k, C=C, alpha=rng.choice([0.0, 0.0, 0.5, 1.0]),
                weights=rng.choice(["gate_up", "down"]) if op == "wgrad" else "")


def _op(c):
    """The entry point of a case."""
    return (c["op"] + " " + c["weights"]).strip()


def _rows(c):
    """Rows of the permuted buffers (the library's formula)."""
    return c["E"] * c["C"] + c["k"] * max(0, c["T"] - c["C"]) if c["C"] else c["T"] * c["k"]


def work(case):
    T, H, F, E, k = (case[n] for n in ("T", "H", "F", "E", "k"))
    R = T * k
    # experts that get a row, from one routing of these sizes
    rs = np.random.RandomState(0)
    lg = rs.standard_normal((T, E)) - case["alpha"] * np.log(1 + rs.permutation(E))
    touched = np.unique(np.argpartition(-lg, k - 1, axis=1)[:, :k]).size
    W = touched * H * F * 2  # one weight tensor of the touched experts
    b, f = {
        "combine_backward": (T * H * 2 + R * H * 2 + R * 12 + R * H * 2 + R * 4 + T * E * 4, 3 * R * H),
        "gather_backward": (R * H * 2 + R * 4 + T * H * 2, R * H),
        "swiglu_checkpoint": (R * H * 2 + 2 * W + R * F * 2 + 2 * R * F + R * F // 16, 4 * R * H * F),
        "down_backward": (R * H * 2 + W + 2 * R * F + R * F // 16 + 3 * R * F * 2, 2 * R * H * F),
        "swiglu_backward": (2 * R * F * 2 + 2 * W + R * H * 2, 4 * R * H * F),
        "wgrad gate_up": (R * H * 2 + 2 * R * F * 2 + 2 * E * H * F * 2, 4 * R * H * F),
        "wgrad down": (R * F * 2 + R * H * 2 + E * H * F * 2, 2 * R * H * F),
    }[_op(case)]
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs --

def _routing(c, gen, dev):
    """Experts, gate weights and the permutation a forward pass of the layer
    leaves behind, by torch sorts."""
    T, E, k, C = c["T"], c["E"], c["k"], c["C"]
    logits = torch.randn(T, E, generator=gen, device=dev)
    if c["alpha"]:
        rank = torch.randperm(E, generator=gen, device=dev) + 1
        logits = logits - c["alpha"] * rank.float().log()
    top, idx = logits.topk(k, dim=1)
    w = torch.softmax(top, 1)
    flat = idx.reshape(-1)
    counts = torch.bincount(flat, minlength=E)
    offs = torch.cumsum(counts, 0) - counts
    order = torch.argsort(flat, stable=True)
    rank_in = torch.empty_like(flat)
    rank_in[order] = torch.arange(T * k, device=dev) - offs[flat[order]]
    if C:
        spill = (counts - C).clamp(min=0)
        spill_off = torch.cumsum(spill, 0) - spill
        dest = torch.where(rank_in < C, flat * C + rank_in, E * C + spill_off[flat] + rank_in - C)
    else:
        dest = offs[flat] + rank_in
    return dict(idx=idx, w=w, dest=dest, rows=dest[order], counts=counts.tolist(), flat=flat,
                tok=torch.arange(T * k, device=dev) // k)


def _randn(gen, dev, std, *shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0.0, std, generator=gen)


def _on_rows(v, r, P):
    """One value row per routed pair, at its permuted row (zeros elsewhere)."""
    out = torch.zeros((P,) + tuple(v.shape[1:]), dtype=v.dtype, device=v.device)
    out[r["dest"]] = v
    return out


def _quantise(v):
    """Codes and scales of the checkpoint: blocks of 32 features, scale byte
    max(c + 119, 1) for the smallest c with max|v| <= 2^c; byte 4 (f % 8) +
    f / 8 of a block's codes is feature f."""
    R, F = v.shape
    b = v.view(R, F // 32, 32)
    m, e = torch.frexp(b.abs().amax(-1))
    c = e - (m == 0.5).to(e.dtype)
    byte = torch.where(m > 0, c + 119, 1).clamp(min=1).to(torch.int32)
    inv = torch.ldexp(torch.ones_like(byte, dtype=v.dtype), 127 - byte)
    q = (b * inv[..., None]).to(torch.float8_e4m3fn)
    q = q.view(R, F // 32, 4, 8).transpose(2, 3).reshape(R, F)
    return q, byte.to(torch.uint8)


def _values(q, byte, dtype):
    """The values codes and scales stand for."""
    R, F = q.shape
    v = q.view(R, F // 32, 8, 4).transpose(2, 3).reshape(R, F // 32, 32).to(dtype)
    return torch.ldexp(v, byte.to(torch.int32)[..., None] - 127).reshape(R, F)


def _inputs(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    (T, H, F, E, k), op = (c[n] for n in ("T", "H", "F", "E", "k")), _op(c)
    P, R = _rows(c), T * k
    r = _routing(c, gen, dev)
    s = dict(case=c, r=r, P=P)
    n = lambda std, *shape: _randn(gen, dev, std, *shape)  # noqa: E731
    if op == "combine_backward":
        s.update(dout=n(1.0, T, H), y=_on_rows(n(0.3, R, H), r, P))
    elif op == "gather_backward":
        s.update(dx_perm=_on_rows(n(0.1, R, H), r, P))
    elif op == "swiglu_checkpoint":
        x = n(1.0, T, H)
        s.update(x_perm=_on_rows(x[r["tok"]], r, P), w_gate=n(0.02, E, H, F), w_up=n(0.02, E, H, F))
    elif op == "down_backward":
        s.update(dy=_on_rows(n(0.5, R, H), r, P), w_down=n(0.02, E, F, H))
        for name in ("g", "u"):
            q, b = _quantise(torch.empty(R, F, device=dev).normal_(0.0, 1.0, generator=gen))
            s[name + "_q"] = _on_rows(q.view(torch.uint8), r, P)
            s[name + "_b"] = _on_rows(b, r, P)
        s["scale"] = torch.stack((s.pop("g_b"), s.pop("u_b")), -1).contiguous()
    elif op == "swiglu_backward":
        s.update(dg=_on_rows(n(0.1, R, F), r, P), du=_on_rows(n(0.1, R, F), r, P), w_gate=n(0.02, E, H, F),
                 w_up=n(0.02, E, H, F))
    elif op == "wgrad gate_up":
        x = n(1.0, T, H)
        s.update(x_perm=_on_rows(x[r["tok"]], r, P), dg=_on_rows(n(0.1, R, F), r, P), du=_on_rows(n(0.1, R, F), r, P))
    else:
        s.update(h=_on_rows(n(0.3, R, F), r, P), dy=_on_rows(n(0.5, R, H), r, P))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # what the forward pass left: routing tensors and the schedule in the
        # workspace; and the caller's output buffers
        import grouped_expert_gemm_router_b200 as moe
        c, r, P, dev = case, s["r"], s["P"], torch.device("cuda")
        T, H, F, E, k = (c[n] for n in ("T", "H", "F", "E", "k"))
        sh = moe.make_shape(T, H, F, E, k, C=c["C"], capacity=c["C"] > 0)
        ws = torch.empty((moe.moe_workspace_bytes(sh) + 255) // 256 * 256, dtype=torch.uint8, device=dev)
        moe.moe_workspace_init(sh, ws)
        i32 = lambda m: torch.empty(m, dtype=torch.int32, device=dev)  # noqa: E731
        s.update(shape=sh, ws=ws, topk_idx=r["idx"].to(torch.int32).contiguous(), topk_w=r["w"].contiguous(),
                 dest_row=i32(T * k), src_token=i32(P))
        moe.moe_dispatch(sh, s["topk_idx"], i32(E), i32(E + 1), s["src_token"], s["dest_row"], ws)
        z = lambda dt, *m: torch.zeros(m, dtype=dt, device=dev)  # noqa: E731
        bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
        s["out"] = {
            "combine_backward": lambda: dict(dy=z(bf, P, H), dtopk_w=z(f32, T, k), dlogits=z(f32, T, E)),
            "gather_backward": lambda: dict(dx=z(bf, T, H)),
            "swiglu_checkpoint": lambda: dict(h=z(bf, P, F), g_q=z(u8, P, F), u_q=z(u8, P, F), scale=z(u8, P, F // 32, 2)),
            "down_backward": lambda: dict(dg=z(bf, P, F), du=z(bf, P, F), h=z(bf, P, F)),
            "swiglu_backward": lambda: dict(dx_perm=z(bf, P, H)),
            "wgrad gate_up": lambda: dict(dw_gate=z(bf, E, H, F), dw_up=z(bf, E, H, F)),
            "wgrad down": lambda: dict(dw_down=z(bf, E, F, H)),
        }[_op(c)]()
    return s


# --------------------------------------------------------------------- run --

def _run_own(s):
    import grouped_expert_gemm_router_b200 as moe
    op, sh, o, ws = _op(s["case"]), s["shape"], s["out"], s["ws"]
    if op == "combine_backward":
        moe.moe_combine_backward(sh, s["dout"], s["y"], s["dest_row"], s["topk_w"], s["topk_idx"], o["dy"],
                                 o["dtopk_w"], o["dlogits"])
    elif op == "gather_backward":
        moe.moe_gather_backward(sh, s["dx_perm"], s["dest_row"], o["dx"])
    elif op == "swiglu_checkpoint":
        moe.moe_grouped_swiglu_checkpoint(sh, s["x_perm"], s["w_gate"], s["w_up"], o["h"], o["g_q"], o["u_q"],
                                          o["scale"], ws)
        return dict(h=o["h"], g_q=o["g_q"].view(torch.float8_e4m3fn), u_q=o["u_q"].view(torch.float8_e4m3fn),
                    scale=o["scale"].view(torch.float8_e8m0fnu))
    elif op == "down_backward":
        moe.moe_grouped_down_backward(sh, s["dy"], s["w_down"], s["g_q"], s["u_q"], s["scale"], o["dg"], o["du"],
                                      o["h"], ws)
    elif op == "swiglu_backward":
        moe.moe_grouped_swiglu_backward(sh, s["dg"], s["du"], s["w_gate"], s["w_up"], o["dx_perm"], ws)
    elif op == "wgrad gate_up":
        moe.moe_grouped_swiglu_wgrad(sh, s["x_perm"], s["dg"], s["du"], o["dw_gate"], o["dw_up"], ws)
    else:
        moe.moe_grouped_down_wgrad(sh, s["h"], s["dy"], o["dw_down"], ws)
    return dict(o)


def _by_expert(a, s):
    """The routed rows of `a` in fp32, one matrix per expert."""
    return a[s["r"]["rows"]].float().split(s["r"]["counts"])


def _products(rows, weights):
    """Each expert's rows times its weights: one row per routed pair, in expert order."""
    return torch.cat([a @ b for a, b in zip(rows, weights.unbind())])


def _weight_grads(rows, grads):
    return torch.stack([a.t() @ b for a, b in zip(rows, grads)])


def run(s):
    if own:
        return _run_own(s)
    c, r, P = s["case"], s["r"], s["P"]
    T, E, k, op = c["T"], c["E"], c["k"], _op(c)
    bf = torch.bfloat16
    if op == "combine_backward":
        d, w = s["dout"].float(), r["w"]
        dy = _on_rows((w[:, :, None] * d[:, None, :]).to(bf).reshape(T * k, -1), r, P)
        dw = (s["y"][r["dest"]].float().view(T, k, -1) * d[:, None, :]).sum(-1)
        dl = w * (dw - (w * dw).sum(1, keepdim=True))
        return dict(dy=dy, dtopk_w=dw, dlogits=torch.zeros(T, E, device=d.device).scatter_(1, r["idx"], dl))
    if op == "gather_backward":
        return dict(dx=s["dx_perm"][r["dest"]].float().view(T, k, -1).sum(1).to(bf))
    to_rows = lambda v: torch.zeros((P,) + tuple(v.shape[1:]), dtype=v.dtype, device=v.device).index_copy_(  # noqa: E731
        0, r["rows"], v)
    if op == "swiglu_checkpoint":
        x = _by_expert(s["x_perm"], s)
        g, u = _products(x, s["w_gate"].float()), _products(x, s["w_up"].float())
        (gq, gb), (uq, ub) = _quantise(g), _quantise(u)
        codes = lambda q: to_rows(q.view(torch.uint8)).view(torch.float8_e4m3fn)  # noqa: E731
        return dict(h=to_rows((g * torch.sigmoid(g) * u).to(bf)), g_q=codes(gq), u_q=codes(uq),
                    scale=to_rows(torch.stack((gb, ub), -1)).view(torch.float8_e8m0fnu))
    if op == "down_backward":
        dh = _products(_by_expert(s["dy"], s), s["w_down"].float().transpose(1, 2))
        g, u = (_values(s[n][r["rows"]].view(torch.float8_e4m3fn), s["scale"][r["rows"]][..., i], torch.float32)
                for i, n in enumerate(("g_q", "u_q")))
        sg = torch.sigmoid(g)
        return dict(dg=to_rows((dh * u * sg * (1 + g * (1 - sg))).to(bf)), du=to_rows((dh * g * sg).to(bf)),
                    h=to_rows((g * sg * u).to(bf)))
    if op == "swiglu_backward":
        dx = _products(_by_expert(s["dg"], s), s["w_gate"].float().transpose(1, 2))
        dx += _products(_by_expert(s["du"], s), s["w_up"].float().transpose(1, 2))
        return dict(dx_perm=to_rows(dx.to(bf)))
    if op == "wgrad gate_up":
        x = _by_expert(s["x_perm"], s)
        return dict(dw_gate=_weight_grads(x, _by_expert(s["dg"], s)).to(bf),
                    dw_up=_weight_grads(x, _by_expert(s["du"], s)).to(bf))
    return dict(dw_down=_weight_grads(_by_expert(s["h"], s), _by_expert(s["dy"], s)).to(bf))


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """The same in float64, expert by expert.  The codes have no value of
    their own here: where a code's rounding falls is decided by the last bits
    of the fp32 sums, so codes and scales are None."""
    s = _inputs(case, seed)
    c, r, P = case, s["r"], s["P"]
    (T, H, F, E, k), op = (c[n] for n in ("T", "H", "F", "E", "k")), _op(c)
    dev, D = torch.device("cuda"), torch.float64
    z = lambda *m: torch.zeros(m, dtype=D, device=dev)  # noqa: E731
    if op == "combine_backward":
        dy, dw, dl = z(P, H), z(T, k), z(T, E)
        d, w, tok = s["dout"].to(D), r["w"].to(D), torch.arange(T, device=dev)
        dest = r["dest"].view(T, k)
        for j in range(k):
            dy[dest[:, j]] = d * w[:, j:j + 1]
            dw[:, j] = torch.einsum("th,th->t", d, s["y"][dest[:, j]].to(D))
        mean = torch.einsum("tk,tk->t", w, dw)
        for j in range(k):
            dl[tok, r["idx"][:, j]] = w[:, j] * (dw[:, j] - mean)
        return dict(dy=dy, dtopk_w=dw, dlogits=dl)
    if op == "gather_backward":
        return dict(dx=z(T, H).index_add_(0, r["tok"], s["dx_perm"][r["dest"]].to(D)))
    pairs = [r["dest"][r["flat"] == e] for e in range(E)]  # permuted rows of each expert
    if op == "swiglu_checkpoint":
        h = z(P, F)
        for e, i in enumerate(pairs):
            x = s["x_perm"][i].to(D)
            g = x @ s["w_gate"][e].to(D)
            h[i] = g / (1 + torch.exp(-g)) * (x @ s["w_up"][e].to(D))
        return dict(h=h, g_q=None, u_q=None, scale=None)
    if op == "down_backward":
        dg, du, h = z(P, F), z(P, F), z(P, F)
        f = torch.arange(F, device=dev)
        at = f // 32 * 32 + 4 * (f % 8) + f % 32 // 8  # where feature f's code sits
        for e, i in enumerate(pairs):
            dh = s["dy"][i].to(D) @ s["w_down"][e].to(D).T
            g, u = (s[n][i][:, at].view(torch.float8_e4m3fn).to(D) * 2.0 ** (s["scale"][i][:, f // 32, m].to(D) - 127)
                    for m, n in enumerate(("g_q", "u_q")))
            a = torch.exp(-g)
            silu = g / (1 + a)
            dg[i], du[i], h[i] = dh * u * (1 + a + g * a) / (1 + a) ** 2, dh * silu, silu * u
        return dict(dg=dg, du=du, h=h)
    if op == "swiglu_backward":
        dx = z(P, H)
        for e, i in enumerate(pairs):
            dx[i] = s["dg"][i].to(D) @ s["w_gate"][e].to(D).T + s["du"][i].to(D) @ s["w_up"][e].to(D).T
        return dict(dx_perm=dx)
    if op == "wgrad gate_up":
        dwg, dwu = z(E, H, F), z(E, H, F)
        for e, i in enumerate(pairs):
            x = s["x_perm"][i].to(D)
            dwg[e], dwu[e] = x.T @ s["dg"][i].to(D), x.T @ s["du"][i].to(D)
        return dict(dw_gate=dwg, dw_up=dwu)
    dwd = z(E, F, H)
    for e, i in enumerate(pairs):
        dwd[e] = s["h"][i].to(D).T @ s["dy"][i].to(D)
    return dict(dw_down=dwd)
