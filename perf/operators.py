"""Cases of the operators that stand around the FP8 linear layers of a training block.

  residual_norm           y = x + scale * gate * post(h), then the RMS norm of y as the FP8 input of the next linear
  residual_norm_backward  the gradients of x, h (as FP8, the dY of the linear before), both weights and the gate
  swiglu                  silu(gate) * up of the fused gate+up projection, as the FP8 input of the down projection
  swiglu_backward         the gradient of the fused projection's output, as its FP8 dY
  orthogonalize           five Newton-Schulz steps of a weight gradient, as the Muon optimiser takes

With `own` false the operators run in elementary torch operations in 32 bits; with `own` true through
fp8_block_scaled_13_b200.  FP8 codes come back as torch.float8_e4m3fn and their scales as torch.float8_e8m0fnu, in
the blocked layout that the GEMMs read; bytes of that layout that stand for no group are zero.

Sizes: hidden 2048 and FFN 6144 at up to 32768 tokens are this repository's full block; the weights 2048 x 2048 and
12288 x 2048 are its projections.  The others are ragged or small ones of the same kind.
"""
import math

import torch

own = False

EPS = 1e-6
NS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7


def listed():
    return [
        # one short decode batch: only the latency counts, and only the forward codes are needed
        {"name": "norm_16", "op": "norm", "t": 16, "d": 2048, "res": True, "post": False, "gate": "none", "layout": "rowwise", "w32": False},
        # the first norm of a micro-batch of two 4096-token sequences: nothing to add yet
        {"name": "norm_8192_pre", "op": "norm", "t": 8192, "d": 2048, "res": False, "post": False, "gate": "none", "layout": "both", "w32": True},
        # the full block's tokens, with norms before and after the block and a gate for each token
        {"name": "norm_32768_post", "op": "norm", "t": 32768, "d": 2048, "res": True, "post": True, "gate": "token", "layout": "both", "w32": True},
        # a ragged token count, a gate for each channel (layer scale)
        {"name": "norm_bwd_1000", "op": "norm_bwd", "t": 1000, "d": 1152, "res": True, "post": False, "gate": "channel", "layout": "both", "w32": False},
        # the full block's backward pass between two linears, gate for each element
        {"name": "norm_bwd_32768", "op": "norm_bwd", "t": 32768, "d": 2048, "res": True, "post": True, "gate": "full", "layout": "both", "w32": True},
        # a few hundred tokens of a narrow FFN
        {"name": "swiglu_300", "op": "swiglu", "t": 300, "f": 384, "layout": "both"},
        # the full block's FFN
        {"name": "swiglu_32768", "op": "swiglu", "t": 32768, "f": 6144, "layout": "both"},
        # its backward pass at one odd token count and at the full one
        {"name": "swiglu_bwd_777", "op": "swiglu_bwd", "t": 777, "f": 1408, "layout": "both"},
        {"name": "swiglu_bwd_16384", "op": "swiglu_bwd", "t": 16384, "f": 6144, "layout": "both"},
        # a small projection in BF16, where the launches cost most; odd sizes
        {"name": "ortho_200x333", "op": "ortho", "n": 200, "k": 333, "g32": False},
        # the attention output projection's FP32 main gradient
        {"name": "ortho_2048x2048", "op": "ortho", "n": 2048, "k": 2048, "g32": True},
        # the gate+up projection's, tall
        {"name": "ortho_12288x2048", "op": "ortho", "n": 12288, "k": 2048, "g32": True},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "swiglu", "swiglu_bwd", "ortho", "ortho"])
    if op == "ortho":
        n, k = _spread(rng, 16, 6144), _spread(rng, 16, 2048)
        n, k = (n, k) if rng.random() < 0.6 else (k, n)
        return {"op": op, "n": n, "k": k, "g32": rng.random() < 0.7}
    t = _spread(rng, 1, 32768)
    layout = rng.choice(["both", "both", "both", "rowwise"])
    if op in ("swiglu", "swiglu_bwd"):
        return {"op": op, "t": min(t, 16384) if op == "swiglu_bwd" else t, "f": 128 * _spread(rng, 1, 48), "layout": layout}
    d = 128 * _spread(rng, 1, 64)
    t = min(t, 32768 * 2048 // d)
    res = rng.random() < 0.85
    return {"op": op, "t": t, "d": d, "res": res, "post": res and rng.random() < 0.5,
            "gate": rng.choice(["none", "token", "channel", "full"]) if res else "none",
            "layout": layout, "w32": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def _gate_shape(case):
    t, d = case["t"], case["d"]
    return {"token": (t, 1), "channel": (1, d), "full": (t, d)}[case["gate"]]


def _scale_bytes(rows, groups):
    return (rows + 127) // 128 * ((groups + 3) // 4) * 512


def _code_buffers(t, d, layout):
    """What a training loop keeps from step to step: the codes' and scales' memory."""
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    out = {"q": z(t, d), "s": z(_scale_bytes(t, d // 128))}
    if layout == "both":
        out["qt"] = z(d, (t + 15) // 16 * 16)
        out["st"] = z(_scale_bytes(d, (t + 127) // 128))
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    op, s = case["op"], {"case": dict(case)}
    if op == "ortho":
        # a weight gradient: a few strong directions over a broad floor
        n, k = case["n"], case["k"]
        r = max(1, min(n, k) // 8)
        grad = randn(n, r) @ randn(r, k) * (1.0 / r ** 0.5) + randn(n, k)
        s["grad"] = (grad * 1e-3).to(torch.float32 if case["g32"] else bf)
        s["out"] = torch.zeros(n, k, dtype=bf, device="cuda")
        return s
    t = case["t"]
    if op in ("swiglu", "swiglu_bwd"):
        f = case["f"]
        s["gu"] = randn(t, 2 * f).to(bf)
        if op == "swiglu_bwd":
            s["da"] = (randn(t, f) * 1e-3).to(bf)
        s["codes"] = _code_buffers(t, f if op == "swiglu" else 2 * f, case["layout"])
        return s
    d = case["d"]
    wt = torch.float32 if case["w32"] else bf
    x = randn(t, d)
    x[:, :: max(1, d // 8)] *= 20.0  # a few strong channels, as residual streams have
    s["x"] = x.to(bf)
    s["w_pre"] = (1.0 + 0.1 * randn(d)).to(wt)
    s["scale"] = 0.5 if case["res"] else 1.0
    s["h"] = randn(t, d).to(bf) if case["res"] else None
    s["w_post"] = (1.0 + 0.1 * randn(d)).to(wt) if case["post"] else None
    s["gate"] = (1.0 + 0.3 * randn(*_gate_shape(case))).to(bf) if case["gate"] != "none" else None
    s["codes"] = _code_buffers(t, d, case["layout"])
    if op == "norm":
        s["y"] = torch.zeros(t, d, dtype=bf, device="cuda") if case["res"] else None
        return s
    # the backward pass finds what the forward pass kept: the residual stream and the two norms' factors
    del s["x"]
    s["y"] = x.to(bf)
    s["rstd"] = torch.rsqrt(s["y"].double().square().mean(1) + EPS).float()
    s["rstd_post"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float() if case["post"] else None
    s["dn"] = (randn(t, d) * 1e-3).to(bf)
    s["dy"] = (randn(t, d) * 1e-3).to(bf)
    s["dx"] = torch.zeros(t, d, dtype=bf, device="cuda")
    if not case["res"]:
        s["codes"] = None
    return s


# ------------------------------------------------------------------ plain forms


def _blocked(b):
    """[rows, groups] scale bytes -> the blocked layout: chunks of 128 rows x 4 groups, padding rows 127, padding groups 0."""
    rows, groups = b.shape
    rp, gp = (rows + 127) // 128 * 128, (groups + 3) // 4 * 4
    full = torch.zeros(rp, gp, dtype=torch.uint8, device=b.device)
    full[:, :groups] = 127
    full[:rows, :groups] = b
    return full.view(rp // 128, 4, 32, gp // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _group_codes(v):
    """Codes and scale bytes of v [rows, groups * 128] (float32 holding BF16 values), one scale for each 128 in a row."""
    rows, cols = v.shape
    g = v.view(rows, cols // 128, 128)
    amax = g.abs().amax(2)
    f, p = torch.frexp(amax)
    e = torch.where(f <= 0.875, p - 9, p - 8).clamp(min=-127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    q = torch.ldexp(g, -e.unsqueeze(2)).to(torch.float8_e4m3fn)
    return q.view(rows, cols), (e + 127).to(torch.uint8)


def _codes(v, layout):
    """The quantised forms of v [rows, cols], rounded to BF16 first: the FP8 path's activations are BF16 tensors."""
    v = v.to(torch.bfloat16).float()
    rows, cols = v.shape
    q, s = _group_codes(v)
    out = {"q": q, "s": _blocked(s).view(torch.float8_e8m0fnu)}
    if layout == "both":
        vt = torch.zeros(cols, (rows + 127) // 128 * 128, device=v.device)
        vt[:, :rows] = v.t()
        qt, st = _group_codes(vt)
        out["qt"] = qt[:, :(rows + 15) // 16 * 16].contiguous()
        out["st"] = _blocked(st).view(torch.float8_e8m0fnu)
    return out


def _plain_norm(s):
    x, h, out = s["x"].float(), s["h"], {}
    if h is not None:
        hn = h.float()
        if s["w_post"] is not None:
            out["rstd_post"] = torch.rsqrt(hn.square().mean(1) + EPS)
            hn = hn * out["rstd_post"].unsqueeze(1) * s["w_post"].float()
        if s["gate"] is not None:
            hn = hn * s["gate"].float()
        y = (x + s["scale"] * hn).to(torch.bfloat16)
        out["y"] = y
        x = y.float()
    out["rstd"] = torch.rsqrt(x.square().mean(1) + EPS)
    return {**out, **_codes(x * out["rstd"].unsqueeze(1) * s["w_pre"].float(), s["case"]["layout"])}


def _plain_norm_bwd(s):
    y, dn, w = s["y"].float(), s["dn"].float(), s["w_pre"].float()
    r = s["rstd"].unsqueeze(1)
    nh = y * r
    tt = dn * w
    g = s["dy"].float() + r * (tt - nh * (tt * nh).mean(1, keepdim=True))
    out = {"dx": g.to(torch.bfloat16), "dw_pre": (dn * nh).sum(0)}
    if s["h"] is None:
        return out
    hh = s["h"].float()
    if s["w_post"] is not None:
        rp = s["rstd_post"].unsqueeze(1)
        hh = hh * rp
    hn = hh * s["w_post"].float() if s["w_post"] is not None else hh
    u = s["scale"] * g
    if s["gate"] is not None:
        kind = s["case"]["gate"]
        dg = u * hn
        out["dgate"] = dg.sum(1, keepdim=True) if kind == "token" else dg.sum(0, keepdim=True) if kind == "channel" else dg.to(torch.bfloat16)
        u = u * s["gate"].float()
    if s["w_post"] is not None:
        out["dw_post"] = (u * hh).sum(0)
        v = u * s["w_post"].float()
        u = rp * (v - hh * (v * hh).mean(1, keepdim=True))
    return {**out, **_codes(u, s["case"]["layout"])}


def _plain_swiglu(s):
    f = s["case"]["f"]
    g, u = s["gu"][:, :f].float(), s["gu"][:, f:].float()
    return _codes(g / (1.0 + torch.exp(-g)) * u, s["case"]["layout"])


def _plain_swiglu_bwd(s):
    f = s["case"]["f"]
    g, u, da = s["gu"][:, :f].float(), s["gu"][:, f:].float(), s["da"].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    return _codes(torch.cat([da * u * sg * (1.0 + g * (1.0 - sg)), da * g * sg], 1), s["case"]["layout"])


def _plain_ortho(s):
    x = s["grad"].float()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (torch.sqrt(x.square().sum()) + NS_EPS)
    a, b, c = NS
    for _ in range(NS_STEPS):
        m = x @ x.t()
        x = a * x + (b * m + c * (m @ m)) @ x
    return {"out": (x.t() if tall else x).to(torch.bfloat16).contiguous()}


# ------------------------------------------------------------------ the framework's calls


def _quant_act(fp8, c, rows, cols):
    return fp8.QuantAct(rows, cols, q=c["q"], s=c["s"], qt=c.get("qt"), st=c.get("st"))


def _views(qa):
    out = {"q": qa.q.view(torch.float8_e4m3fn), "s": qa.s.view(torch.float8_e8m0fnu)}
    if qa.qt is not None:
        out["qt"] = qa.qt.view(torch.float8_e4m3fn)
        out["st"] = qa.st.view(torch.float8_e8m0fnu)
    return out


def _own(s):
    import fp8_block_scaled_13_b200 as fp8
    case = s["case"]
    op = case["op"]
    if op == "ortho":
        return {"out": fp8.orthogonalize(s["grad"], steps=NS_STEPS, coefficients=NS, eps=NS_EPS, out=s["out"])}
    if op == "swiglu":
        return _views(fp8.swiglu(s["gu"], layout=case["layout"], out=_quant_act(fp8, s["codes"], case["t"], case["f"])))
    if op == "swiglu_bwd":
        return _views(fp8.swiglu_backward(s["da"], s["gu"], layout=case["layout"],
                                          out=_quant_act(fp8, s["codes"], case["t"], 2 * case["f"])))
    block = dict(w_post=s["w_post"], gate=s["gate"], scale=s["scale"], layout=case["layout"])
    if op == "norm":
        r = fp8.residual_norm(s["x"], s["w_pre"], s["h"], eps=EPS, y=s["y"],
                              out=_quant_act(fp8, s["codes"], case["t"], case["d"]), **block)
        out = {"rstd": r.rstd, **_views(r.n)}
        if s["h"] is not None:
            out["y"] = r.y
        if r.rstd_post is not None:
            out["rstd_post"] = r.rstd_post
        return out
    r = fp8.residual_norm_backward(s["dn"], s["y"], s["rstd"], s["w_pre"], s["h"], dy=s["dy"], rstd_post=s["rstd_post"],
                                   dx=s["dx"], out=None if s["h"] is None else _quant_act(fp8, s["codes"], case["t"], case["d"]),
                                   **block)
    out = {"dx": r.dx, "dw_pre": r.dw_pre}
    if s["h"] is not None:
        out.update(_views(r.dh))
    if r.dw_post is not None:
        out["dw_post"] = r.dw_post
    if r.dgate is not None:
        out["dgate"] = r.dgate
    return out


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "swiglu": _plain_swiglu, "swiglu_bwd": _plain_swiglu_bwd,
            "ortho": _plain_ortho}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without


def _code_bytes(t, d, layout):
    return t * d * (1 + 1 / 128) * (2 if layout == "both" else 1)


def work(case):
    op = case["op"]
    if op == "ortho":
        n, k = case["n"], case["k"]
        m, w = min(n, k), max(n, k)
        # the Gram matrix and its square are symmetric: half of their products
        return {"bytes": n * k * ((4 if case["g32"] else 2) + 2), "flops": NS_STEPS * (m * m * w + m * m * m + 2 * m * m * w)}
    t = case["t"]
    if op == "swiglu":
        f = case["f"]
        return {"bytes": t * f * 4 + _code_bytes(t, f, case["layout"]), "flops": 6 * t * f}
    if op == "swiglu_bwd":
        f = case["f"]
        return {"bytes": t * f * 6 + _code_bytes(t, 2 * f, case["layout"]), "flops": 14 * t * f}
    d = case["d"]
    e, wb = t * d, 4 if case["w32"] else 2
    gate = {"none": 0, "token": 2 * t, "channel": 2 * d, "full": 2 * e}[case["gate"]]
    params = d * wb * (2 if case["post"] else 1)
    factors = 4 * t * (2 if case["post"] else 1)
    if op == "norm":
        return {"bytes": 2 * e * (3 if case["res"] else 1) + gate + params + factors + _code_bytes(t, d, case["layout"]), "flops": 10 * e}
    read = 2 * e * (4 if case["res"] else 3) + gate + params + factors
    written = 2 * e + (_code_bytes(t, d, case["layout"]) if case["res"] else 0) + (2 * gate if case["gate"] != "full" else gate) + 4 * d * (2 if case["post"] else 1)
    return {"bytes": read + written, "flops": 25 * e}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_codes(v, layout):
    """What the codes stand for, before their rounding: v times the reciprocal of its group's scale.  The scales follow
    from BF16 values and have no value of their own in 64 bits."""
    rows, cols = v.shape

    def scaled(m, valid):
        big = m.to(torch.bfloat16).double().abs().view(m.shape[0], -1, 128).amax(2).clamp(min=2.0 ** -140)
        e = torch.ceil(torch.log2(big / 448.0) - 1e-6).clamp(min=-127)  # the next BF16 value is 0.006 or more away
        e = torch.where(big > 2.0 ** -140, e, torch.zeros_like(e))
        return (m.view(m.shape[0], -1, 128) / torch.exp2(e).unsqueeze(2)).view(m.shape)[:, :valid].contiguous()

    out = {"q": scaled(v, cols), "s": None}
    if layout == "both":
        vt = torch.nn.functional.pad(v.t(), (0, -rows % 128)).contiguous()
        out["qt"] = scaled(vt, (rows + 15) // 16 * 16)
        out["st"] = None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ortho":
        x = s["grad"].double()
        x = x / (torch.linalg.vector_norm(x) + NS_EPS)
        wide = x.shape[0] <= x.shape[1]
        for _ in range(NS_STEPS):
            # sum of odd powers, without the polynomial of the Gram matrix: X, (X X^T) X, (X X^T)^2 X
            m = x @ x.mT if wide else x.mT @ x
            once = m @ x if wide else x @ m
            twice = m @ once if wide else once @ m
            x = NS[0] * x + NS[1] * once + NS[2] * twice
        return {"out": x}
    if op in ("swiglu", "swiglu_bwd"):
        gu = s["gu"].double().requires_grad_(op == "swiglu_bwd")
        g, u = gu.chunk(2, 1)
        a = g * torch.sigmoid(g) * u
        if op == "swiglu":
            return _exact_codes(a, case["layout"])
        a.backward(s["da"].double())
        return _exact_codes(gu.grad, case["layout"])
    leaf = lambda v: None if v is None else v.double().requires_grad_(op == "norm_bwd")  # noqa: E731
    h, gate, w_pre, w_post = leaf(s["h"]), leaf(s["gate"]), leaf(s["w_pre"]), leaf(s["w_post"])
    out, branch = {}, 0.0
    if h is not None:
        branch = h
        if w_post is not None:
            rp = (h.square().mean(1) + EPS) ** -0.5
            out["rstd_post"] = rp
            branch = branch * rp.unsqueeze(1) * w_post
        if gate is not None:
            branch = branch * gate
        branch = s["scale"] * branch
    if op == "norm":
        y = s["x"].double() + branch
        if h is not None:
            out["y"] = y
            y = y.to(torch.bfloat16).double()
        out["rstd"] = (y.square().mean(1) + EPS) ** -0.5
        return {**out, **_exact_codes(y * out["rstd"].unsqueeze(1) * w_pre, case["layout"])}
    x = (s["y"].double() - (branch.detach() if h is not None else 0.0)).requires_grad_(True)
    y = x + branch
    n = y * ((y.square().mean(1, keepdim=True) + EPS) ** -0.5) * w_pre
    torch.autograd.backward([n, y], [s["dn"].double(), s["dy"].double()])
    out = {"dx": x.grad, "dw_pre": w_pre.grad}
    if h is None:
        return out
    if w_post is not None:
        out["dw_post"] = w_post.grad
    if gate is not None:
        out["dgate"] = gate.grad
    return {**out, **_exact_codes(h.grad, case["layout"])}
