"""Measured cases of the layer operators: the fused linear layer, its backward and the mixture-of-experts layer.

Every operator multiplies by packed ternary (or binary) weights w = s * t, one fp16 scale s per 128
weights along K. `run` computes it either in plain form (torch: unpack, fp32 products, activation,
residual, one rounding at the end) or, with `own`, through the package's entry points.

    linear    y = act(W x + b) (+ residual);  gated: y = act(z[:n/2]) * z[n/2:] (+ residual)
    backward  dz = dy * act'(z), db = sum_m dz, dx = dz W
    moe       y[t] = sum_j p[t,j] D_e (act(G_e x[t]) * U_e x[t]) (+ residual), e = ids[t,j], the top_k
              experts of softmax(R x[t]), p renormalised over the chosen ones
"""
import math

import torch

own = False

Q2, T3, Q1 = 1, 2, 3  # 2-bit codes; base-3, five trits a byte; binary, eight signs a byte
LAYOUT = {"q2": Q2, "t3": T3, "q1": Q1}
GROUP = 128


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # attention output projection of an 8B-class layer, one token, added to the residual stream
        {"name": "proj_1", "op": "linear", "layout": "q2", "m": 1, "n": 4096, "k": 4096, "act": "none", "gated": False,
         "bias": False, "residual": True, "preact": False},
        # fused gate/up of the same layer, one token, dense base-3 weights
        {"name": "gate_up_t3_1", "op": "linear", "layout": "t3", "m": 1, "n": 24576, "k": 4096, "act": "silu", "gated": True,
         "bias": False, "residual": False, "preact": False},
        # down projection for a handful of sequences decoded together
        {"name": "down_5", "op": "linear", "layout": "q2", "m": 5, "n": 4096, "k": 12288, "act": "none", "gated": False,
         "bias": True, "residual": True, "preact": False},
        # a plain two-matrix block's first half on binary weights: odd width, odd batch, bias and gelu
        {"name": "fc_q1_13", "op": "linear", "layout": "q1", "m": 13, "n": 5001, "k": 2176, "act": "gelu", "gated": False,
         "bias": True, "residual": False, "preact": False},
        # prompt of 512 tokens through a 27B-class fused gate/up
        {"name": "gate_up_512", "op": "linear", "layout": "q2", "m": 512, "n": 34816, "k": 5120, "act": "silu", "gated": True,
         "bias": False, "residual": False, "preact": False},
        # ragged prompt through the 27B-class down projection, base-3, with the residual
        {"name": "down_t3_1999", "op": "linear", "layout": "t3", "m": 1999, "n": 5120, "k": 17408, "act": "none", "gated": False,
         "bias": False, "residual": True, "preact": False},
        # training step of a small layer on a short sequence, base-3 latents re-packed each step
        {"name": "train_t3_77", "op": "backward", "layout": "t3", "m": 77, "n": 2560, "k": 1024, "act": "gelu_tanh", "gated": False},
        # training step of the 8B-class fused gate/up over a 2048-token batch
        {"name": "train_q2_2048", "op": "backward", "layout": "q2", "m": 2048, "n": 24576, "k": 4096, "act": "silu", "gated": True},
        # one token through 64 small experts, eight of them chosen
        {"name": "moe_1", "op": "moe", "layout": "q2", "m": 1, "d": 2048, "f": 1024, "experts": 64, "top_k": 8, "act": "silu",
         "renorm": True, "residual": True},
        # a decode batch over many small experts: about one token for each expert
        {"name": "moe_t3_16", "op": "moe", "layout": "t3", "m": 16, "d": 2048, "f": 768, "experts": 128, "top_k": 8, "act": "silu",
         "renorm": True, "residual": False},
        # the largest decode batch over a few wide experts, all of them in use
        {"name": "moe_64", "op": "moe", "layout": "q2", "m": 64, "d": 4096, "f": 12288, "experts": 8, "top_k": 2, "act": "silu",
         "renorm": True, "residual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "moe"])
    layout = rng.choice(["q2", "t3", "q1"])
    if op == "moe":
        while True:
            experts = rng.choice([4, 8, 16, 40, 64, 128, 160])
            d, f = GROUP * _log(rng, 2, 32), GROUP * _log(rng, 1, 96)
            if 3 * experts * d * f <= 3 * 8 * 4096 * 12288:
                break
        return {"op": op, "layout": layout, "m": _log(rng, 1, 64), "d": d, "f": f, "experts": experts,
                "top_k": rng.randint(1, min(8, experts)), "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu2"]),
                "renorm": rng.random() < 0.5, "residual": rng.random() < 0.5}
    while True:
        m = _log(rng, 1, 2048)
        n, k = _log(rng, 64, 34816), GROUP * _log(rng, 1, 136)
        if m * n * k <= 1999 * 5120 * 17408:
            break
    gated = rng.random() < 0.5
    n += n % 2 if gated else 0
    case = {"op": op, "layout": layout, "m": m, "n": n, "k": k, "gated": gated,
            "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu", "relu2"] if gated else ["none", "silu", "gelu", "gelu_tanh", "relu", "relu2"])}
    if op == "linear":
        case.update(bias=rng.random() < 0.5, residual=rng.random() < 0.5, preact=rng.random() < 0.3)
    return case


# ----------------------------------------------------------------------------------------- inputs
def _row_bytes(layout, k):
    b = {Q2: k // 4, T3: (k + 4) // 5, Q1: k // 8}[layout]
    return (b + 15) // 16 * 16


def _table(layout, device):
    """Packed byte of each 4- or 5-digit decimal number: digits 0-3 are t = 0, 4-6 t = +1, 7-9 t = -1."""
    digits = 4 if layout == Q2 else 5
    v = torch.arange(10 ** digits, device=device)
    byte = torch.zeros_like(v)
    for i in range(digits):
        d = v // 10 ** i % 10
        t = torch.where(d < 4, 0, torch.where(d < 7, 1, -1))
        byte += (t & 3) << (2 * i) if layout == Q2 else (t + 1) * 3 ** i
    return byte.to(torch.uint8)


def _weights(layout, n, k, g):
    """Packed codes (P(0) = 0.4, P(+1) = P(-1) = 0.3; binary: 1/2 each) and scales fp16(|N(0,1)| * 0.02)."""
    rb, dev = _row_bytes(layout, k), g.device
    codes = torch.empty(n, rb, dtype=torch.uint8, device=dev)
    if layout == Q1:
        codes.random_(0, 256, generator=g)
        codes[:, k // 8:] = 0
    else:
        table = _table(layout, dev)
        rows = max(1, (1 << 26) // rb)
        for r in range(0, n, rows):
            part = codes[r:r + rows]
            part.copy_(table[torch.randint(0, table.numel(), part.shape, generator=g, device=dev, dtype=torch.int32)])
        if layout == T3:
            full, rest = divmod(k, 5)
            if rest:
                last = codes[:, full].int()
                codes[:, full] = (last % 3 ** rest + sum(3 ** i for i in range(rest, 5))).to(torch.uint8)
            codes[:, (k + 4) // 5:] = 121
    stride = (k // GROUP + 7) // 8 * 8  # rows of scales are 16-byte aligned
    scales = torch.zeros(n, stride, dtype=torch.float16, device=dev)
    scales[:, :k // GROUP] = (torch.randn(n, k // GROUP, generator=g, device=dev).abs() * 0.02).half()
    return {"layout": layout, "n": n, "k": k, "codes": codes, "scales": scales}


def _activations(m, k, g):
    """N(0,1) with a few channels ten times as large, as a residual stream has."""
    x = torch.randn(m, k, generator=g, device=g.device)
    x[:, torch.randint(0, k, (max(1, k // 512),), generator=g, device=g.device)] *= 10
    return x.half()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    layout, m = LAYOUT[case["layout"]], case["m"]
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    st = {"case": case}
    if case["op"] == "moe":
        d, f, e = case["d"], case["f"], case["experts"]
        st["gate_up"], st["down"] = _weights(layout, e * 2 * f, d, g), _weights(layout, e * d, f, g)
        st["router"] = (rand(e, d) * (1.5 / math.sqrt(d))).half()
        st["x"] = rand(m, d).half()
        st["residual"] = rand(m, d).half() if case["residual"] else None
        return st
    n, k = case["n"], case["k"]
    out = n // 2 if case["gated"] else n
    st["W"] = _weights(layout, n, k, g)
    if case["op"] == "linear":
        st["x"] = _activations(m, k, g)
        st["bias"] = (rand(n) * 0.5).half() if case["bias"] else None
        st["residual"] = rand(m, out).half() if case["residual"] else None
    else:
        st["preact"] = rand(m, n).half()
        st["dy"] = rand(m, out).half()
    return st


# ------------------------------------------------------------------------------------- plain form
def _unpack(layout, codes, scales, k):
    """fp32 [..., k] = s * t of packed rows."""
    c = codes[..., :(k * {Q2: 2, T3: 8, Q1: 1}[layout] + (39 if layout == T3 else 7)) // (40 if layout == T3 else 8)]
    if layout == Q2:
        t = (c[..., None] >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=c.device)) & 3
        t = t.to(torch.int8)
        t = t - 4 * (t == 3).to(torch.int8)
    elif layout == T3:
        t = c[..., None] // torch.tensor([1, 3, 9, 27, 81], dtype=torch.uint8, device=c.device) % 3
        t = t.to(torch.int8) - 1
    else:
        t = (c[..., None] >> torch.arange(8, dtype=torch.uint8, device=c.device)) & 1
        t = 2 * t.to(torch.int8) - 1
    t = t.flatten(-2)[..., :k].unflatten(-1, (k // GROUP, GROUP))
    return (t.float() * scales[..., :k // GROUP, None].float()).flatten(-2)


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp_min(0)
    if name == "relu2":
        return z.clamp_min(0) ** 2
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def _act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "relu2":
        return 2 * z.clamp_min(0)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


def _plain_linear(st):
    c, W = st["case"], st["W"]
    z = st["x"].float() @ _unpack(W["layout"], W["codes"], W["scales"], W["k"]).T
    if st["bias"] is not None:
        z = z + st["bias"].float()
    if c["gated"]:
        gate, up = z.chunk(2, dim=1)
        y = _act(c["act"], gate) * up
    else:
        y = _act(c["act"], z)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    out = {"y": y.half()}
    if c["preact"]:
        out["z"] = z.half()
    return out


def _plain_backward(st):
    c, W = st["case"], st["W"]
    z, dy = st["preact"].float(), st["dy"].float()
    if c["gated"]:
        gate, up = z.chunk(2, dim=1)
        dz = torch.cat([dy * up * _act_grad(c["act"], gate), dy * _act(c["act"], gate)], dim=1)
    else:
        dz = dy * _act_grad(c["act"], z)
    dx = dz @ _unpack(W["layout"], W["codes"], W["scales"], W["k"])
    return {"dx": dx.half(), "dz": dz.half(), "db": dz.sum(0)}


def _plain_moe(st):
    c, G, D = st["case"], st["gate_up"], st["down"]
    d, f, e, k = c["d"], c["f"], c["experts"], c["top_k"]
    x = st["x"].float()
    logits = st["x"].double() @ st["router"].double().T
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    top, ids = torch.sort(p, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    if c["renorm"]:
        top = top / top.sum(1, keepdim=True)
    top = top.float()
    gc, gs = G["codes"].unflatten(0, (e, 2 * f)), G["scales"].unflatten(0, (e, 2 * f))
    dc, ds = D["codes"].unflatten(0, (e, d)), D["scales"].unflatten(0, (e, d))
    if x.shape[0] * k <= e:  # the chosen experts' weights, token by token
        flat = ids.flatten()
        h = torch.einsum("td,tkfd->tkf", x, _unpack(G["layout"], gc[flat], gs[flat], d).unflatten(0, (-1, k)))
        h = _act(c["act"], h[..., :f]) * h[..., f:]
        y = torch.einsum("tk,tkf,tkdf->td", top, h, _unpack(D["layout"], dc[flat], ds[flat], f).unflatten(0, (-1, k)))
    else:  # every expert on every token, weighted by what the router gave it
        w = torch.zeros_like(logits, dtype=torch.float32).scatter(1, ids, top)
        h = torch.matmul(x, _unpack(G["layout"], gc, gs, d).transpose(1, 2))
        h = _act(c["act"], h[..., :f]) * h[..., f:] * w.T[:, :, None]
        y = torch.matmul(h, _unpack(D["layout"], dc, ds, f).transpose(1, 2)).sum(0)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return {"y": y.half(), "weights": top, "ids": ids.int()}


# --------------------------------------------------------------------------------- the operators
def _matrix(T, w):
    return T.TernMatrix(w["layout"], w["n"], w["k"], w["codes"], w["scales"])


def run(st):
    c = st["case"]
    if not own:
        return {"linear": _plain_linear, "backward": _plain_backward, "moe": _plain_moe}[c["op"]](st)
    import gemm_tern_gemv_b200 as T

    if c["op"] == "linear":
        z = torch.empty(c["m"], c["n"], dtype=torch.float16, device="cuda") if c["preact"] else None
        y = T.linear(_matrix(T, st["W"]), st["x"], bias=st["bias"], act=c["act"], gated=c["gated"], residual=st["residual"],
                     preact=z)
        return {"y": y, "z": z} if c["preact"] else {"y": y}
    if c["op"] == "backward":
        dx, dz, db = T.linear_backward(_matrix(T, st["W"]), st["dy"], st["preact"], act=c["act"], gated=c["gated"])
        return {"dx": dx, "dz": dz, "db": db}
    y, weights, ids = T.moe(_matrix(T, st["gate_up"]), _matrix(T, st["down"]), st["router"], st["x"], c["top_k"], act=c["act"],
                            renormalize=c["renorm"], residual=st["residual"], return_routing=True)
    return {"y": y, "weights": weights, "ids": ids}


# -------------------------------------------------------------------------------------- the work
def _packed(layout, n, k):
    return n * (_row_bytes(layout, k) + 2 * (k // GROUP))


def work(case):
    layout, m = LAYOUT[case["layout"]], case["m"]
    if case["op"] == "moe":
        d, f, e, k = case["d"], case["f"], case["experts"], case["top_k"]
        active = e * (1 - (1 - k / e) ** m)  # experts with a token, for routing without preference
        b = active * (_packed(layout, 2 * f, d) + _packed(layout, d, f)) + 2 * e * d
        return {"bytes": b + 2 * m * d * (3 if case["residual"] else 2) + 8 * m * k, "flops": 2.0 * m * (k * 3 * d * f + e * d)}
    n, k = case["n"], case["k"]
    out = n // 2 if case["gated"] else n
    b = _packed(layout, n, k)
    if case["op"] == "linear":
        b += 2 * m * k + 2 * m * out * (2 if case["residual"] else 1) + (2 * n if case["bias"] else 0) + (2 * m * n if case["preact"] else 0)
    else:
        b += 2 * m * out + 2 * m * n * 2 + 4 * n + 2 * m * k
    return {"bytes": b, "flops": 2.0 * m * n * k}


# ------------------------------------------------------------------------- definition in 64 bits
def _dense64(w, rows):
    """fp64 weights of some rows, from the layouts' definitions: code value times its group's scale."""
    layout, k, codes = w["layout"], w["k"], w["codes"][rows]
    j = torch.arange(k, device=codes.device)
    if layout == Q2:
        field = torch.bitwise_right_shift(codes[:, j // 4].int(), (2 * (j % 4)).int()) % 4
        t = torch.tensor([0.0, 1.0, math.nan, -1.0], dtype=torch.float64, device=codes.device)[field]
    elif layout == T3:
        power = torch.tensor([1, 3, 9, 27, 81], device=codes.device)[j % 5]
        t = torch.div(codes[:, j // 5].long(), power, rounding_mode="floor").remainder(3).double() - 1
    else:
        bit = torch.bitwise_right_shift(codes[:, j // 8].int(), (j % 8).int()) % 2
        t = torch.where(bit == 1, 1.0, -1.0).double()
    return t.mul_(w["scales"][rows].double()[:, j // GROUP])


def _product64(w, x, transposed=False, lo=0, hi=None):
    """x W^T (or x W) in fp64 over rows lo..hi of w, some rows of W at a time."""
    hi = w["n"] if hi is None else hi
    step = max(1, (1 << 25) // w["k"])
    starts = range(lo, hi, step)
    if transposed:
        total = torch.zeros(x.shape[0], w["k"], dtype=torch.float64, device=x.device)
        for r in starts:
            total += x[:, r - lo:min(r + step, hi) - lo] @ _dense64(w, slice(r, min(r + step, hi)))
        return total
    return torch.cat([x @ _dense64(w, slice(r, min(r + step, hi))).T for r in starts], 1)


def _phi64(act, z):
    """act and its derivative in fp64."""
    n01 = torch.distributions.Normal(torch.zeros((), dtype=torch.float64, device=z.device), 1.0, validate_args=False)
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.relu(z), torch.heaviside(z, torch.zeros_like(z))
    if act == "relu2":
        return torch.relu(z).square(), 2 * torch.relu(z)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if act == "gelu":
        return z * torch.special.ndtr(z), torch.special.ndtr(z) + z * n01.log_prob(z).exp()
    u = math.sqrt(8 / math.pi) * (z + 0.044715 * z * z * z)  # (1 + tanh(u/2)) / 2 = sigmoid(u)
    s = torch.sigmoid(u)
    return z * s, s + z * s * torch.sigmoid(-u) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z * z)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "moe":
        d, f, e, k, m = case["d"], case["f"], case["experts"], case["top_k"], case["m"]
        x = st["x"].double()
        p = torch.softmax(x @ st["router"].double().T, 1)
        # rank of each expert in its row, ties to the lower index
        higher = (p[:, None, :] > p[:, :, None]) | ((p[:, None, :] == p[:, :, None]) & (torch.arange(e, device=x.device) < torch.arange(e, device=x.device)[:, None]))
        rank = higher.sum(2)
        ids = rank.argsort(1)[:, :k]
        weights = p.gather(1, ids)
        if case["renorm"]:
            weights = weights / weights.sum(1, keepdim=True)
        y = st["residual"].double() if case["residual"] else torch.zeros(m, d, dtype=torch.float64, device=x.device)
        for ex in ids.unique().tolist():
            t, j = (ids == ex).nonzero(as_tuple=True)
            z = _product64(st["gate_up"], x[t], lo=ex * 2 * f, hi=(ex + 1) * 2 * f)
            h = _phi64(case["act"], z[:, :f])[0] * z[:, f:]
            y.index_add_(0, t, _product64(st["down"], h, lo=ex * d, hi=(ex + 1) * d) * weights[t, j][:, None])
        return {"y": y, "weights": weights, "ids": ids.int()}
    n = case["n"]
    if case["op"] == "linear":
        z = _product64(st["W"], st["x"].double())
        z = z if st["bias"] is None else z + st["bias"].double()
        y = _phi64(case["act"], z[:, :n // 2])[0] * z[:, n // 2:] if case["gated"] else _phi64(case["act"], z)[0]
        y = y if st["residual"] is None else y + st["residual"].double()
        return {"y": y, "z": z} if case["preact"] else {"y": y}
    z, dy = st["preact"].double(), st["dy"].double()
    if case["gated"]:
        a, da = _phi64(case["act"], z[:, :n // 2])
        dz = torch.cat([dy * z[:, n // 2:] * da, dy * a], 1)
    else:
        dz = dy * _phi64(case["act"], z)[1]
    return {"dx": _product64(st["W"], dz, transposed=True), "dz": dz, "db": dz.sum(0)}
