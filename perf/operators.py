"""Cases of the 4-bit expert products and of the router's gradients, with plain forms.

Four operators of the routed MoE FFN layer: the layer over 4-bit expert weights
with group scales (`q4_layer`), the balance loss with per-expert counts and
the gradient of the router logits (`balance`), the gradient of the routing
weights (`finalize_backward`) and the gradient of the router's weight and bias
(`router_weight_grad`).

With `own` false, `run` computes them with elementary torch operations in 32
bits (the router in 64, as the layer defines it); with `own` true it calls the
library.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# nibble position -> element of an 8-element word, by format
NIBBLES = {"int4": (0, 2, 4, 6, 1, 3, 5, 7), "e2m1": (0, 1, 2, 3, 4, 5, 6, 7)}


# ---------------------------------------------------------------- cases

def _q4(name, T, H, E, k, Im, mu, dtype, fmt, group, renorm=True, bias=False):
    c = dict(kind="q4_layer", T=T, H=H, E=E, k=k, Im=Im, mu=mu, dtype=dtype, fmt=fmt, group=group, renorm=renorm, bias=bias)
    return dict(c, name=name) if name else c


def _balance(name, T, E, k, renorm, mask, d_w=True):
    c = dict(kind="balance", T=T, E=E, k=k, renorm=renorm, mask=mask, d_w=d_w)
    return dict(c, name=name) if name else c


def _finalize(name, T, H, k, dtype):
    c = dict(kind="finalize_backward", T=T, H=H, k=k, dtype=dtype)
    return dict(c, name=name) if name else c


def _wgrad(name, T, H, E, dtype, mask):
    c = dict(kind="router_weight_grad", T=T, H=H, E=E, dtype=dtype, mask=mask)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence's next token: 8 active experts, latency counts
        _q4("q4 one token", 1, 4096, 64, 8, 768, 1, "bf16", "int4", 128),
        # the decode layer of the benchmark, its experts in 4 bits
        _q4("q4 decode", 8, 4096, 64, 8, 768, 1, "bf16", "int4", 128),
        # the same layer at the decode path's last token count, float codes, the finest scales
        _q4("q4 decode e2m1", 16, 4096, 64, 8, 768, 1, "bf16", "e2m1", 32),
        # many sequences' tokens in one call, both micro-shards
        _q4("q4 batch", 256, 4096, 64, 8, 768, 2, "bf16", "int4", 64, renorm=False, bias=True),
        # a small fp32 layer of odd sizes: rows and groups that end inside a tile
        _q4("q4 f32 odd", 37, 448, 7, 3, 160, 2, "f32", "int4", 32, bias=True),
        # a short batch with padding
        _balance("balance short", 37, 64, 8, True, "some"),
        # the denoise layer's tokens, padded batch
        _balance("balance", 4096, 64, 8, True, "some"),
        # a training batch of many sequences, routing weights not renormalised
        _balance("balance long", 65535, 64, 8, False, "none"),
        # the denoise layer's routes
        _finalize("weights gradient", 4096, 4096, 8, "bf16"),
        # a small fp32 layer
        _finalize("weights gradient f32", 333, 448, 3, "f32"),
        # the denoise layer's tokens
        _wgrad("router gradient", 4096, 4096, 64, "bf16", "none"),
        # a long padded batch
        _wgrad("router gradient long", 32767, 4096, 64, "bf16", "some"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("q4", "q4", "balance", "finalize", "wgrad"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    H = 64 * _log(rng, 1, 64)
    E = rng.randint(1, 64)
    k = rng.randint(1, min(E, 8))
    mask = rng.choice(("none", "some", "most"))
    if kind == "q4":
        # half the draws take the layer's own sizes at another token count, half any size of the envelope
        if rng.random() < 0.5:
            return _q4("", _log(rng, 1, 256), 4096, 64, 8, 768, 1, "bf16", rng.choice(("int4", "e2m1")), rng.choice((32, 64, 128)),
                       rng.random() < 0.7, rng.random() < 0.5)
        group = rng.choice((32, 32, 64, 128))
        H = max(1, H // group) * group if group > 64 else H
        Im = group * _log(rng, 1, 768 // group)
        return _q4("", _log(rng, 1, 256), H, E, k, Im, rng.randint(1, 2), dtype, rng.choice(("int4", "e2m1")), group,
                   rng.random() < 0.7, rng.random() < 0.5)
    if kind == "balance":
        E = max(E, 2)
        k = min(k, E - 1)  # with every expert chosen the loss has no gradient
        return _balance("", _log(rng, 1, 65535), E, k, rng.random() < 0.5, mask, rng.random() < 0.8)
    if kind == "finalize":
        return _finalize("", _log(rng, 1, 4096), H, k, dtype)
    return _wgrad("", _log(rng, 1, 32767 if dtype == "bf16" else 8191), H, E, dtype, mask)


# ---------------------------------------------------------------- inputs

def _gen(seed, tag):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 64 + tag)
    return g


def _randn(shape, g, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _raw_weights(case, seed, tag, rows, K):
    """Codes [mu, E, rows, K] uint8 and scales [mu, E, rows, K / group] of one weight: codes of normal values, scales around 0.02 / 3."""
    g = _gen(seed, tag)
    shape = (case["mu"], case["E"], rows, K)
    v = torch.randn(shape, generator=g, device=DEV)
    if case["fmt"] == "int4":
        codes = v.mul_(2.7).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
    else:
        mag = v.abs().mul_(3.0).floor_().clamp_(0, 7).to(torch.uint8)
        codes = mag + 8 * torch.randint(0, 2, shape, generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(shape[:3] + (K // case["group"],), generator=g, device=DEV) * 0.008 + 0.004
    return codes, s.to(_dtype(case))


def _pack(case, codes, scales, gate_up):
    """The library's storage: 1 KB tiles of 16 rows x 128 columns, and scales padded per row."""
    mu, E, N, K = codes.shape
    if gate_up:  # a tile's rows: 8 gate rows, then their 8 up rows
        codes = codes.view(mu, E, 2, N // 16, 8, K).transpose(2, 3).reshape(mu, E, N, K)
        scales = scales.view(mu, E, 2, N // 16, 8, -1).transpose(2, 3).reshape(mu, E, N, -1)
    KB = -(-K // 128)
    zero = 8 if case["fmt"] == "int4" else 0
    if KB * 128 > K:
        codes = torch.nn.functional.pad(codes, (0, KB * 128 - K), value=zero)
    t = codes.view(mu, E, N // 16, 16, KB, 4, 4, 8).permute(0, 1, 2, 4, 6, 3, 5, 7)  # ..., kb, lane / 16, lane % 16, word, element
    at = NIBBLES[case["fmt"]]
    packed = torch.stack([t[..., at[2 * b]] | (t[..., at[2 * b + 1]] << 4) for b in range(4)], dim=-1)
    G = scales.shape[-1]
    S = 4 * (-(-KB // 4)) * (128 // case["group"])
    scales = torch.nn.functional.pad(scales, (0, S - G)) if S > G else scales
    return packed.reshape(mu, E, N // 16, KB, 1024).contiguous(), scales.contiguous()


def _mask(case, seed):
    T = case["T"]
    if case["mask"] == "none":
        return None
    keep = {"some": 0.9, "most": 0.1}[case["mask"]]  # the share of valid tokens, at least one
    mask = (torch.rand(T, generator=_gen(seed, 20), device=DEV) < keep).to(torch.uint8)
    mask[T // 2] = 1
    return mask


def _q4_inputs(case, seed):
    T, H, E = case["T"], case["H"], case["E"]
    x = _randn((T, H), _gen(seed, 1), _dtype(case))
    wg = _randn((E, H), _gen(seed, 2), scale=1.5 / math.sqrt(H))
    bias = _randn((E,), _gen(seed, 3), scale=0.5) if case["bias"] else None
    return x, wg, bias


def _balance_inputs(case, seed):
    T, E, k = case["T"], case["E"], case["k"]
    logits = _randn((T, E), _gen(seed, 1), scale=1.3) + _randn((E,), _gen(seed, 2), scale=0.7)
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k].double(), ids[:, :k].to(torch.int32).contiguous()
    w = torch.softmax(top, 1) if case["renorm"] else torch.exp(top - torch.logsumexp(logits.double(), 1, keepdim=True))
    d_w = _randn((T, k), _gen(seed, 4), scale=1e-3) if case["d_w"] else None
    mask = _mask(case, seed)
    if mask is not None:  # padded rows hold anything
        pad = mask == 0
        logits[pad] = math.nan
        if d_w is not None:
            d_w[pad] = math.inf
    d_loss = torch.full((1,), 1e-2, device=DEV)
    return dict(logits=logits, ids=ids, w=w.float().contiguous(), mask=mask, d_w=d_w, d_loss=d_loss)


def _finalize_inputs(case, seed):
    T, H, k = case["T"], case["H"], case["k"]
    R = T * k
    inv = torch.randperm(R, generator=_gen(seed, 1), device=DEV).to(torch.int32)
    d_out = _randn((T, H), _gen(seed, 2), _dtype(case), scale=1e-2)
    y = _randn((R, H), _gen(seed, 3), scale=0.6)
    if case["dtype"] == "f32":
        return dict(y=y, inv=inv, d_out=d_out)
    # block-scaled half: per 256 columns one power of two that brings the largest value to [2^14, 2^15)
    B = -(-H // 256)
    amax = torch.nn.functional.pad(y, (0, B * 256 - H)).view(R, B, 256).abs().amax(-1)
    e = torch.frexp(amax)[1] - 15
    values = torch.ldexp(y, -e.repeat_interleave(256, 1)[:, :H]).to(torch.float16)
    buf = torch.cat([values.view(torch.uint8).reshape(-1), e.to(torch.int8).view(torch.uint8).reshape(-1)])
    return dict(y=buf, inv=inv, d_out=d_out)


def _wgrad_inputs(case, seed):
    T, H, E = case["T"], case["H"], case["E"]
    x = _randn((T, H), _gen(seed, 1), _dtype(case))
    d_logits = _randn((T, E), _gen(seed, 2), scale=1e-3)
    mask = _mask(case, seed)
    if mask is not None:
        pad = mask == 0
        x[pad] = math.nan
        d_logits[pad] = 0
    return dict(x=x, d_logits=d_logits, mask=mask)


def prepare(case, seed):
    state = {"case": dict(case)}
    kind = case["kind"]
    if kind == "q4_layer":
        x, wg, bias = _q4_inputs(case, seed)
        w1 = _pack(case, *_raw_weights(case, seed, 10, 2 * case["Im"], case["H"]), True)
        w2 = _pack(case, *_raw_weights(case, seed, 11, case["H"], case["Im"]), False)
        state.update(x=x, wg=wg, bias=bias, w1=w1, w2=w2)
    elif kind == "balance":
        state.update(_balance_inputs(case, seed))
    elif kind == "finalize_backward":
        state.update(_finalize_inputs(case, seed))
    else:
        state.update(_wgrad_inputs(case, seed))
    return state


# ---------------------------------------------------------------- plain forms

def _unpack(case, packed, scales, K):
    """fp32 weights [..., rows in tile order, K] of stored codes and scales."""
    lead, (NT, KB) = packed.shape[:-3], packed.shape[-3:-1]
    b = packed.view(lead + (NT, KB, 4, 16, 4, 4))
    nib = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)  # by nibble position
    at = torch.tensor([NIBBLES[case["fmt"]].index(i) for i in range(8)], device=nib.device)
    nib = nib[..., at]  # by element
    n = len(lead)
    nib = nib.permute(*range(n), n, n + 3, n + 1, n + 4, n + 2, n + 5).reshape(lead + (NT * 16, KB * 128))[..., :K]
    if case["fmt"] == "int4":
        v = nib.float() - 8.0
    else:
        table = torch.tensor(E2M1 + tuple(-e for e in E2M1), device=nib.device)
        v = table[nib.long()]
    G = K // case["group"]
    s = scales[..., :G].float()
    return (v.view(v.shape[:-1] + (G, case["group"])) * s[..., None]).flatten(-2)


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _plain_q4(state):
    case = state["case"]
    T, H, E, k, Im, mu = (case[n] for n in ("T", "H", "E", "k", "Im", "mu"))
    x, wg, bias = state["x"], state["wg"], state["bias"]
    logits = x.double() @ wg.double().T
    logits = (logits + bias.double() if bias is not None else logits).float()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k].double(), ids[:, :k]
    ex = torch.exp(top - top[:, :1])
    total = ex.sum(1, keepdim=True) if case["renorm"] else torch.exp(logits.double() - top[:, :1]).sum(1, keepdim=True)
    w = (ex / total).float()
    xf = x.float()
    (c1, s1), (c2, s2) = state["w1"], state["w2"]
    if T * k < E:  # the routed experts' weights, one copy a route
        e = ids.reshape(-1)
        g = torch.matmul(_unpack(case, c1[:, e], s1[:, e], H), xf.repeat_interleave(k, 0)[None, :, :, None])
        g = g.view(mu, T * k, Im // 8, 2, 8, 1)
        h = (_silu(g[:, :, :, 0]) * g[:, :, :, 1]).reshape(mu, T * k, Im, 1)
        y = torch.matmul(_unpack(case, c2[:, e], s2[:, e], Im), h).sum(0)  # [R, H, 1]
        out = (w[:, :, None] * y.view(T, k, H)).sum(1)
    else:  # every expert for every token, weighted
        g = torch.matmul(_unpack(case, c1, s1, H), xf.T.contiguous()).view(mu, E, Im // 8, 2, 8, T)
        h = (_silu(g[:, :, :, 0]) * g[:, :, :, 1]).reshape(mu, E, Im, T)
        y = torch.matmul(_unpack(case, c2, s2, Im), h).sum(0)  # [E, H, T]
        c = torch.zeros(T, E, device=x.device).scatter_(1, ids, w)
        out = (y * c.T[:, None, :]).sum(0).T
    return out.contiguous().to(x.dtype)


def _plain_balance(state):
    case = state["case"]
    T, E, k = case["T"], case["E"], case["k"]
    mask = state["mask"]
    ok = torch.ones(T, dtype=torch.bool, device=DEV) if mask is None else mask != 0
    logits = torch.where(ok[:, None], state["logits"], torch.zeros((), device=DEV))
    ids = state["ids"].long()
    ex = torch.exp(logits - logits.amax(1, keepdim=True))
    p = ex / ex.sum(1, keepdim=True) * ok[:, None]
    onehot = torch.zeros(T, E, device=DEV).scatter_(1, ids, 1.0) * ok[:, None]
    counts = onehot.double().sum(0)
    n = ok.double().sum().clamp(min=1.0)
    mean = p.double().sum(0) / n
    f = counts / (n * k)
    loss = (E * (f * mean).sum()).float().reshape(1)
    f = f.float()
    d = state["d_loss"] * (E / n).float() * p * (f - (p * f).sum(1, keepdim=True))
    if state["d_w"] is not None:
        d_w = torch.where(ok[:, None], state["d_w"], torch.zeros((), device=DEV))
        w = state["w"]
        dot = (w * d_w).sum(1, keepdim=True)
        if case["renorm"]:
            d = d + torch.zeros(T, E, device=DEV).scatter_(1, ids, w * (d_w - dot)) * ok[:, None]
        else:
            d = d + p * (torch.zeros(T, E, device=DEV).scatter_(1, ids, d_w) - dot)
    return dict(counts=counts.to(torch.int32), mean_prob=mean.float(), loss=loss, d_logits=d)


def _plain_finalize(state):
    case = state["case"]
    T, H, k = case["T"], case["H"], case["k"]
    R, y = T * k, state["y"]
    if case["dtype"] == "bf16":
        values = y[:R * H * 2].view(torch.float16).view(R, H)
        e = y[R * H * 2:].view(torch.int8).view(R, -1)
        y = values.float() * torch.exp2(e.float()).repeat_interleave(256, 1)[:, :H]
    return (y[state["inv"].long()].view(T, k, H) * state["d_out"].float()[:, None, :]).sum(-1)


def _plain_wgrad(state):
    x, d = state["x"].float(), state["d_logits"]
    if state["mask"] is not None:
        x = torch.where((state["mask"] != 0)[:, None], x, torch.zeros((), device=DEV))
    return dict(d_wg=d.T.contiguous() @ x, d_bias=d.sum(0))


# ---------------------------------------------------------------- the library's calls

def _own_q4(state):
    import mixture_experts_ffn_moe_amd as moe
    case = state["case"]
    if "buffers" not in state:  # what a serving program keeps: output and workspace
        shape = moe.make_shape(case["T"], case["H"], case["E"], case["k"], case["Im"], case["mu"], case["dtype"], case["renorm"])
        state["buffers"] = moe.MoELayerBuffers(shape)
        state["q4"] = moe.make_q4(case["fmt"], case["group"])
    return state["buffers"].forward_q4(state["q4"], state["x"], state["wg"], state["bias"], *state["w1"], *state["w2"])


def _own_balance(state):
    import mixture_experts_ffn_moe_amd as moe
    case = state["case"]
    T, E, k = case["T"], case["E"], case["k"]
    if "shape" not in state:
        state["shape"] = moe.make_shape(T, 64, E, k, 32, 1, "bf16", case["renorm"])
        state["workspace"] = torch.empty(moe.moe_balance_workspace_size(state["shape"]), dtype=torch.uint8, device=DEV)
    counts = torch.empty(E, dtype=torch.int32, device=DEV)
    mean, loss, d = torch.empty(E, device=DEV), torch.empty(1, device=DEV), torch.empty(T, E, device=DEV)
    s = state["shape"]
    moe.moe_balance_loss(s, state["logits"], state["ids"], state["mask"], counts, mean, loss, state["workspace"])
    moe.moe_route_backward(s, state["logits"], state["ids"], state["w"], state["mask"], counts, state["d_w"], state["d_loss"], d)
    return dict(counts=counts, mean_prob=mean, loss=loss, d_logits=d)


def _own_finalize(state):
    import mixture_experts_ffn_moe_amd as moe
    case = state["case"]
    if "shape" not in state:
        state["shape"] = moe.make_shape(case["T"], case["H"], max(case["k"], 8), case["k"], 32, 1, case["dtype"])
    d_w = torch.empty(case["T"], case["k"], device=DEV)
    moe.moe_finalize_backward(state["shape"], state["y"], state["inv"], state["d_out"], d_w)
    return d_w


def _own_wgrad(state):
    import mixture_experts_ffn_moe_amd as moe
    case = state["case"]
    T, H, E = case["T"], case["H"], case["E"]
    if "shape" not in state:
        state["shape"] = moe.make_shape(T, H, E, 1, 32, 1, case["dtype"])
        state["workspace"] = torch.empty(moe.moe_router_grad_workspace_size(state["shape"]), dtype=torch.uint8, device=DEV)
    d_wg, d_bias = torch.empty(E, H, device=DEV), torch.empty(E, device=DEV)
    moe.moe_router_weight_grad(state["shape"], state["x"], state["d_logits"], state["mask"], d_wg, d_bias, state["workspace"])
    return dict(d_wg=d_wg, d_bias=d_bias)


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"q4_layer": _own_q4, "balance": _own_balance, "finalize_backward": _own_finalize, "router_weight_grad": _own_wgrad}[kind](state)
    return {"q4_layer": _plain_q4, "balance": _plain_balance, "finalize_backward": _plain_finalize, "router_weight_grad": _plain_wgrad}[kind](state)


# ---------------------------------------------------------------- work and exact values

def work(case):
    T, kind = case["T"], case["kind"]
    size = 2 if case.get("dtype") == "bf16" else 4
    if kind == "q4_layer":
        H, E, k, I = case["H"], case["E"], case["k"], case["Im"] * case["mu"]
        active = E * (1.0 - (1.0 - k / E) ** T)  # experts that any token chose
        weights = active * 3 * I * H * (0.5 + size / case["group"])
        return {"bytes": weights + 2 * T * H * size + 4 * E * H, "flops": 6.0 * T * k * H * I + 2.0 * T * H * E}
    if kind == "balance":
        E, k = case["E"], case["k"]
        return {"bytes": 8.0 * T * E + 4 * T * k * (3 if case["d_w"] else 1) + (0 if case["mask"] == "none" else T) + 8 * E,
                "flops": 12.0 * T * E}
    if kind == "finalize_backward":
        H, R = case["H"], T * case["k"]
        y = R * H * 2 + R * (-(-H // 256)) if size == 2 else R * H * 4
        return {"bytes": float(y + T * H * size + 8 * R), "flops": 2.0 * R * H}
    H, E = case["H"], case["E"]
    return {"bytes": float(T * H * size + 4 * T * E + 4 * E * H + (0 if case["mask"] == "none" else T)), "flops": 2.0 * T * E * H}


def _exact_q4(case, seed):
    T, H, E, k, Im, mu, group = (case[n] for n in ("T", "H", "E", "k", "Im", "mu", "group"))
    x, wg, bias = _q4_inputs(case, seed)
    x64 = x.double()
    logits = torch.nn.functional.linear(x64, wg.double(), None if bias is None else bias.double()).float()  # the layer selects on 32 bits
    order = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    lg = logits.double()
    p = torch.softmax(lg, 1)
    weight = torch.gather(p, 1, order)
    if case["renorm"]:
        weight = weight / weight.sum(1, keepdim=True)

    def value(codes, scales):
        if case["fmt"] == "int4":
            v = codes.double() - 8
        else:
            m = (codes & 7).double()
            # a subnormal pair 0, 0.5, then (1 + mantissa / 2) 2^(exponent - 1)
            v = torch.where(m < 2, m * 0.5, (1 + (m % 2) * 0.5) * torch.exp2(torch.floor(m / 2) - 1))
            v = torch.where(codes >= 8, -v, v)
        return v * scales.double().repeat_interleave(group, -1)

    c1, s1 = _raw_weights(case, seed, 10, 2 * Im, H)
    c2, s2 = _raw_weights(case, seed, 11, H, Im)
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = torch.nonzero(order == e, as_tuple=True)
        if not len(t):
            continue
        y = 0
        for m in range(mu):
            a = x64[t] @ value(c1[m, e], s1[m, e]).T
            gate, up = a[:, :Im], a[:, Im:]
            y = y + (gate * torch.sigmoid(gate) * up) @ value(c2[m, e], s2[m, e]).T
        out[t] += weight[t, j][:, None] * y
    return out


def _exact_balance(case, seed):
    T, E, k = case["T"], case["E"], case["k"]
    s = _balance_inputs(case, seed)
    rows = torch.arange(T, device=DEV) if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
    n = len(rows)
    d = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    p = torch.softmax(s["logits"][rows].double(), 1)
    ids = s["ids"][rows].long()
    f = torch.bincount(ids.reshape(-1), minlength=E).double() / (n * k)
    mean = p.mean(0)
    d_p = float(s["d_loss"].double()) * E / n * f.expand(n, E)
    if s["d_w"] is not None and not case["renorm"]:
        d_p = d_p.scatter_add(1, ids, s["d_w"][rows].double())
    g = p * (d_p - (p * d_p).sum(1, keepdim=True))
    if s["d_w"] is not None and case["renorm"]:
        q = torch.gather(p, 1, ids)
        q = q / q.sum(1, keepdim=True)
        dw = s["d_w"][rows].double()
        g.scatter_add_(1, ids, q * (dw - (q * dw).sum(1, keepdim=True)))
    d[rows] = g
    return dict(counts=None, mean_prob=mean, loss=(E * (f * mean).sum()).reshape(1), d_logits=d)


def _exact_finalize(case, seed):
    T, H, k = case["T"], case["H"], case["k"]
    s, R = _finalize_inputs(case, seed), case["T"] * case["k"]
    y = s["y"]
    if case["dtype"] == "bf16":
        e = y[R * H * 2:].view(torch.int8).view(R, -1).to(torch.int32)
        y = torch.ldexp(y[:R * H * 2].view(torch.float16).view(R, H).double(), e[:, torch.arange(H, device=DEV) // 256])
    rows = s["inv"].long().view(T, k)
    d_out = s["d_out"].double()
    return torch.stack([torch.linalg.vecdot(y[rows[:, j]].double(), d_out) for j in range(k)], 1)


def _exact_wgrad(case, seed):
    s = _wgrad_inputs(case, seed)
    rows = torch.arange(case["T"], device=DEV) if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
    d = s["d_logits"][rows].double()
    return dict(d_wg=d.T.contiguous() @ s["x"][rows].double(), d_bias=d.sum(0))


def exact(case, seed):
    return {"q4_layer": _exact_q4, "balance": _exact_balance, "finalize_backward": _exact_finalize, "router_weight_grad": _exact_wgrad}[case["kind"]](case, seed)
