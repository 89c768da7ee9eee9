"""Cases of the shared expert's training step, of its request adapters and of dropout, with plain forms.

Three operators beside the routed experts:

- `ffn_train`: the shared expert as a gated feed-forward block that is trained. Gate and up projections, SwiGLU,
  dropout of the hidden values and the down projection with a residual, then the gradients of x and of both weights;
- `lora_w13`, `lora_down`, `lora_ffn`: the shared expert's two projections, and both in a row, each with low-rank
  adapters of many requests at once (every token names its adapter, or none);
- `dropout`: dropout of a layer's output with the residual added, and its backward pass. The mask comes from a counter
  and a seed and is stored nowhere.

With `own` false, `run` computes them with elementary torch operations in 32 bits; with `own` true it calls the
library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def _named(name, c):
    return dict(c, name=name) if name else c


def _ffn(name, T, H, Is, dtype, p, residual):
    return _named(name, dict(kind="ffn_train", T=T, H=H, Is=Is, dtype=dtype, p=p, residual=residual))


def _lora(name, kind, T, H, Is, L, r, dtype, ids):
    return _named(name, dict(kind=kind, T=T, H=H, Is=Is, L=L, r=r, dtype=dtype, ids=ids))


def _dropout(name, T, H, dtype, p, residual):
    return _named(name, dict(kind="dropout", T=T, H=H, dtype=dtype, p=p, residual=residual))


def listed():
    return [
        # a test-sized fp32 layer: launches count
        _ffn("ffn f32 small", 64, 256, 128, "f32", 0.0, False),
        # one short image's tokens at a narrow model: no size is a multiple of a tile
        _ffn("ffn ragged", 333, 1024, 352, "bf16", 0.1, True),
        # the decode layer's shared width, a medium batch
        _ffn("ffn medium", 2048, 4096, 768, "bf16", 0.0, True),
        # two denoise sequences in one training step
        _ffn("ffn long", 8192, 4096, 2048, "bf16", 0.1, True),
        # fp32 training at odd sizes
        _ffn("ffn f32 odd", 1001, 1024, 704, "f32", 0.25, False),
        # one request's next token
        _lora("lora one token", "lora_ffn", 1, 4096, 768, 8, 16, "bf16", "tokens"),
        # a decode step, every token of another request
        _lora("lora decode", "lora_ffn", 16, 4096, 768, 64, 32, "bf16", "tokens"),
        # many requests' next tokens, some without an adapter
        _lora("lora batch", "lora_w13", 300, 4096, 768, 64, 16, "bf16", "tokens"),
        # prompts and images of a few requests, one after the other
        _lora("lora prefill", "lora_down", 8192, 4096, 2048, 16, 64, "bf16", "requests"),
        # a small fp32 layer of odd sizes
        _lora("lora f32 odd", "lora_ffn", 77, 448, 160, 5, 8, "f32", "requests"),
        # the denoise layer's output
        _dropout("dropout", 4096, 4096, "bf16", 0.1, True),
        # a few tokens in fp32: latency counts
        _dropout("dropout f32 small", 5, 320, "f32", 0.3, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["ffn_train", "ffn_train", "lora_w13", "lora_down", "lora_ffn", "dropout"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    H = 64 * _log(rng, 4, 64)
    if kind == "dropout":
        T = min(_log(rng, 1, 16384), 4096 * 4096 // H)
        return _dropout(None, T, H, dtype, round(rng.uniform(0.02, 0.6), 3), rng.random() < 0.5)
    Is = 32 * _log(rng, 2, 64)
    if kind == "ffn_train":
        T = _log(rng, 1, 8192)
        if dtype == "f32":
            T = min(T, max(1, 2 ** 31 // (H * Is)))
        return _ffn(None, T, H, Is, dtype, rng.choice([0.0, round(rng.uniform(0.02, 0.5), 3)]), rng.random() < 0.7)
    T = _log(rng, 1, 8192)
    if dtype == "f32":
        T = min(T, max(1, 2 ** 31 // (H * Is)))
    r = 8 * rng.choice([1, 1, 2, 2, 3, 4, 6, 8])
    L = _log(rng, 1, 64)
    return _lora(None, kind, T, H, Is, L, r, dtype, rng.choice(["tokens", "requests"]))


# ---------------------------------------------------------------- inputs

def _gen(seed, tag):
    return torch.Generator(device=DEV).manual_seed((seed * 1000003 + tag * 7919) % (2 ** 62))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _randn(shape, gen, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def _rng_state(seed):
    # seed and offset of the random stream, as the training program holds them on the device
    return torch.tensor([(seed * 6364136223846793005 + 1442695040888963407) % (2 ** 63), 3 + seed % 1000], dtype=torch.int64, device=DEV)


def _ffn_inputs(case, seed):
    T, H, Is, dt = case["T"], case["H"], case["Is"], _dtype(case)
    return dict(
        x=_randn((T, H), _gen(seed, 1), dt), w1=_randn((2 * Is, H), _gen(seed, 2), dt, 0.02), w2=_randn((H, Is), _gen(seed, 3), dt, 0.02),
        residual=_randn((T, H), _gen(seed, 4), dt) if case["residual"] else None, d_out=_randn((T, H), _gen(seed, 5), dt, 1e-2),
        rng=_rng_state(seed) if case["p"] > 0 else None)


def _ids(case, seed):
    """Adapter of every token, -1 for none: each token its own request, or requests one after the other."""
    T, L = case["T"], case["L"]
    host = np.random.default_rng(seed * 31 + 7)
    if case["ids"] == "tokens":
        ids = host.integers(0, L, T)
        ids[host.random(T) < 0.1] = -1
    else:
        n = max(1, min(T, 2 * L))
        cuts = np.sort(host.integers(0, T + 1, n - 1))
        ids = np.repeat(host.integers(-1, L, n), np.diff(np.concatenate([[0], cuts, [T]])))
    return torch.from_numpy(ids.astype(np.int32)).to(DEV)


def _lora_inputs(case, seed):
    T, H, Is, L, r, dt, kind = case["T"], case["H"], case["Is"], case["L"], case["r"], _dtype(case), case["kind"]
    s = dict(ids=_ids(case, seed), scale=0.5 + 1.5 * torch.rand(L, generator=_gen(seed, 9), device=DEV))
    if kind != "lora_down":
        s.update(x=_randn((T, H), _gen(seed, 1), dt), w1=_randn((2 * Is, H), _gen(seed, 2), dt, 0.02),
                 a1=_randn((L, r, H), _gen(seed, 3), dt, H ** -0.5), b1=_randn((L, 2 * Is, r), _gen(seed, 4), dt, 0.5 * r ** -0.5))
    else:
        s.update(hs=_randn((T, Is), _gen(seed, 1), dt))
    if kind != "lora_w13":
        s.update(w2=_randn((H, Is), _gen(seed, 5), dt, 0.02), a2=_randn((L, r, Is), _gen(seed, 6), dt, Is ** -0.5),
                 b2=_randn((L, H, r), _gen(seed, 7), dt, 0.5 * r ** -0.5), residual=_randn((T, H), _gen(seed, 8), dt))
    return s


def _dropout_inputs(case, seed):
    T, H, dt = case["T"], case["H"], _dtype(case)
    return dict(y=_randn((T, H), _gen(seed, 1), dt, 0.6), residual=_randn((T, H), _gen(seed, 2), dt) if case["residual"] else None,
                d_out=_randn((T, H), _gen(seed, 3), dt, 1e-2), rng=_rng_state(seed))


def prepare(case, seed):
    make = {"ffn_train": _ffn_inputs, "dropout": _dropout_inputs}.get(case["kind"], _lora_inputs)
    return dict(make(case, seed), case=dict(case))


# ---------------------------------------------------------------- plain forms

def _keep(rng, n, p):
    """Dropout factors [n], n a multiple of 8: 0 or 1 / (1 - p), p rounded to 1/65536. Eight elements share one
    Philox 4x32-10 block of the counter (element // 8, offset) under the key seed, 16 bits each, lowest first."""
    low = 0xFFFFFFFF
    i = torch.arange(n // 8, device=DEV, dtype=torch.int64)
    seed, offset = rng[0], rng[1]
    c = [i & low, i >> 32, (offset & low).expand_as(i), ((offset >> 32) & low).expand_as(i)]
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # 64-bit products, kept modulo 2^64
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, 1)
    u = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)
    cut = int(math.floor(p * 65536 + 0.5))
    return (u >= cut).float() * (65536.0 / (65536 - cut))


def _plain_ffn(s):
    case = s["case"]
    T, Is, dt = case["T"], case["Is"], s["x"].dtype
    x, w1, w2, d = s["x"].float(), s["w1"].float(), s["w2"].float(), s["d_out"].float()
    z = x @ w1.T
    g, u = z[:, :Is], z[:, Is:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    act = g * sig
    keep = _keep(s["rng"], T * Is, case["p"]).view(T, Is) if case["p"] > 0 else None
    h = act * u if keep is None else act * u * keep
    out = h @ w2.T
    if s["residual"] is not None:
        out = out + s["residual"].float()
    dh = d @ w2
    if keep is not None:
        dh = dh * keep
    dz = torch.cat([dh * u * (sig * (1.0 + g * (1.0 - sig))), dh * act], 1)
    return dict(out=out.to(dt), d_x=(dz @ w1).to(dt), d_w1=(dz.T @ x).to(dt), d_w2=(d.T @ h).to(dt))


def _plain_project(x, w, a, b, scale, ids):
    """x w^T plus every token's own adapter: all adapters' low-rank values, those of the others struck out."""
    T, (L, r, K) = x.shape[0], a.shape
    v = (x @ a.reshape(L * r, K).float().T).view(T, L, r)
    mine = (ids[:, None] == torch.arange(L, device=DEV)[None, :]).float() * scale
    v = (v * mine[:, :, None]).reshape(T, L * r)
    return x @ w.float().T + v @ b.float().permute(0, 2, 1).reshape(L * r, -1)


def _plain_lora(s):
    case = s["case"]
    kind, Is = case["kind"], case["Is"]
    dt = _dtype(case)
    out = {}
    if kind != "lora_down":
        z = _plain_project(s["x"].float(), s["w1"], s["a1"], s["b1"], s["scale"], s["ids"])
        g, u = z[:, :Is], z[:, Is:]
        out["hs"] = (g / (1.0 + torch.exp(-g)) * u).to(dt)
    if kind != "lora_w13":
        hs = out["hs"] if kind == "lora_ffn" else s["hs"]
        out["out"] = (_plain_project(hs.float(), s["w2"], s["a2"], s["b2"], s["scale"], s["ids"]) + s["residual"].float()).to(dt)
    return out


def _plain_dropout(s):
    case = s["case"]
    T, H, dt = case["T"], case["H"], s["y"].dtype
    keep = _keep(s["rng"], T * H, case["p"]).view(T, H)
    out = s["y"].float() * keep
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return dict(out=out.to(dt), d_y=(s["d_out"].float() * keep).to(dt))


# ---------------------------------------------------------------- the library's calls

def _shape(moe, case):
    return moe.make_shape(case["T"], case["H"], 1, 1, 32, 1, case["dtype"])


def _own_ffn(s):
    import mixture_experts_ffn_moe_amd as moe
    case = s["case"]
    T, H, Is, dt = case["T"], case["H"], case["Is"], s["x"].dtype
    if "shape" not in s:
        s["shape"] = _shape(moe, case)
        s["workspace"] = torch.empty(moe.moe_shared_backward_workspace_size(s["shape"], Is), dtype=torch.uint8, device=DEV)
    e = lambda *dims: torch.empty(*dims, dtype=dt, device=DEV)  # noqa: E731
    gu, hs, out = torch.empty(T, 2 * Is, device=DEV), e(T, Is), e(T, H)
    d_x, d_w1, d_w2 = e(T, H), e(2 * Is, H), e(H, Is)
    moe.moe_shared_ffn_train(s["shape"], Is, case["p"], s["rng"], s["x"], s["w1"], s["w2"], s["residual"], gu, hs, out)
    moe.moe_shared_ffn_backward(s["shape"], Is, case["p"], s["rng"], s["x"], s["w1"], s["w2"], gu, hs, s["d_out"], d_x, d_w1, d_w2,
                                s["workspace"])
    return dict(out=out, d_x=d_x, d_w1=d_w1, d_w2=d_w2)


def _own_lora(s):
    import mixture_experts_ffn_moe_amd as moe
    case = s["case"]
    T, H, Is, kind, dt = case["T"], case["H"], case["Is"], case["kind"], _dtype(case)
    if "shape" not in s:
        s["shape"], s["lora"] = _shape(moe, case), moe.make_lora(case["L"], case["r"])
        s["workspace"] = torch.empty(moe.moe_lora_workspace_size(s["shape"], Is, s["lora"]), dtype=torch.uint8, device=DEV)
    shape, lora, ws = s["shape"], s["lora"], s["workspace"]
    hs = torch.empty(T, Is, dtype=dt, device=DEV) if kind != "lora_down" else s["hs"]
    if kind == "lora_w13":
        moe.moe_lora_w13_swiglu(shape, Is, lora, s["x"], s["w1"], s["a1"], s["b1"], s["scale"], s["ids"], hs, ws)
        return dict(hs=hs)
    out = torch.empty(T, H, dtype=dt, device=DEV)
    if kind == "lora_down":
        moe.moe_lora_down(shape, Is, lora, hs, s["w2"], s["a2"], s["b2"], s["scale"], s["ids"], s["residual"], out, ws)
        return dict(out=out)
    moe.moe_shared_ffn_lora(shape, Is, lora, s["x"], s["w1"], s["w2"], s["a1"], s["b1"], s["a2"], s["b2"], s["scale"], s["ids"],
                            s["residual"], hs, out, ws)
    return dict(hs=hs, out=out)


def _own_dropout(s):
    import mixture_experts_ffn_moe_amd as moe
    case = s["case"]
    if "shape" not in s:
        s["shape"] = _shape(moe, case)
    out, d_y = torch.empty_like(s["y"]), torch.empty_like(s["y"])
    moe.moe_dropout_add(s["shape"], case["p"], s["rng"], s["y"], s["residual"], out)
    moe.moe_dropout_backward(s["shape"], case["p"], s["rng"], s["d_out"], d_y)
    return dict(out=out, d_y=d_y)


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"ffn_train": _own_ffn, "dropout": _own_dropout}.get(kind, _own_lora)(state)
    return {"ffn_train": _plain_ffn, "dropout": _plain_dropout}.get(kind, _plain_lora)(state)


# ---------------------------------------------------------------- work and exact values

def work(case):
    T, H, kind = case["T"], case["H"], case["kind"]
    size = 2 if case["dtype"] == "bf16" else 4
    if kind == "dropout":
        return {"bytes": float(T * H * size * (5 if case["residual"] else 4)), "flops": 3.0 * T * H}
    Is = case["Is"]
    if kind == "ffn_train":
        # reads x, residual, d_out and the weights, writes out, d_x and the weights' gradients
        return {"bytes": float(size * (T * H * (5 if case["residual"] else 4) + 2 * 3 * H * Is)), "flops": 18.0 * T * H * Is}
    L, r = case["L"], case["r"]
    n = T if case["ids"] == "tokens" else min(T, 2 * L)
    active = L * (1.0 - (1.0 - 1.0 / L) ** n) if L > 1 else 1.0  # adapters that any token names
    w13 = size * (T * (H + Is) + 2 * Is * H + active * r * (H + 2 * Is)), T * (4.0 * H * Is + 2.0 * r * (H + 2 * Is))
    down = size * (T * (Is + 2 * H) + H * Is + active * r * (H + Is)), T * (2.0 * H * Is + 2.0 * r * (H + Is))
    if kind == "lora_w13":
        return {"bytes": float(w13[0]), "flops": w13[1]}
    if kind == "lora_down":
        return {"bytes": float(down[0]), "flops": down[1]}
    return {"bytes": float(w13[0] + down[0] - size * T * Is), "flops": w13[1] + down[1]}


def _factors(state, rows, cols, p):
    """Dropout factors [rows, cols] in 64 bits, the generator written out over numpy's unsigned integers."""
    seed, offset = (int(v) % 2 ** 64 for v in state.tolist())
    u32 = np.uint64(0xFFFFFFFF)
    index = np.arange(rows * cols // 8, dtype=np.uint64)
    x0, x1 = index & u32, index >> np.uint64(32)
    x2, x3 = np.full_like(index, offset & 0xFFFFFFFF), np.full_like(index, offset >> 32)
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        m0, m1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = (m1 >> np.uint64(32)) ^ x1 ^ np.uint64(key[0]), m1 & u32, (m0 >> np.uint64(32)) ^ x3 ^ np.uint64(key[1]), m0 & u32
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = np.empty((len(index), 8), dtype=np.int64)
    for word, v in enumerate((x0, x1, x2, x3)):
        bits[:, 2 * word] = v % np.uint64(65536)
        bits[:, 2 * word + 1] = v // np.uint64(65536)
    cut = int(p * 65536 + 0.5)
    f = np.where(bits.reshape(rows, cols) < cut, 0.0, 65536.0 / (65536 - cut))
    return torch.from_numpy(f).to(DEV)


def _exact_ffn(case, seed):
    s = _ffn_inputs(case, seed)
    T, Is = case["T"], case["Is"]
    x, w1, w2, d = (s[n].double() for n in ("x", "w1", "w2", "d_out"))
    gate, up = torch.split(torch.nn.functional.linear(x, w1), Is, dim=1)
    f = _factors(s["rng"], T, Is, case["p"]) if case["p"] > 0 else torch.ones((), dtype=torch.float64, device=DEV)
    sigma = torch.sigmoid(gate)
    hidden = f * gate * sigma * up
    out = torch.nn.functional.linear(hidden, w2)
    if s["residual"] is not None:
        out += s["residual"].double()
    back = f * torch.mm(d, w2)
    d_gate = back * up * (sigma + gate * sigma * (1 - sigma))
    d_up = back * gate * sigma
    d_x = torch.mm(d_gate, w1[:Is]) + torch.mm(d_up, w1[Is:])
    d_w1 = torch.cat([torch.mm(d_gate.t(), x), torch.mm(d_up.t(), x)])
    return dict(out=out, d_x=d_x, d_w1=d_w1, d_w2=torch.mm(d.t(), hidden))


def _exact_project(x, w, a, b, scale, ids):
    out = torch.nn.functional.linear(x, w.double())
    for adapter in range(a.shape[0]):
        rows = torch.nonzero(ids == adapter)[:, 0]
        if len(rows):
            low = torch.nn.functional.linear(x[rows], a[adapter].double())
            out[rows] += torch.nn.functional.linear(low, b[adapter].double()) * scale[adapter].double()
    return out


def _exact_lora(case, seed):
    s = _lora_inputs(case, seed)
    out = {}
    if case["kind"] != "lora_down":
        gate, up = torch.split(_exact_project(s["x"].double(), s["w1"], s["a1"], s["b1"], s["scale"], s["ids"]), case["Is"], dim=1)
        out["hs"] = torch.nn.functional.silu(gate) * up
    if case["kind"] != "lora_w13":
        hs = out["hs"] if case["kind"] == "lora_ffn" else s["hs"].double()
        out["out"] = _exact_project(hs, s["w2"], s["a2"], s["b2"], s["scale"], s["ids"]) + s["residual"].double()
    return out


def _exact_dropout(case, seed):
    s = _dropout_inputs(case, seed)
    f = _factors(s["rng"], case["T"], case["H"], case["p"])
    out = f * s["y"].double()
    if s["residual"] is not None:
        out += s["residual"].double()
    return dict(out=out, d_y=f * s["d_out"].double())


def exact(case, seed):
    return {"ffn_train": _exact_ffn, "dropout": _exact_dropout}.get(case["kind"], _exact_lora)(case, seed)
