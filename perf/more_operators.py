"""The operators that end a pair stack's training step, and its linear layers in 8 bits.

Two families: AdamW over many tensors at once, with states in 32 bits or in 8 (e4m3 with a scale for
each 128 neighbours), which takes the gradients' clipping factor from their norm on the device; and a
linear layer whose operands are e4m3 with a power of two for each block of 128, forward and with its
gradients.  With `own` false, `run` is their plain form in elementary torch operations.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
DEV = "cuda"
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.999, 1e-8, 1e-3, 0.01
BLOCK = 128


# ------------------------------------------------------------------ the cases
def _adamw(name, bits, layers, C, D, param, grad, copy, clip, stochastic, count):
    return {"name": name, "op": "adamw", "bits": bits, "layers": layers, "C": C, "D": D, "param": param, "grad": grad,
            "copy": copy, "clip": clip, "stochastic": stochastic, "count": count}


def _linear(name, train, rows, K, N, weight, bias, spread):
    return {"name": name, "op": "linear", "train": train, "rows": rows, "K": K, "N": N, "weight": weight, "bias": bias,
            "spread": spread}


def listed():
    return [
        # one layer's ten parameters at the start of a training run: the call's latency
        _adamw("adamw_1_layer_d128", 32, 1, 128, 128, "fp32", "fp32", "bf16", 0.0, False, 0),
        # a stack of 48 blocks with two layers each, 960 tensors, its gradients clipped in the same pass
        _adamw("adamw_96_layers_d256", 32, 96, 256, 256, "fp32", "fp32", "bf16", 0.5, False, 5000),
        # weights kept in bf16 alone, which stochastic rounding lets take small steps; odd widths
        _adamw("adamw_24_layers_d136_bf16", 32, 24, 200, 136, "bf16", "bf16", "none", 2.0, True, 700),
        # the same three with states in 8 bits
        _adamw("adamw8_1_layer_d128", 8, 1, 128, 128, "fp32", "fp32", "bf16", 0.0, True, 0),
        _adamw("adamw8_96_layers_d256", 8, 96, 256, 256, "fp32", "fp32", "bf16", 0.5, True, 5000),
        _adamw("adamw8_24_layers_d136_bf16", 8, 24, 200, 136, "bf16", "bf16", "none", 0.0, True, 700),
        # a transition's first product in inference: the smallest complex
        _linear("linear8_n64_32x128", False, 64 * 64, 32, 128, "bf16", False, 1.0),
        # an odd crop
        _linear("linear8_333x257_136x544", False, 333 * 257, 136, 544, "bf16", True, 4.0),
        # a long complex
        _linear("linear8_n1024_256x1024", False, 1024 * 1024, 256, 1024, "bf16", True, 1.0),
        # a wide layer over tokens, where the tensor cores count
        _linear("linear8_8192_4096x4096", False, 8192, 4096, 4096, "bf16", False, 1.0),
        # a training step of a transition's first product at a crop: new weights laid out, forward, gradients
        _linear("linear8_train_n256_128x512", True, 256 * 256, 128, 512, "fp32", True, 1.0),
        # the same of its second product at a long complex
        _linear("linear8_train_n1024_1024x256", True, 1024 * 1024, 1024, 256, "fp32", False, 4.0),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    if rng.random() < 0.5:
        param = rng.choice(["fp32", "fp32", "bf16"])
        c = _adamw("", rng.choice([32, 8]), size(1, 96), 8 * size(2, 32), 8 * size(2, 32), param,
                   rng.choice(["fp32", "bf16", "fp16"]), rng.choice(["none", "bf16", "fp16"]) if param == "fp32" else "none",
                   rng.choice([0.0, 0.3, 2.0]), rng.random() < 0.6, rng.choice([0, 1, 10, 3000, 100000]))
    else:
        K, N = 8 * size(1, 256), 8 * size(1, 256)
        most = min((1 << 38) // (K * N), (1280 << 20) // (K + N))
        c = _linear("", rng.random() < 0.5, min(size(1, 1 << 20), most), K, N, rng.choice(["bf16", "fp32"]),
                    rng.random() < 0.5, rng.choice([1.0, 4.0]))
    c.pop("name")
    return c


def work(case):
    w = {"bf16": 2, "fp32": 4, "fp16": 2, "none": 0}
    if case["op"] == "adamw":
        weights, vectors = _sizes(case)
        n = sum(weights) + sum(vectors)
        blocks = sum(-(-k // BLOCK) for k in weights + vectors)
        state = 16 * n if case["bits"] == 32 else 4 * n + 16 * blocks
        return {"bytes": n * (2 * w[case["param"]] + w[case["grad"]]) + state + sum(weights) * w[case["copy"]] + 8, "flops": 16 * n}
    rows, K, N = case["rows"], case["K"], case["N"]
    bias = 4 * N if case["bias"] else 0
    if not case["train"]:  # the weight as it is kept: its codes
        return {"bytes": 2 * rows * (K + N) + N * K + bias, "flops": 2 * rows * K * N}
    return {"bytes": 2 * rows * (2 * K + 2 * N) + N * K * (w[case["weight"]] + 4) + 2 * bias, "flops": 6 * rows * K * N}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _sizes(case):
    """The weights' sizes, layer by layer, and the vectors' (the norms' scales and shifts)."""
    C, D, L = case["C"], case["D"], case["layers"]
    return [n for _ in range(L) for n in (C * D, C * D, C * D, C * D, D * C, D * D)], [n for _ in range(L) for n in (D, D, C, C)]


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "linear":
        rows, K, N = case["rows"], case["K"], case["N"]
        # activations whose channels differ in size, some of them far above the others
        wide = torch.exp(math.log(case["spread"]) * _randn(g, K))
        s["x"] = (_randn(g, rows, K) * wide).to(torch.bfloat16)
        s["w"] = (_randn(g, N, K) / math.sqrt(K)).to(DT[case["weight"]])
        s["b"] = 0.1 * _randn(g, N) if case["bias"] else None
        s["dy"] = (1e-3 * _randn(g, rows, N) * torch.exp(math.log(case["spread"]) * _randn(g, N))).to(torch.bfloat16) if case["train"] else None
        if own:
            from co_folding_pair_gb300 import train_ops as P
            s["plan"] = P.Linear8(s["w"], s["b"])
        elif not case["train"]:
            s["w8"] = _blocks_plain(s["w"])
        return s
    weights, vectors = _sizes(case)
    sizes = weights + vectors
    padded = [-(-n // BLOCK) * BLOCK for n in sizes]
    total, starts = sum(padded), [0]
    for n in padded[:-1]:
        starts.append(starts[-1] + n)
    n, at = torch.tensor(sizes, device=DEV), torch.tensor(padded, device=DEV)
    which = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), at)
    index = torch.arange(total, device=DEV) - torch.tensor(starts, device=DEV)[which]
    real = index < n[which]
    s["which"], s["index"], s["weights"] = which, index, sum(padded[: len(weights)])
    # parameters near the scale of a layer's, gradients whose tensors differ in size, states of a run under way
    size = torch.exp(1.5 * _randn(g, len(sizes)))[which] * 1e-2
    s["p"] = torch.where(real, 0.05 * _randn(g, total), 0.0).to(DT[case["param"]])
    s["g"] = torch.where(real, size * _randn(g, total), 0.0).to(DT[case["grad"]])
    m = torch.where(real, 0.3 * size * _randn(g, total), 0.0) if case["count"] else torch.zeros(total, device=DEV)
    r = torch.where(real, size * torch.exp(0.5 * _randn(g, total)), 0.0) if case["count"] else torch.zeros(total, device=DEV)
    if case["bits"] == 32:
        s["m"], s["v"] = m, r * r
    else:
        for key, x in (("m", m), ("v", r)):
            scale = x.view(-1, BLOCK).abs().amax(1).clamp(min=2.0**-90) / 448
            s[key], s[key + "_scale"] = (x.view(-1, BLOCK) / scale[:, None]).to(E4M3).view(-1), scale
    s["count_now"] = torch.full((), case["count"], dtype=torch.int32, device=DEV)
    s["copies"] = torch.zeros(s["weights"], dtype=DT[case["copy"]], device=DEV) if case["copy"] != "none" else None
    s["norm"] = s["g"].double().square().sum().sqrt().float() if case["clip"] else None
    s["max_norm"] = case["clip"] * float(s["norm"]) if case["clip"] else None
    s["seed_bits"] = seed % (1 << 31)
    if own:
        from co_folding_pair_gb300 import pair_ops
        from co_folding_pair_gb300 import train_ops as P

        def views(flat, count=len(sizes)):
            return [flat[a:a + k] for a, k in zip(starts[:count], sizes)]

        copies = None if s["copies"] is None else views(s["copies"], len(weights)) + [None] * len(vectors)
        s["plan"] = P.AdamW(views(s["p"]), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=[DECAY] * len(weights) + [0.0] * len(vectors),
                            states="8bit" if case["bits"] == 8 else "float32", copies=copies,
                            rounding="stochastic" if case["stochastic"] else "nearest", seed=s["seed_bits"])
        for key, flat in s["plan"].state.items():  # as a program that goes on from a checkpoint fills them
            flat.copy_(s["count_now"] if key == "count" else s[key])
        s["grads"] = pair_ops.GradSet(views(s["g"]))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return _linear_plain(s) if s["op"] == "linear" else _adamw_plain(s)


def _run_own(s):
    if s["op"] == "adamw":
        s["plan"].step(s["grads"], norm=s["norm"], max_norm=s["max_norm"])
        return {"p": s["p"], "copies": s["copies"], **s["plan"].state}
    if not s["train"]:
        return {"y": s["plan"].forward(s["x"])}
    s["plan"].pack(s["w"])
    y = s["plan"].forward(s["x"])
    return {"y": y, **s["plan"].backward(s["x"], s["dy"])}


# ------------------------------------------------------------------ plain forms
def _codes_plain(v, amax):
    """v 2^-e as e4m3, and 2^e, for the least e >= -126 with amax <= 448 2^e = 0.875 2^(e + 9)."""
    share, power = torch.frexp(amax)
    e = torch.where(amax > 0, power - 9 + (share > 0.875).int(), -126).clamp(min=-126)
    return (v * ((127 - e) << 23).view(torch.float32)).to(E4M3).float(), ((127 + e) << 23).view(torch.float32)


def _rows_plain(x):
    """x as its 8-bit form stands for it, a power of two for each 128 neighbours of a row."""
    rows, K = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).view(rows, -1, BLOCK)
    q, two = _codes_plain(v, v.abs().amax(2, keepdim=True))
    return (q * two).view(rows, -1)[:, :K]


def _blocks_plain(w):
    """The same with a power of two for each 128 x 128 block."""
    N, K = w.shape
    v = torch.nn.functional.pad(w.float(), (0, -K % BLOCK, 0, -N % BLOCK))
    v = v.view(v.shape[0] // BLOCK, BLOCK, -1, BLOCK)
    q, two = _codes_plain(v, v.abs().amax((1, 3), keepdim=True))
    return (q * two).view(N + -N % BLOCK, -1)[:N, :K].contiguous()


def _linear_plain(s):
    w = _blocks_plain(s["w"]) if s["train"] else s["w8"]
    y = _rows_plain(s["x"]) @ w.t()
    y = (y if s["b"] is None else y + s["b"]).to(torch.bfloat16)
    if not s["train"]:
        return {"y": y}
    dx = (_rows_plain(s["dy"]) @ w).to(torch.bfloat16)
    # sums over as many as a million rows: parts of 4096 in 32 bits, the parts in 64
    a, b = (torch.nn.functional.pad(_rows_plain(t.t().contiguous()), (0, -s["rows"] % 4096)) for t in (s["dy"], s["x"]))
    a, b = a.view(s["N"], -1, 4096).transpose(0, 1), b.view(s["K"], -1, 4096).permute(1, 2, 0)
    dw = torch.bmm(a, b).double().sum(0).float()
    return {"y": y, "dx": dx, "dw": dw, "dbias": None if s["b"] is None else s["dy"].double().sum(0).float()}


def _hash_plain(x):
    """32 bits of each x: the PCG hash of Jarzynski and Olano, "Hash Functions for GPU Rendering" (2020)."""
    x = (x * 747796405 + 2891336453) & 0xFFFFFFFF
    x = (((x >> ((x >> 28) + 4)) ^ x) * 277803737) & 0xFFFFFFFF
    return (x >> 22) ^ x


def _bits_plain(s, t):
    """32 random bits for each number of each tensor, for this step."""
    key = _hash_plain((s["which"] + _hash_plain((t + _hash_plain(torch.tensor(s["seed_bits"], device=DEV))) & 0xFFFFFFFF)) & 0xFFFFFFFF)
    key = _hash_plain((key + (s["index"] >> 32)) & 0xFFFFFFFF)
    return _hash_plain(key ^ (s["index"] & 0xFFFFFFFF))


def _pack_plain(x, least, bits):
    """x as e4m3 with a scale for each 128 neighbours; bits: what to add below the three that are kept."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1).clamp(min=2.0**-90) * (1 / 448)
    y = x * (1 / scale)[:, None]
    if bits is not None:  # below 2^-6 the steps are as at 2^-6
        a = y.abs()
        base = torch.where(a < 2.0**-6, 2.0**-6, 0.0)
        a = (((a + base).view(torch.int32) + (bits << 4).int().view(-1, BLOCK)) & -(1 << 20)).view(torch.float32) - base
        y = torch.copysign(a.clamp(max=448.0), y)
    q = y.clamp(-448.0, 448.0).to(E4M3).float()
    if least is not None:
        q = torch.where(least.view(-1, BLOCK), q.clamp(min=2.0**-9), q)
    return q.to(E4M3).view(-1), scale


def _adamw_plain(s):
    t = s["count_now"].long() + 1
    td = t.double()
    c1, c2 = (1 - BETA1**td).float(), (1 - BETA2**td).float()
    clip = 1.0 if s["norm"] is None else (s["max_norm"] / (s["norm"] + 1e-6)).clamp(max=1.0)
    g = s["g"].float() * clip
    if s["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).square().view(-1)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    p = s["p"].float()
    step = LR * (m / c1) / ((v / c2).sqrt() + EPS)
    p = torch.cat([p[: s["weights"]] * (1 - LR * DECAY), p[s["weights"]:]]) - step
    bits = _bits_plain(s, t) if s["stochastic"] and (s["bits"] == 8 or s["param"] == "bf16") else None
    if s["param"] == "bf16" and bits is not None:
        p16 = ((p.view(torch.int32) + (_hash_plain(bits) & 0xFFFF).int()) & -(1 << 16)).view(torch.float32)
    else:
        p16 = p
    s["p"].copy_(p16)
    if s["copies"] is not None:
        s["copies"].copy_(p[: s["weights"]])
    s["count_now"].add_(1)
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {"p": s["p"], "copies": s["copies"], "m": s["m"], "v": s["v"], "count": s["count_now"]}
    for key, x, least, b in (("m", m, None, None if bits is None else bits & 0xFFFF), ("v", v.sqrt(), v > 0, None if bits is None else bits >> 16)):
        q, scale = _pack_plain(x, least, b)
        s[key].view(torch.uint8).copy_(q.view(torch.uint8))
        s[key + "_scale"].copy_(scale)
    return {"p": s["p"], "copies": s["copies"], "count": s["count_now"], **{k: s[k] for k in ("m", "m_scale", "v", "v_scale")}}


# ------------------------------------------------------------------ the definitions in 64 bits
def _e4m3_exact(x):
    """x to the nearest number that e4m3 has, ties to even, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0**-6))) - 3)
    return torch.round(x / step) * step


def _quantized_exact(x, axes):
    """x in groups over `axes`, each divided by the least power of two that brings it into e4m3's range, and back."""
    most = x.abs().amax(axes, keepdim=True)
    two = torch.exp2(torch.ceil(torch.log2(most.clamp(min=448 * 2.0**-126) / 448)))
    return _e4m3_exact(x / two) * two


def _grid(x, down, along):
    """[rows, columns] as [rows / down, down, columns / along, along], zeros past the end."""
    R, C = x.shape
    full = torch.zeros(-(-R // down) * down, -(-C // along) * along, dtype=torch.float64, device=DEV)
    full[:R, :C] = x
    return full.view(full.shape[0] // down, down, full.shape[1] // along, along)


def _exact_rows(x):
    return _quantized_exact(_grid(x, 1, BLOCK), (3,)).flatten(2).flatten(0, 1)[: x.shape[0], : x.shape[1]]


def _exact_columns(x):
    return _quantized_exact(_grid(x, BLOCK, 1), (1,)).flatten(2).flatten(0, 1)[: x.shape[0], : x.shape[1]]


def _linear_exact(s):
    w = _quantized_exact(_grid(s["w"], BLOCK, BLOCK), (1, 3)).flatten(2).flatten(0, 1)[: s["N"], : s["K"]]
    y = torch.einsum("rk,nk->rn", _exact_rows(s["x"]), w)
    if s["b"] is not None:
        y = y + s["b"].double()
    if not s["train"]:
        return {"y": y}
    dx = torch.einsum("rn,nk->rk", _exact_rows(s["dy"]), w)
    dw = torch.einsum("rn,rk->nk", _exact_columns(s["dy"]), _exact_columns(s["x"]))
    return {"y": y, "dx": dx, "dw": dw, "dbias": None if s["b"] is None else s["dy"].double().sum(0)}


def _pcg_exact(x):
    """The same hash in the wrapping arithmetic of 64-bit whole numbers, written for a list of stages."""
    mask = (1 << 32) - 1
    state = torch.remainder(x * 747796405 + 2891336453, 1 << 32)
    word = torch.bitwise_xor(torch.bitwise_right_shift(state, torch.bitwise_right_shift(state, 28) + 4), state)
    word = torch.bitwise_and(word * 277803737, mask)
    return torch.bitwise_xor(torch.bitwise_right_shift(word, 22), word)


def _codes_exact(x, chance, positive):
    """The e4m3 numbers of groups of 128 and their scales: `chance` in [0, 1) decides between the two neighbours."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1).clamp(min=2.0**-90) / 448
    y = x / scale[:, None]
    if chance is None:
        q = _e4m3_exact(y)
    else:
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
        q = torch.sign(y) * (torch.floor(y.abs() / step + chance.view(-1, BLOCK)) * step).clamp(max=448.0)
    if positive:
        q = torch.where(x > 0, q.clamp(min=2.0**-9), q)
    return q.view(-1), scale


def _adamw_exact(s):
    d = {k: s[k].double() for k in ("p", "g", "m", "v")}
    if s["bits"] == 8:
        d["m"] = (d["m"].view(-1, BLOCK) * s["m_scale"].double()[:, None]).view(-1)
        d["v"] = (d["v"].view(-1, BLOCK) * s["v_scale"].double()[:, None]).view(-1) ** 2
    t = s["count"] + 1
    clip = 1.0 if s["norm"] is None else min(1.0, s["max_norm"] / (float(s["norm"]) + 1e-6))
    g = clip * d["g"]
    m = BETA1 * d["m"] + (1 - BETA1) * g
    v = BETA2 * d["v"] + (1 - BETA2) * g**2
    decay = torch.where(torch.arange(g.numel(), device=DEV) < s["weights"], LR * DECAY, 0.0)
    p = d["p"] - decay * d["p"] - LR * (m / (1 - BETA1**t)) / (torch.sqrt(v / (1 - BETA2**t)) + EPS)
    h = None
    if s["stochastic"]:
        seed = _pcg_exact(torch.tensor(s["seed_bits"], device=DEV))
        key = _pcg_exact(torch.remainder(s["which"] + _pcg_exact(torch.remainder(seed + t, 1 << 32)), 1 << 32))
        h = _pcg_exact(torch.bitwise_xor(_pcg_exact(key), s["index"]))
    q = p
    if s["param"] == "bf16" and h is not None:  # one of the two neighbours among numbers of eight bits
        step = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=1e-30))) - 7)
        q = torch.sign(p) * torch.floor(p.abs() / step + torch.remainder(_pcg_exact(h), 1 << 16) / (1 << 16)) * step
    out = {"p": q, "copies": p[: s["weights"]] if s["copies"] is not None else None, "count": None}
    if s["bits"] == 32:
        return {**out, "m": m, "v": v}
    low, high = (None, None) if h is None else (torch.remainder(h, 1 << 16) / (1 << 16), torch.div(h, 1 << 16, rounding_mode="floor") / (1 << 16))
    out["m"], out["m_scale"] = _codes_exact(m, low, False)
    out["v"], out["v_scale"] = _codes_exact(torch.sqrt(v), high, True)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _linear_exact(s) if case["op"] == "linear" else _adamw_exact(s)
