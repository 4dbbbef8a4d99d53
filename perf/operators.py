"""The operators around a TriMul layer, as a pair stack's training step and inference use them.

Three operators: the relative position bias that the pair representation starts from (with its
table's gradient), the residual step from a layer's output back into the stream (norm after, gate,
scale, norm before the next layer; forward and backward), and the global norm of the gradients
with clipping.  With `own` false, `run` is their plain form in elementary torch operations.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp16": torch.float16}
DEV = "cuda"
EPS = 1e-5


# ------------------------------------------------------------------ the cases
def _relpos(name, back, layout, kind, B, I, J, D, M, K, two, chains, pad, base, table, dtype):
    return {"name": name, "op": "relpos", "back": back, "layout": layout, "kind": kind, "B": B, "I": I, "J": J, "D": D,
            "M": M, "K": K, "two": two, "chains": chains, "pad": pad, "base": base, "table": table, "dtype": dtype}


def _residual(name, back, B, I, J, D, stream, post, pre, gate, sigmoid, channel, pad):
    return {"name": name, "op": "residual", "back": back, "B": B, "I": I, "J": J, "D": D, "stream": stream, "post": post,
            "pre": pre, "gate": gate, "sigmoid": sigmoid, "channel": channel, "pad": pad}


def _clip(name, layers, C, D, dtype, kind, share):
    return {"name": name, "op": "clip", "layers": layers, "C": C, "D": D, "dtype": dtype, "kind": kind, "share": share}


def listed():
    return [
        # the smallest complex: the pair representation's start, where the call's latency is all
        _relpos("relpos_fwd_n64_d32", False, "pair", "linear", 1, 64, 64, 32, 32, 65, True, 1, 0.0, False, "bf16", "bf16"),
        # two padded complexes of several chains; the bias joins a pair representation that is there already
        _relpos("relpos_fwd_b2_n1024_d128", False, "pair", "linear", 2, 1024, 1024, 128, 32, 65, True, 3, 0.15, True, "bf16", "bf16"),
        # an attention's bias by log-spaced buckets, for queries of one length and keys of another
        _relpos("relpos_fwd_heads_515x1030", False, "heads", "log", 4, 515, 1030, 8, 128, 32, True, 1, 0.0, False, "fp32", "fp32"),
        # the table's gradient at a training crop
        _relpos("relpos_bwd_n256_d128", True, "pair", "linear", 1, 256, 256, 128, 32, 65, True, 2, 0.1, False, "bf16", "bf16"),
        # the same at a long complex
        _relpos("relpos_bwd_n2048_d256", True, "pair", "linear", 1, 2048, 2048, 256, 32, 65, True, 4, 0.0, False, "bf16", "bf16"),
        # a causal attention bias's gradient at an odd length
        _relpos("relpos_bwd_heads_1001", True, "heads", "log", 2, 1001, 1001, 16, 128, 32, False, 1, 0.0, False, "fp32", "bf16"),
        # the smallest complex after a layer
        _residual("residual_fwd_n64_d32", False, 1, 64, 64, 32, "bf16", "none", "layer", "none", False, False, 0.0),
        # a long complex in inference with a norm after the layer, a gate shared by a row, and the next layer's norm
        _residual("residual_fwd_n2048_d256", False, 1, 2048, 2048, 256, "bf16", "layer", "rms", "row", False, False, 0.0),
        # a training step on an odd, padded crop: a dropout mask shared by a column, a scale for each channel
        _residual("residual_bwd_333x257_d136", True, 1, 333, 257, 136, "bf16", "rms", "layer", "col", False, True, 0.1),
        # a training step with the stream in 32 bits, a learned gate for each pair, and both norms
        _residual("residual_bwd_n1024_d256", True, 1, 1024, 1024, 256, "fp32", "layer", "layer", "pair", True, False, 0.0),
        # one layer's ten gradients
        _clip("clip_1_layer_d128", 1, 128, 128, "fp32", "2", 0.5),
        # a whole stack of 48 blocks with two layers each: 960 tensors
        _clip("clip_96_layers_d256", 96, 256, 256, "fp32", "2", 0.1),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["relpos", "relpos", "residual", "residual", "clip"])
    if op == "clip":
        D = 8 * size(2, 32)
        c = _clip("", size(1, 96), 8 * size(2, 32), D, rng.choice(["fp32", "fp32", "bf16", "mixed"]),
                  rng.choice(["2", "2", "inf"]), rng.choice([0.01, 0.5, 2.0]))
    elif op == "relpos":
        back, layout = rng.random() < 0.5, rng.choice(["pair", "heads"])
        D = 8 * size(1, 32) if layout == "pair" else size(1, 24)
        B, I = rng.choice([1, 1, 2, 3]), size(1, 1400)
        J = I if rng.random() < 0.6 else size(1, 1400)
        kind, two, chains = rng.choice(["linear", "log"]), True, rng.choice([1, 1, 2, 5])
        if kind == "linear":
            M = size(1, 200)
            K = 2 * M + 1
        else:
            two = rng.random() < 0.5
            K = rng.choice([8, 16, 32, 64])
            M = size(K, 1000)
        base = rng.random() < 0.5 and not back
        c = _relpos("", back, layout, kind, B, I, J, D, M, K, two, chains, rng.choice([0.0, 0.1]) if chains > 1 else 0.0,
                    base, rng.choice(["bf16", "fp32"]), rng.choice(["bf16", "bf16", "fp32"]))
    else:
        back = rng.random() < 0.5
        gate = rng.choice(["none", "pair", "row", "col"])
        I = size(1, 800)
        c = _residual("", back, rng.choice([1, 1, 2]), I, I if rng.random() < 0.6 else size(1, 800), 8 * size(1, 32),
                      rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["none", "layer", "rms"]),
                      rng.choice(["none", "layer", "rms"]), gate, gate == "pair" and rng.random() < 0.5,
                      rng.random() < 0.4, rng.choice([0.0, 0.15]))
    c.pop("name")
    return c


def work(case):
    w = {"bf16": 2, "fp32": 4}
    if case["op"] == "relpos":
        pairs, D = case["B"] * case["I"] * case["J"], case["D"]
        rows = case["K"] + (case["chains"] > 1)
        small = 4 * case["B"] * (case["I"] + case["J"]) * (2 if case["chains"] > 1 else 1)
        if case["back"]:
            return {"bytes": pairs * D * w[case["dtype"]] + small + 4 * rows * D, "flops": pairs * D}
        return {"bytes": pairs * D * w[case["dtype"]] * (2 if case["base"] else 1) + small + rows * D * w[case["table"]],
                "flops": pairs * D * (1 if case["base"] else 0)}
    if case["op"] == "residual":
        B, I, J, D = (case[k] for k in "BIJD")
        n, s = B * I * J * D, w[case["stream"]]
        gate = {"none": 0, "pair": n, "row": B * J * D, "col": B * I * D}[case["gate"]] * 2
        mask = 2 * B * I * J if case["pad"] else 0
        params = 4 * D * ((case["post"] != "none") + (case["post"] == "layer") + (case["pre"] != "none") + (case["pre"] == "layer") + case["channel"])
        pre = 2 * n if case["pre"] != "none" else 0
        if case["back"]:
            dgate = gate if case["gate"] == "pair" else 0
            return {"bytes": n * (3 * s + 4) + gate + dgate + mask + pre + 2 * params, "flops": 40 * n}
        return {"bytes": n * (2 * s + 2) + gate + mask + pre + params, "flops": 20 * n}
    sizes = _clip_sizes(case)
    b = sum(n * _clip_type(case, k).itemsize for k, n in enumerate(sizes))
    return {"bytes": 2 * b + 4, "flops": 3 * sum(sizes)}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _tokens(B, N, chains, pad, g):
    """Residue numbers that start anew, and jump, at each chain; the chain of each token, -1 for padding."""
    cuts = torch.rand(B, chains - 1, generator=g, device=DEV).mul(N).to(torch.int64) if chains > 1 else torch.zeros(B, 0, dtype=torch.int64, device=DEV)
    at = torch.arange(N, device=DEV).expand(B, N)
    group = (at[:, :, None] >= cuts[:, None, :]).sum(2)
    starts = torch.randint(0, 500, (B, chains), generator=g, device=DEV)
    pos = at + torch.gather(starts, 1, group)
    real = N - (torch.rand(B, generator=g, device=DEV) * pad * N).to(torch.int64)
    group = torch.where(at < real[:, None], group, -1)
    return pos.to(torch.int32).contiguous(), group.to(torch.int32).contiguous()


def _clip_sizes(case):
    C, D = case["C"], case["D"]
    return [n for _ in range(case["layers"]) for n in (C * D, C * D, C * D, C * D, D * C, D * D, D, D, C, C)]


def _clip_type(case, k):
    return DT[case["dtype"]] if case["dtype"] != "mixed" else (torch.float32 if k % 10 >= 6 else torch.bfloat16)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "relpos":
        B, I, J, D, dt = case["B"], case["I"], case["J"], case["D"], DT[case["dtype"]]
        s["qpos"], s["qgroup"] = _tokens(B, I, case["chains"], case["pad"], g)
        s["kpos"], s["kgroup"] = (s["qpos"], s["qgroup"]) if I == J else _tokens(B, J, case["chains"], case["pad"], g)
        if I != J and case["kind"] == "log" and not case["two"]:  # the queries are the last tokens of the keys' sequence
            s["qpos"] = s["qpos"] + max(0, J - I)
        rows = case["K"] + (case["chains"] > 1)
        shape = (B, I, J, D) if case["layout"] == "pair" else (B, D, I, J)
        s["table"] = (0.5 * _randn(g, rows, D)).to(DT[case["table"]])
        s["base"] = _randn(g, *shape).to(dt) if case["base"] else None
        s["dout"] = _randn(g, *shape).to(dt) if case["back"] else None
        if own:
            from co_folding_pair_gb300 import pair_ops as P
            s["plan"] = P.RelPos(case["kind"], case["M"], num_buckets=case["K"] if case["kind"] == "log" else None,
                                 bidirectional=case["two"], groups=case["chains"] > 1)
        return s
    if case["op"] == "residual":
        B, I, J, D, dt = case["B"], case["I"], case["J"], case["D"], DT[case["stream"]]
        s["x"] = (2 * _randn(g, B, I, J, D)).to(dt)
        s["u"] = _randn(g, B, I, J, D).to(torch.bfloat16)
        s["params"] = {}
        for which in ("post", "pre"):
            if case[which] != "none":
                s["params"][which + "_gamma"] = 1 + 0.1 * _randn(g, D)
            if case[which] == "layer":
                s["params"][which + "_beta"] = 0.1 * _randn(g, D)
        if case["channel"]:
            s["params"]["channel"] = 0.5 + 0.1 * _randn(g, D)
        s["gate"] = None
        if case["gate"] == "pair":
            s["gate"] = _randn(g, B, I, J, D).to(torch.bfloat16)
        elif case["gate"] != "none":  # a dropout mask of a quarter
            shape = (B, 1, J, D) if case["gate"] == "row" else (B, I, 1, D)
            s["gate"] = ((torch.rand(shape, generator=g, device=DEV) >= 0.25).float() / 0.75).to(torch.bfloat16)
        s["mask"] = None
        if case["pad"]:
            ti = torch.arange(I, device=DEV) < I - (torch.rand(B, 1, generator=g, device=DEV) * case["pad"] * I).to(torch.int64)
            tj = torch.arange(J, device=DEV) < J - (torch.rand(B, 1, generator=g, device=DEV) * case["pad"] * J).to(torch.int64)
            s["mask"] = (ti[:, :, None] & tj[:, None, :]).to(torch.bfloat16)
        s["scale"] = 0.7
        if case["back"]:
            s["dout"] = _randn(g, B, I, J, D).to(dt)
            s["dnormed"] = _randn(g, B, I, J, D).to(torch.bfloat16) if case["pre"] != "none" else None
        if own:
            from co_folding_pair_gb300 import pair_ops as P
            s["plan"] = P.Residual(s["params"], post_norm=case["post"], pre_norm=case["pre"], scale=s["scale"],
                                   gate_sigmoid=case["sigmoid"], eps=EPS)
        return s
    sizes = _clip_sizes(case)
    kinds = [_clip_type(case, k) for k in range(len(sizes))]
    s["flat"], s["tensors"] = {}, [None] * len(sizes)
    for dt in sorted(set(kinds), key=str):
        which = [k for k, t in enumerate(kinds) if t == dt]
        flat = (0.02 * _randn(g, sum(sizes[k] for k in which))).to(dt)
        s["flat"][str(dt)] = flat
        for k, t in zip(which, flat.split([sizes[k] for k in which])):
            s["tensors"][k] = t
    s["out"] = {k: torch.empty_like(v) for k, v in s["flat"].items()}
    s["norm_type"] = 2.0 if case["kind"] == "2" else math.inf
    n = sum(sizes)
    s["max_norm"] = case["share"] * (0.02 * math.sqrt(n) if case["kind"] == "2" else 0.02 * math.sqrt(2 * math.log(n)))
    if own:
        from co_folding_pair_gb300 import pair_ops as P
        outs = {k: list(v.split([sizes[i] for i in range(len(sizes)) if str(kinds[i]) == k])) for k, v in s["out"].items()}
        s["plan"] = P.GradSet(s["tensors"], outs=[outs[str(kinds[i])].pop(0) for i in range(len(sizes))])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "relpos":
        return _relpos_plain(s)
    if s["op"] == "residual":
        return _residual_bwd_plain(s) if s["back"] else _residual_fwd_plain(s)
    return _clip_plain(s)


def _run_own(s):
    if s["op"] == "relpos":
        groups = {"q_group": s["qgroup"], "k_group": s["kgroup"]} if s["chains"] > 1 else {}
        if s["back"]:
            return s["plan"].backward(s["dout"], s["qpos"], s["kpos"], layout=s["layout"], **groups)
        return s["plan"].forward(s["table"], s["qpos"], s["kpos"], base=s["base"], layout=s["layout"], dtype=DT[s["dtype"]], **groups)
    if s["op"] == "residual":
        if s["back"]:
            return s["plan"].backward(s["x"], s["u"], s["dout"], dnormed=s["dnormed"], gate=s["gate"], mask=s["mask"])
        out, normed = s["plan"].forward(s["x"], s["u"], gate=s["gate"], mask=s["mask"])
        return {"out": out, "normed": normed}
    return {"norm": s["plan"].clip(s["max_norm"], norm_type=s["norm_type"]), "out": s["out"]}


# ------------------------------------------------------------------ plain forms
def _buckets_plain(s):
    d = s["qpos"].long()[:, :, None] - s["kpos"].long()[:, None, :]
    M = s["M"]
    if s["kind"] == "linear":
        b = d.clamp(-M, M) + M
    else:
        K = s["K"] // 2 if s["two"] else s["K"]
        E = K // 2
        n = d.abs() if s["two"] else d.clamp(min=0)
        # in 64 bits; a border that falls on a whole number is kept on its upper side
        far = E + torch.floor(torch.log(n.clamp(min=1).double() / E) / math.log(M / E) * (K - E) + 1e-9).long()
        b = torch.where(n < E, n, far.clamp(max=K - 1))
        if s["two"]:
            b = b + K * (d < 0)
    if s["chains"] > 1:
        gq, gk = s["qgroup"][:, :, None], s["kgroup"][:, None, :]
        b = torch.where(gq == gk, b, torch.full_like(b, s["K"]))
        b = torch.where((gq < 0) | (gk < 0), torch.full_like(b, -1), b)
    return b


def _relpos_plain(s):
    b = _buckets_plain(s)
    rows = s["K"] + (s["chains"] > 1)
    if s["back"]:
        d = s["dout"] if s["layout"] == "pair" else s["dout"].permute(0, 2, 3, 1)
        hot = (b.reshape(-1, 1) == torch.arange(rows, device=DEV)).double()
        return (hot.t() @ d.reshape(-1, s["D"]).double()).float()
    bias = s["table"].float()[b.clamp(min=0)] * (b >= 0)[..., None]
    if s["layout"] == "heads":
        bias = bias.permute(0, 3, 1, 2)
    if s["base"] is not None:
        bias = bias + s["base"].float()
    return bias.to(DT[s["dtype"]]).contiguous()


def _norm_plain(v, kind, gamma, beta):
    """(normalised, 1 / its deviation, the affine result) of v's last axis."""
    if kind == "none":
        return None, None, v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    hat = v * r
    return hat, r, hat * gamma + (beta if beta is not None else 0.0)


def _norm_back_plain(dy, hat, r, kind, gamma):
    if kind == "none":
        return dy
    t = dy * gamma
    d = t - hat * (t * hat).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - t.mean(-1, keepdim=True)
    return d * r


def _weight_plain(s):
    """s m c and the gate's value, 32 bits, and where a pair is real."""
    g = None if s["gate"] is None else torch.sigmoid(s["gate"].float()) if s["sigmoid"] else s["gate"].float()
    real = None if s["mask"] is None else (s["mask"] != 0)[..., None]
    k = torch.tensor(s["scale"], device=DEV) if s["mask"] is None else s["scale"] * s["mask"].float()[..., None]
    return k, g, real


def _residual_fwd_plain(s):
    p = s["params"]
    k, g, real = _weight_plain(s)
    y = _norm_plain(s["u"].float(), s["post"], p.get("post_gamma"), p.get("post_beta"))[2]
    w = k * y
    if "channel" in p:
        w = w * p["channel"]
    if g is not None:
        w = w * g
    x = s["x"].float()
    out = x + w if real is None else torch.where(real, x + w, x)
    n = None
    if s["pre"] != "none":
        n = _norm_plain(out, s["pre"], p["pre_gamma"], p.get("pre_beta"))[2]
        n = (n if real is None else torch.where(real, n, 0.0)).to(torch.bfloat16)
    return {"out": out.to(s["x"].dtype), "normed": n}


def _residual_bwd_plain(s):
    p = s["params"]
    k, g, real = _weight_plain(s)
    hat, r, y = _norm_plain(s["u"].float(), s["post"], p.get("post_gamma"), p.get("post_beta"))
    w = k if "channel" not in p else k * p["channel"]
    wg = w if g is None else w * g
    grads = {}
    d = s["dout"].float()
    if s["pre"] != "none":
        xhat, xr, _ = _norm_plain(s["x"].float() + wg * y, s["pre"], p["pre_gamma"], p.get("pre_beta"))
        dn = s["dnormed"].float() if real is None else torch.where(real, s["dnormed"].float(), 0.0)
        grads["pre_gamma"] = (dn * xhat).sum((0, 1, 2))
        if s["pre"] == "layer":
            grads["pre_beta"] = dn.sum((0, 1, 2))
        d = d + _norm_back_plain(dn, xhat, xr, s["pre"], p["pre_gamma"])
    dy = wg * d
    if s["post"] != "none":
        grads["post_gamma"] = (dy * hat).sum((0, 1, 2))
    if s["post"] == "layer":
        grads["post_beta"] = dy.sum((0, 1, 2))
    if "channel" in p:
        grads["channel"] = (k * y * d * (1.0 if g is None else g)).sum((0, 1, 2))
    dgate = None
    if s["gate"] is not None and s["gate"].shape == s["x"].shape:
        dgate = w * y * d
        dgate = (dgate * g * (1 - g) if s["sigmoid"] else dgate).to(torch.bfloat16)
    du = _norm_back_plain(dy, hat, r, s["post"], p.get("post_gamma"))
    return {"dx": d.to(s["x"].dtype), "du": du.to(torch.bfloat16), "dgate": dgate, "grads": grads}


def _clip_plain(s):
    flat = torch.cat([t.float() for t in s["tensors"]])
    norm = flat.double().square().sum().sqrt() if s["norm_type"] == 2.0 else flat.abs().max().double()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    parts = (flat.double() * coef).split([t.numel() for t in s["tensors"]])
    return {"norm": norm.float(), "out": {k: torch.cat([p for p, t in zip(parts, s["tensors"]) if str(t.dtype) == k]).to(v.dtype)
                                          for k, v in s["flat"].items()}}


# ------------------------------------------------------------------ the definitions in 64 bits
def _log_border(k, E, M, steps):
    """The least whole n with log(n / E) / log(M / E) * steps >= k, in whole numbers: n^steps E^k >= M^k E^steps."""
    lo, hi = E, M
    while lo < hi:
        mid = (lo + hi) // 2
        if mid ** steps * E ** k >= M ** k * E ** steps:
            hi = mid
        else:
            lo = mid + 1
    return lo


def _relpos_exact(s):
    d = (s["qpos"].double()[:, :, None] - s["kpos"].double()[:, None, :]).long()
    if s["kind"] == "linear":
        b = torch.minimum(torch.maximum(d, torch.tensor(-s["M"], device=DEV)), torch.tensor(s["M"], device=DEV)) + s["M"]
    else:
        K = s["K"] // 2 if s["two"] else s["K"]
        E = K // 2
        borders = torch.tensor(list(range(1, E)) + [_log_border(k, E, s["M"], K - E) for k in range(K - E)], device=DEV)
        n = torch.maximum(d, -d) if s["two"] else torch.maximum(d, torch.zeros_like(d))
        b = torch.searchsorted(borders, n, right=True)
        if s["two"]:
            b = torch.where(d < 0, b + K, b)
    rows = s["K"]
    if s["chains"] > 1:
        rows += 1
        same = s["qgroup"][:, :, None] == s["kgroup"][:, None, :]
        pad = (s["qgroup"] < 0)[:, :, None] | (s["kgroup"] < 0)[:, None, :]
        b = b.masked_fill(~same, rows - 1).masked_fill(pad, rows)
    if s["back"]:
        v = s["dout"].double() if s["layout"] == "pair" else s["dout"].double().movedim(1, 3)
        return torch.zeros(rows + 1, s["D"], dtype=torch.float64, device=DEV).index_add_(0, b.reshape(-1), v.reshape(-1, s["D"]))[: s["K"] + (s["chains"] > 1)].contiguous()
    table = torch.cat([s["table"].double(), torch.zeros(1, s["D"], dtype=torch.float64, device=DEV)])
    v = torch.nn.functional.embedding(b, table)
    v = v if s["layout"] == "pair" else v.movedim(3, 1)
    return (v if s["base"] is None else v + s["base"].double()).contiguous()


def _norm_exact(v, kind, gamma, beta):
    if kind == "none":
        return v
    if kind == "layer":
        var, mean = torch.var_mean(v, dim=-1, unbiased=False, keepdim=True)
        return (v - mean) / torch.sqrt(var + EPS) * gamma + beta
    return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + EPS) * gamma


def _residual_exact(s):
    p = {k: v.double().requires_grad_(s["back"]) for k, v in s["params"].items()}
    x, u = s["x"].double().requires_grad_(s["back"]), s["u"].double().requires_grad_(s["back"])
    gate = None
    if s["gate"] is not None:
        gate = s["gate"].double().requires_grad_(s["back"] and s["gate"].shape == s["x"].shape)
    m = torch.ones((), dtype=torch.float64, device=DEV) if s["mask"] is None else s["mask"].double().unsqueeze(-1)
    with torch.set_grad_enabled(s["back"]):
        t = _norm_exact(u, s["post"], p.get("post_gamma"), p.get("post_beta")) * (s["scale"] * m)
        t = t * p["channel"] if "channel" in p else t
        t = t if gate is None else t * (1 / (1 + torch.exp(-gate))) if s["sigmoid"] else t * gate
        out = x + t
        n = None if s["pre"] == "none" else _norm_exact(out, s["pre"], p["pre_gamma"], p.get("pre_beta")) * (m > 0)
        if not s["back"]:
            return {"out": out, "normed": n}
        outs, seeds = [out], [s["dout"].double()]
        if n is not None:
            outs, seeds = outs + [n], seeds + [s["dnormed"].double()]
        wanted = [x, u] + ([gate] if gate is not None and gate.requires_grad else []) + list(p.values())
        got = list(torch.autograd.grad(outs, wanted, seeds))
    res = {"dx": got.pop(0), "du": got.pop(0), "dgate": got.pop(0) if gate is not None and gate.requires_grad else None}
    return {**res, "grads": dict(zip(p, got))}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "relpos":
        return _relpos_exact(s)
    if case["op"] == "residual":
        return _residual_exact(s)
    ts = [t.double() for t in s["tensors"]]
    norm = torch.stack([(t * t).sum() if case["kind"] == "2" else t.abs().max() for t in ts])
    norm = norm.sum().sqrt() if case["kind"] == "2" else norm.max()
    factor = torch.where(norm + 1e-6 > s["max_norm"], s["max_norm"] / (norm + 1e-6), torch.ones_like(norm))
    return {"norm": norm, "out": {k: v.double() * factor for k, v in s["flat"].items()}}
