"""A block's training step as it is used, on a GB300: a TriMul layer, its residual step, a transition of two linear layers in 8
bits, their gradients, the norm of all of them, AdamW, and the new weights in 8 bits again.
"""

import numpy as np
import pytest
import torch
import torch.nn.functional as Fn

from oracle import pair_ops_oracle as OP
from oracle import train_ops_oracle as O
from oracle import trimul_backward as OB
from oracle import trimul_oracle as OT

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
N, D, HIDDEN = 24, 32, 136
U = 2.0**-24


def f64(t):
    return t.detach().double().cpu().numpy()


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


class Block:
    """z1, h = z + channel LayerNorm(TriMul(z)), LayerNorm(z1);  z2 = z1 + W2 silu(W1 h + b1) + b2."""

    def __init__(self, states):
        from co_folding_pair_gb300 import pair_ops as P
        from co_folding_pair_gb300 import synthetic as S
        from co_folding_pair_gb300 import train_ops as R
        from co_folding_pair_gb300 import trimul as T

        self.P, self.T = P, T
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
        layer = S.make_case(S.custom(1, N, D, D, seed=91))[2]
        self.p = {"layer." + k: layer[k].to("cuda", F32).contiguous() for k in T.GRAD_NAMES}
        self.other = {k: v for k, v in layer.items() if k not in T.GRAD_NAMES}
        for k in P.RESIDUAL_PARAMS:
            self.p["step." + k] = 1.0 * k.endswith("gamma") + 0.1 * randn(D) + 0.5 * (k == "channel")
        self.p.update(w1=randn(HIDDEN, D) / D**0.5, b1=0.1 * randn(HIDDEN), w2=randn(D, HIDDEN) / HIDDEN**0.5, b2=0.1 * randn(D))
        self.w = {k: self.p[k].to(BF) for k in ("w1", "w2")}
        self.z, self.dout = randn(1, N, N, D).to(BF), randn(1, N, N, D).to(BF)
        self.make_layer()
        self.first = P.Residual({k: self.p["step." + k] for k in P.RESIDUAL_PARAMS}, post_norm="layer", pre_norm="layer")
        self.second = P.Residual()
        self.l1, self.l2 = R.Linear8(self.w["w1"], self.p["b1"]), R.Linear8(self.w["w2"], self.p["b2"])
        self.opt = R.AdamW(self.p, lr=1e-2, weight_decay=[0.1 if v.dim() == 2 else 0.0 for v in self.p.values()], states=states,
                           copies=[self.w.get(k) for k in self.p], seed=3)

    def make_layer(self):
        self.layer = self.T.TriMul({**self.other, **{k[6:]: v for k, v in self.p.items() if k.startswith("layer.")}}, "outgoing")

    def forward(self):
        u = self.layer(self.z)
        z1, h = self.first.forward(self.z, u)
        a = self.l1(h)
        s = Fn.silu(a.float()).to(BF)
        z2, _ = self.second.forward(z1, self.l2(s))
        return u, z1, h, a, s, z2

    def backward(self, u, z1, h, a, s):
        down = self.second.backward(z1, z1, self.dout)  # (its update's values do not enter: no norm, no gate)
        g2 = self.l2.backward(s, down["du"])
        x = a.float()
        sig = torch.sigmoid(x)
        da = (g2["dx"].float() * sig * (1 + x * (1 - sig))).to(BF)
        g1 = self.l1.backward(h, da)
        up = self.first.backward(self.z, u, down["dx"], dnormed=g1["dx"])
        dz, lay = self.T.trimul_backward(self.layer.handle, self.z, None, up["du"], "outgoing")
        grads = {**{"layer." + k: lay[k] for k in self.T.GRAD_NAMES}, **{"step." + k: v for k, v in up["grads"].items()},
                 "w1": g1["dw"], "b1": g1["dbias"], "w2": g2["dw"], "b2": g2["dbias"]}
        return up["dx"].float() + dz.float(), {k: grads[k] for k in self.p}, da, down["du"]

    def update(self, grads):
        gs = self.P.GradSet(grads)
        norm = gs.norm()
        self.opt.step(gs, norm=norm, max_norm=1.0)
        self.l1.pack(self.w["w1"])
        self.l2.pack(self.w["w2"])
        return norm


def definition(b, p):
    """z2, the gradients and dz in 64 bits, nothing rounded."""
    z, dout = f64(b.z), f64(b.dout)
    step = {k[5:]: v for k, v in p.items() if k.startswith("step.")}
    lay = {**{k: f64(v) for k, v in b.other.items()}, **{k[6:]: v for k, v in p.items() if k.startswith("layer.")}}
    u = OT.trimul_forward(z, None, lay, "outgoing")
    z1, h = OP.residual_forward(z, u, step, post="layer", pre="layer")
    a = h @ p["w1"].T + p["b1"]
    sig = 1 / (1 + np.exp(-a))
    s = a * sig
    z2 = z1 + s @ p["w2"].T + p["b2"]
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    da = (dout @ p["w2"]) * sig * (1 + a * (1 - sig))
    dx, du, _, dp = OP.residual_backward(z, u, dout, step, post="layer", pre="layer", dnormed=da @ p["w1"])
    back = OB.trimul_backward(z, None, lay, "outgoing", du)
    grads = {**{"layer." + k: back[k] for k in b.T.GRAD_NAMES}, **{"step." + k: dp[k][0] for k in step},
             "w1": flat(da).T @ flat(h), "b1": flat(da).sum(0), "w2": flat(dout).T @ flat(s), "b2": flat(dout).sum(0)}
    return z2, grads, dx + back["dz"]


@pytest.mark.parametrize("states", ["float32", "8bit"])
def test_a_block_and_its_training_step(states):
    """The linear layers against their own definition at the inputs that they get, bit of rounding by bit; the whole against 64 bits
    without roundings; the norm and the optimiser's step from the gradients that they get.

    An e4m3 number is off by at most 2^-4, evenly spread by 2^-4 / 3^0.5 = 0.036.  z2 has two rounded operands a product,
    two products deep, 0.072 of the transition's part of z2; the gradients of w1 and of all above have six on their way (h and W1
    in a, dout and W2, then da and h or W1): 0.09 of the transition's part.  TriMul's own bounds are 5e-3 and 1.5e-2, bf16's
    2^-8 a tensor: 0.12 in all."""
    b = Block(states)
    p0 = {k: f64(v) for k, v in b.p.items()}
    p0.update({k: f64(v) for k, v in b.w.items()})  # what the layers multiply by
    u, z1, h, a, s, z2 = b.forward()
    dz, grads, da, do = b.backward(u, z1, h, a, s)
    flat = lambda t: f64(t).reshape(-1, t.shape[-1])  # noqa: E731

    def check(y, w, bias):  # of h; four sums of up to 32 products, the bias below one
        ref, mag = O.linear8(flat(h), w, bias)
        tol = 12 * U * (mag + 1)
        assert (np.abs(flat(y) - ref) <= 2.0**-8 * (np.abs(ref) + tol) + tol).all()

    check(a, p0["w1"], p0["b1"])
    for x, dy, w, bias in ((s, do, "w2", "b2"), (h, da, "w1", "b1")):
        _, (dw, dwm), (db, dbm) = O.linear8_backward(flat(x), p0[w], flat(dy))
        assert (np.abs(f64(grads[w]) - dw) <= 200 * U * dwm).all() and (np.abs(f64(grads[bias]) - db) <= 850 * U * dbm).all()
    ref_z2, ref, ref_dz = definition(b, p0)
    assert rel(f64(z2), ref_z2) < 0.12 and rel(f64(dz), ref_dz) < 0.12
    for k in ref:
        assert rel(f64(grads[k]).reshape(ref[k].shape), ref[k]) < 0.12, k

    norm = float(b.update(grads))
    total = float(OP.grad_norm([f64(v) for v in grads.values()]))
    assert abs(norm - total) <= 64 * U * total
    for k, before in p0.items():
        if k in b.w:
            continue
        g = f64(grads[k]).reshape(before.shape)
        want = O.adamw(before, g, 0.0 * g, 0.0 * g, 1, 1e-2, (0.9, 0.999), 1e-8, 0.1 if before.ndim == 2 else 0.0, O.clip_factor(norm, 1.0))
        tol = 40 * U * want[4] + 6 * U * np.abs(before)
        assert (np.abs(f64(b.p[k]) - want[0]) <= tol + U * (np.abs(want[0]) + tol)).all(), k
    for k in b.w:
        assert torch.equal(b.w[k], b.p[k].to(BF))  # the copies that were packed
    check(b.l1(h), f64(b.w["w1"]), f64(b.p["b1"]))


@pytest.mark.parametrize("states", ["float32", "8bit"])
def test_captured_steps_are_those_run_one_by_one(states):
    """The transition's part of the step (the layer's weights are laid out on the host's call), three times: captured and replayed,
    and run.  One stream, nothing else on it: the same bits."""
    def step(b, u):
        z1, h = b.first.forward(b.z, u)
        a = b.l1(h)
        s = Fn.silu(a.float()).to(BF)
        _, grads, _, _ = b.backward(u, z1, h, a, s)
        return b.update(grads)

    run, cap = Block(states), Block(states)
    u = run.layer(run.z)
    norms = [float(step(run, u)) for _ in range(4)]
    first = float(step(cap, u))  # what is made at first use is made before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step(cap, u)
    got = [first]
    for _ in range(3):
        graph.replay()
        got.append(float(norm))
    assert got == norms
    for k in run.p:
        assert torch.equal(run.p[k], cap.p[k]), k
    for k in run.opt.state:
        x, y = (o.state[k].view(torch.uint8) if o.state[k].element_size() == 1 else o.state[k] for o in (run.opt, cap.opt))
        assert torch.equal(x, y), k
    assert int(run.opt.state["count"]) == 4
    assert torch.equal(run.l1(run.z), cap.l1(cap.z))  # the weights as they were packed (bytes between the numbers are nobody's)
