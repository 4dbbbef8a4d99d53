"""The operators around the layer at the ends of their ranges, on a GB300."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    from co_folding_pair_gb300 import pair_ops
    return pair_ops


@pytest.mark.parametrize("dt", [BF, F32])
def test_head_planes_smaller_than_a_group(P, dt):
    """Planes of one to nine elements, several of them within 16 bytes; small whole numbers, so sums are exact."""
    r = P.RelPos("linear", 3)
    for I, J in [(1, 1), (1, 2), (3, 1), (2, 2), (1, 5), (2, 3), (7, 1), (2, 4), (3, 3)]:
        for B in (1, 2, 3):
            for D in (1, 2, 3, 5, 9):
                qp = torch.arange(B * I, device="cuda").int().view(B, I) % 5
                kp = torch.arange(B * J, device="cuda").int().view(B, J) % 7
                b = (qp[:, :, None] - kp[:, None, :]).clamp(-3, 3).long() + 3
                dout = (torch.arange(B * D * I * J, device="cuda") % 9 - 4).view(B, D, I, J).to(dt)
                want = torch.zeros(7, D, device="cuda").index_add_(0, b.reshape(-1), dout.float().permute(0, 2, 3, 1).reshape(-1, D))
                assert torch.equal(r.backward(dout, qp, kp, layout="heads"), want), (B, I, J, D)
                table = torch.arange(7 * D, device="cuda").float().view(7, D)
                got = r.forward(table, qp, kp, base=dout, layout="heads")
                assert torch.equal(got.float(), dout.float() + table[b].permute(0, 3, 1, 2)), (B, I, J, D)


def test_a_log_plan_is_ready_for_any_stream(P):
    """A plan used at once on a stream that does not wait for the one that its table was copied on."""
    pos = torch.arange(-3000, 3001, device="cuda").int()[None]
    zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    table = torch.arange(1024, dtype=F32, device="cuda")[:, None].repeat(1, 8)
    want = P.RelPos("log", 32768, 1024).forward(table, pos, zero, dtype=F32)
    torch.cuda.synchronize()
    assert want[0, :, 0, 0].unique().numel() > 700
    stream = torch.cuda.Stream()
    for _ in range(5):
        plan = P.RelPos("log", 32768, 1024)
        got = plan.forward(table, pos, zero, dtype=F32, stream=stream)
        stream.synchronize()
        assert torch.equal(got, want)
        plan.free()


@pytest.mark.parametrize("layout", ["pair", "heads"])
def test_tables_and_their_gradients_within_flat_buffers(P, layout):
    """dtable at any float, and the head layout's table at any element: as parts of one buffer of parameters."""
    r = P.RelPos("linear", 4)
    pos = torch.arange(37, device="cuda").int()[None]
    dout = torch.randn(*((1, 37, 37, 24) if layout == "pair" else (1, 24, 37, 37)), device="cuda")
    want = r.backward(dout, pos, layout=layout)
    flat = torch.full((4 * 220,), 7.0, device="cuda")
    for at in (1, 222, 443, 660):
        part = flat[at:at + 216].view(9, 24)
        r.backward(dout, pos, layout=layout, dtable=part)
        assert torch.equal(part, want)
        r.backward(dout, pos, layout=layout, dtable=part, flags=P.FLAG_ACCUMULATE)
        assert torch.equal(part, 2 * want)
        assert (flat[at + 216:at + 220] == 7.0).all() and flat[at - 1] == 7.0
    if layout == "heads":
        for dt in (BF, F32):
            flat = torch.randn(300, device="cuda").to(dt)
            for at in (1, 2, 3, 5):
                part = flat[at:at + 216].view(9, 24)
                assert torch.equal(r.forward(part, pos, layout=layout, dtype=dt), r.forward(part.clone(), pos, layout=layout, dtype=dt))


@pytest.mark.parametrize("layout,D,dt", [("heads", 2, BF), ("heads", 2, F32), ("pair", 8, BF)])
def test_the_most_pairs(P, layout, D, dt):
    """One query and 2^31 - 1 keys: positions in a plane reach past 31 bits where a tile, or a plane's early elements,
    go past its end."""
    n = 2**31 - 1
    r = P.RelPos("linear", 32)
    qp, kp = torch.full((1, 1), n - 6, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")[None]
    table = torch.randn(65, D, device="cuda").to(dt)
    out = r.forward(table, qp, kp, layout=layout, dtype=dt)
    view = out.view(D, n) if layout == "heads" else out.view(n, D).t()
    last = 100
    b = ((n - 6) - torch.arange(n - last, n, device="cuda")).clamp(-32, 32) + 32
    assert torch.equal(view[:, n - last:], table[b].t())
    for c in range(D):
        assert not (view[c, :n - last] != table[64, c]).any()
    out.zero_()
    for j, v in ((n - 1, 1.0), (n - 6, 2.0), (0, 4.0)):
        view[:, j] = v
    want = torch.zeros(65, D, device="cuda")
    want[27], want[32], want[64] = 1.0, 2.0, 4.0
    assert torch.equal(r.backward(out, qp, kp, layout=layout), want)
