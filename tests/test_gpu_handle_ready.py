"""A layer's handle may be used on any stream as soon as it is made, on a GB300."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_handle_is_ready_for_any_stream():
    """A handle used at once on a stream that does not wait for the one that its weights were copied on."""
    from co_folding_pair_gb300 import synthetic as S
    from co_folding_pair_gb300 import trimul as T

    z, mask, params = S.make_case(S.custom(1, 40, 256, 256, seed=7))[:3]
    z, mask = z.cuda(), None if mask is None else mask.cuda()
    want = T.TriMul(params)(z, mask, flags=T.FLAG_CHECK)
    stream = torch.cuda.Stream()
    for _ in range(5):
        out = torch.empty_like(z)
        torch.cuda.synchronize()
        layer = T.TriMul(params)
        layer(z, mask, out=out, stream=stream)
        stream.synchronize()
        assert torch.equal(out, want)
        layer.free()
