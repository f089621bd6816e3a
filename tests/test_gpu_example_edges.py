"""The decoder-layer example refuses requests that outgrow their pages or the
rotary table. (A page looked up past a request's last one would end the process
in a failed device assertion, so nothing may be enqueued.)"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("positions,pages", [(4096, 32), (24, 4096)])
def test_requests_stop_at_the_end_of_their_room(positions, pages):
    import decoder_layers as E
    model = E.Decoder(layers=1, hidden=256, heads=4, kv_heads=2, experts=4, intermediate=128,
                      max_positions=positions)
    cache = E.Cache(model.attn, 1, 2, pages)
    room = min(positions, pages)
    assert cache.tokens == room
    xs = [torch.randn(n, 256, device="cuda").bfloat16() for n in (room - 2, 3)]
    with pytest.raises(ValueError, match="the cache holds"):
        E.prompt(model, cache, [torch.randn(room + 1, 256, device="cuda").bfloat16(), xs[1]])
    E.prompt(model, cache, xs)
    graph = E.DecodeGraph(model, cache, [room - 2, 3])
    x = torch.randn(2, 256, device="cuda").bfloat16()
    for _ in range(2):
        assert torch.isfinite(graph.step(x).float()).all()
    with pytest.raises(ValueError, match="the cache holds"):
        graph.step(x)
    with pytest.raises(ValueError, match="the cache holds"):
        E.DecodeGraph(model, cache, [room, 3])
    torch.cuda.synchronize()
    assert graph.lens.tolist() == [room, 5]
