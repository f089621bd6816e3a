"""The shared-prompt example refuses what does not fit. (A page looked up past a
row's last one would end the process in a failed device assertion, so nothing may
be enqueued for such a prompt.)"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _model(**kw):
    import decoder_layers as E
    torch.manual_seed(3)
    return E.Decoder(layers=1, hidden=256, heads=4, kv_heads=2, experts=2, intermediate=128, **kw)


def _rows(n):
    return torch.randn(n, 256, device="cuda").bfloat16()


@pytest.mark.parametrize("tokens,n", [(32, 1), (33, 2), (300, 2), (5, 0), (5, 3)])
def test_prompts_and_samples_without_room_are_refused(tokens, n):
    import shared_prompt as S
    model = _model()
    cache = S.PoolCache(model.attn, 1, 2, 32, pages=8)
    with pytest.raises(ValueError, match="the cache holds"):
        S.sample(model, cache, _rows(tokens), n)
    torch.cuda.synchronize()
    assert not cache.held.any() and not cache.refs.any()
    _, samples = S.sample(model, cache, _rows(31), 2)      # the cache is as it was
    assert torch.isfinite(samples.step(_rows(2)).float()).all()


def test_prompts_end_at_the_rotary_table():
    import shared_prompt as S
    model = _model(max_positions=24)
    cache = S.PoolCache(model.attn, 1, 2, 64, pages=8)
    with pytest.raises(ValueError, match="the cache holds"):
        S.sample(model, cache, _rows(24), 1)
    assert not cache.held.any()
