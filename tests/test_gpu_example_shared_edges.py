"""The shared-prompt example refuses what does not fit, and says so when a pool has
no page left. (A page looked up past a row's last one would end the process in a
failed device assertion, so nothing may be enqueued for such a prompt.)"""
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


def test_a_prompt_that_finds_no_pages_is_refused():
    import shared_prompt as S
    model = _model()
    cache = S.PoolCache(model.attn, 1, 2, 64, pages=2)
    with pytest.raises(RuntimeError, match="no free page"):
        S.sample(model, cache, _rows(33), 2)
    assert not cache.held.any()


def test_samples_that_find_no_page_say_so_and_go_on_when_there_is_one():
    """The token is taken again by the next call. The same steps with pages enough
    give the same rows (the same calls on other pages; the bound is that of the
    example's other test, 8 * 2^-8 of a row's norm)."""
    import shared_prompt as S
    model, prompt, steps = _model(), _rows(32), [_rows(3) for _ in range(20)]
    outs = []
    for pages in (5, 40):
        cache = S.PoolCache(model.attn, 1, 4, 64, pages=pages)
        row = torch.tensor([3], dtype=torch.int32, device="cuda")
        cache.reserve(row, row * 0, row * 0 + 16)              # another request's page
        _, samples = S.sample(model, cache, prompt, 3)         # and the prompt's two
        if pages == 5:
            for _ in range(2):                                 # three pages, and two are free
                with pytest.raises(RuntimeError, match="no free page"):
                    samples.step(steps[0])
                assert samples.host_len == 32 and samples.lens.tolist() == [32] * 3
            cache.release(row)
        outs.append([samples.step(x).clone() for x in steps[:16]])
        if pages == 5:
            with pytest.raises(RuntimeError, match="no free page"):
                samples.step(steps[16])
    for a, b in zip(*outs):
        err = (a.float() - b.float()).norm(dim=-1) / b.float().norm(dim=-1)
        assert (err <= 8 * 2.0 ** -8).all()
