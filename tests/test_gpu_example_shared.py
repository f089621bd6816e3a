"""The shared-prompt example: samples forked from one prompt decode as if each had
run the prompt itself.

The same codes are stored either way; attention is summed in another order (the
prefix for all samples, or each request by itself), and the prompt's last tokens go
through other kernels. The bound is test_gpu_example's: two layers of two
sub-layers, each a rounding of bf16 per way: 8 * 2^-8 of a row's norm. (A sample
that read another one's token would be off by its own size.) It holds where the
layers are continuous, so that both of two experts are chosen here: the second and
third of eight logits of 360 tokens come as near as 0.0002, and a rounding of the
norm (2^-8 of a row of norm 32, against router rows of norm 1) moves them by more."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,tokens", [(3, 77), (20, 130), (1, 40)])
def test_samples_equal_requests_of_their_own(n, tokens):
    import decoder_layers as E
    import shared_prompt as S
    torch.manual_seed(1)
    model = E.Decoder(experts=2)
    prompt = torch.randn(tokens, 1024, device="cuda").bfloat16()
    steps = [torch.randn(n, 1024, device="cuda").bfloat16() for _ in range(18)]
    cache = S.PoolCache(model.attn, 2, n + 2, 256, pages=n * 4 + 16)
    _, samples = S.sample(model, cache, prompt, n)
    got = [samples.step(x).clone() for x in steps]
    cache.check()
    whole = E.Cache(model.attn, 2, n, 256)
    E.prompt(model, whole, [prompt] * n)
    alone = E.DecodeGraph(model, whole, [tokens] * n)
    for i, x in enumerate(steps):
        want = alone.step(x)
        err = (got[i].float() - want.float()).norm(dim=-1) / want.float().norm(dim=-1)
        assert (err <= 8 * 2.0 ** -8).all(), (i, err)
    # the prompt's whole pages once, the others by sample
    page = model.attn.page_size
    own = -(-(tokens + len(steps)) // page) - tokens // page
    assert int((cache.refs > 0).sum()) == tokens // page + n * own
    assert (cache.refs[cache.page_table[:n, :tokens // page].long()] == n).all()


def test_samples_stop_at_the_end_of_their_room():
    import decoder_layers as E
    import shared_prompt as S
    model = E.Decoder(layers=1, hidden=256, heads=4, kv_heads=2, experts=4, intermediate=128)
    cache = S.PoolCache(model.attn, 1, 2, 32, pages=8)
    _, samples = S.sample(model, cache, torch.randn(31, 256, device="cuda").bfloat16(), 2)
    x = torch.randn(2, 256, device="cuda").bfloat16()
    assert torch.isfinite(samples.step(x).float()).all()
    with pytest.raises(ValueError, match="the cache holds"):
        samples.step(x)
    cache.check()


def test_example_runs():
    import shared_prompt
    shared_prompt.main()
