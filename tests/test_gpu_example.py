"""The decoder-layer example: a token decoded from the graph equals the same
token run as the last one of a prompt.

Both ways store the same codes for the earlier tokens and compute the last
token's attention by different kernels (split and prompt), whose outputs agree
to a rounding of bf16 each (2^-8), as do the MoE layers' (grouped GEMMs of
different tile widths). A rounding in layer 1 moves the inputs of layer 2 by as
much: for two layers of two sub-layers, each adding a term of the residual's
size, 8 * 2^-8 of the row's norm is an upper bound, and a wrong page, position or
mask moves the row by its whole size.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_decoded_token_equals_the_prompts_last():
    import decoder_layers as E
    torch.manual_seed(0)
    model = E.Decoder()
    lens = [140, 17, 64]
    xs = [torch.randn(n, 1024, device="cuda").bfloat16() for n in lens]
    whole = E.Cache(model.attn, 2, 3, 256)
    want = E.prompt(model, whole, xs)[torch.tensor(lens).cumsum(0) - 1]
    cache = E.Cache(model.attn, 2, 3, 256)
    E.prompt(model, cache, [x[:-2] for x in xs])
    graph = E.DecodeGraph(model, cache, [n - 2 for n in lens])
    graph.step(torch.stack([x[-2] for x in xs]))
    got = graph.step(torch.stack([x[-1] for x in xs]))
    torch.cuda.synchronize()
    assert graph.lens.tolist() == lens
    err = (got.float() - want.float()).norm(dim=-1) / want.float().norm(dim=-1)
    assert (err <= 8 * 2.0 ** -8).all(), err


def test_example_runs():
    import decoder_layers as E
    E.main()
