"""The attention block between the framework's own quantizers and GEMMs, as examples/attention_block.py runs it."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

puro = pytest.importorskip("blockwise_fp8_gemm_act_amd")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4)])
@pytest.mark.parametrize("tokens,sequences", [(256, 1), (480, 3)])
def test_training_step_and_decoding_loop(tokens, sequences, window, sinks):
    import attention_block as ex
    block = ex.Block(window=window, sinks=sinks, positions=512)
    errors, x, y, *_ = ex.train(block, tokens, sequences)
    # bf16 roundings of q, k, P, o (2^-8 at most each, independent): far below their sum.  dx passes the FP8 quantizer
    # on both sides, whose codes (3 mantissa bits) differ where an input difference crosses a rounding boundary.
    assert errors["o"] < 4 * 2.0 ** -8
    assert errors["dx"] < 2.0 ** -4
    # the FP8 activations of o differ in the same way between the two passes
    assert ex.decode(block, x, y, sequences) < 2.0 ** -4


def test_values_left_in_the_projection_output():
    """Gradients of queries, keys and values written side by side into one tensor, nothing else touched."""
    import attention_block as ex
    block = ex.Block(positions=256)
    _, x, y, pos, starts, dy = ex.train(block, 256, 1)
    _, saved = block.forward(x, pos, starts)
    a, b = block.backward(dy, saved), block.backward(dy, saved)
    for p, q in zip(a, b):
        assert torch.equal(p, q) and bool(torch.isfinite(p.float()).all())
