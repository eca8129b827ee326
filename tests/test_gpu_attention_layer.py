"""The operators together, as the example runs them: a token's attention over the paged cache is
the same token's attention over the whole sequence at once.

Both round their weights and outputs to bf16 (unit 2^-8, twice, independently: 4 units of the
output's norm bound the 2-norm difference generously); an int8 cache adds half a step of each
row's scale, max / 254, on keys and values, 2% of a row of normal values at worst."""
import pytest
import torch

import int8_weight_quantized_gb300 as ck
from int8_weight_quantized_gb300 import attention_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,steps,window,sinks", [(1, 1, 0, 0), (37, 3, 0, 0), (700, 5, 0, 0), (700, 5, 128, 4),
                                                       (300, 2, 16, 0)])
@pytest.mark.parametrize("cache,bound", [(torch.bfloat16, 4 * 2.0 ** -8), (torch.int8, 0.04)])
def test_cached_attention_is_the_whole_sequences(tokens, steps, window, sinks, cache, bound):
    _, _, off = attention_layer.run(tokens, steps, cache, window, sinks, hidden=512, q_heads=8, kv_heads=2)
    assert off <= bound
    assert ck.ck_device_error() == 0


def test_batched_prompts_match_single_ones():
    layer = attention_layer.AttentionLayer(512, 8, 2, 64, 300, batch=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    lengths = [41, 300, 7]
    x = torch.randn((sum(lengths), 512), generator=g, device="cuda").to(torch.bfloat16)
    y = layer.prompt(x, lengths)
    lo = 0
    for n in lengths:
        alone = layer.prompt(x[lo:lo + n], [n])
        assert torch.equal(y[lo:lo + n], alone)
        lo += n
    out, _ = layer.step(x[:3], torch.tensor([41, 299, 7], device="cuda"))
    assert out.shape == (3, 512) and out.isfinite().all()


def test_command_line(capsys):
    attention_layer.main(["--tokens", "64", "--steps", "2", "--cache", "int8", "--window", "32", "--sinks", "4"])
    assert "prompt of 64 tokens" in capsys.readouterr().out
