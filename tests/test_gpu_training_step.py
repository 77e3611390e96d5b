"""The example's prompt step and training step through the operators and the
collectives, against the same model in 64 bits, whose gradients are automatic.

The projections are library products in the model's type. In binary32 a step chains
some ten sums of up to 501 products, each off by at most 501 u of its magnitudes
(u = 2^-24, 3e-5): 3e-4 of a gradient's norm is ten of them in a row. In bf16 each of as
many stages rounds to 2^-8 of its values, in both directions; a tenth of the norm is
twenty-five of them. A log probability, of order ten, follows the bounds that the
decoding steps have: 1e-4, and 0.5."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("ranks,lens,dtype", [(4, (50, 1, 77), "f32"), (2, (130,), "f32"), (8, (3, 0, 200, 31), "bf16"),
                                              (2, (1,), "bf16")])
@pytest.mark.parametrize("graph", [True, False])
def test_training_step(ranks, lens, dtype, graph):
    import tensor_parallel_step as example
    f32 = dtype == "f32"
    worst, off = example.train(ranks, lens, torch.float32 if f32 else torch.bfloat16, graph=graph)
    assert worst <= (1e-4 if f32 else 0.5)
    if sum(max(0, n - 1) for n in lens) == 0:
        return  # nothing to learn from: every gradient is 0
    assert max(off.values()) <= (3e-4 if f32 else 0.1), off


@pytest.mark.parametrize("ranks,lens,dtype", [(4, (1, 40, 17), "f32"), (8, (100, 1, 16, 15, 33), "bf16"), (2, (90,), "f32")])
def test_prompts_then_decoding(ranks, lens, dtype):
    import tensor_parallel_step as example
    words = ranks * example.WORDS
    prompts = [[(11 * i + 5 * r + 2) % words for i in range(n)] for r, n in enumerate(lens)]
    f32 = dtype == "f32"
    decoder, worst = example.run(ranks, len(lens), 6, torch.float32 if f32 else torch.bfloat16, prompts=prompts)
    assert worst <= (1e-4 if f32 else 0.5)
    assert decoder.lens.tolist() == [n + 6 for n in lens]
