"""The example that runs the operators and the collectives together, against the
same steps in 64 bits. The example's projections are library products in the
model's type, so the bound is theirs: f32 sums of 256 products a layer leave a
log probability, of order ten, within 1e-4; bf16 rounds hidden values and logits
of order ten to 2^-8 of them, a few times over."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ranks,requests,steps,dtype,bound", [
    (8, 6, 40, torch.float32, 1e-4), (2, 1, 5, torch.float32, 1e-4), (4, 33, 20, torch.bfloat16, 0.5)])
def test_step(ranks, requests, steps, dtype, bound):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_parallel_step as example
    decoder, worst = example.run(ranks, requests, steps, dtype)
    assert worst <= bound
    assert decoder.lens.tolist() == [steps] * requests
    dlogits, dqkv, grads, summed = decoder.backward()
    total = grads.double().sum(0)
    size = grads.double().abs().sum(0)
    for r in range(ranks):
        assert bool(((summed[r].double() - total).abs() <= ranks * 2.0 ** -24 * size).all())
    # the logits' gradient of a row sums to zero over the vocabulary: sum(1[i == token] - p_i)
    assert float(dlogits.float().sum((0, 2)).abs().max()) <= (1e-4 if dtype == torch.float32 else 0.1)
