"""Few experts that many of the tokens choose: more items than experts, in small layers whose down launch is planned by the
experts' number. The bounds of test_gpu_few, and a token's bits whatever the others are."""
import copy

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_few import B, Layer  # noqa: E402, F401


@pytest.mark.parametrize("typ", [0, 1], ids=["fp16", "bf16"])
@pytest.mark.parametrize("E,k,d,f,fmt", [(8, 8, 256, 128, 0), (16, 8, 512, 192, 1), (16, 4, 128, 1024, 2), (8, 2, 1024, 64, 0), (1, 1, 384, 320, 1),
                                         (9, 8, 2048, 256, 0)])
def test_shared_experts(B, E, k, d, f, fmt, typ):
    layer = Layer(B, 32, d, f, E, k, 64, 64, fmt, 0, typ, seed=E + d)
    whole = layer.run()
    layer.check(whole)
    for tokens in (slice(0, 1), slice(3, 5), slice(7, 11), slice(0, 16), slice(8, 32), slice(1, 30)):
        part = copy.copy(layer)  # in memory of their own: rows of a few logits are not aligned where they stand
        part.x, part.logits, part.residual = (t[tokens].clone() for t in (layer.x, layer.logits, layer.residual))
        assert all(torch.equal(a[tokens], b) for a, b in zip(whole, part.run()))
