"""One token whose logits tie within the choice, many times over beside other work: the same choice and the same bits.

The choice and the weights are exact (equal logits go to the lower expert, equal values have equal weights); the output is
held to the bounds of test_gpu_few.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_few import B, Layer  # noqa: E402, F401


@pytest.mark.parametrize("E,k,d,f,typ", [(128, 8, 2048, 704, 0), (200, 8, 512, 192, 1), (17, 5, 256, 64, 0), (256, 6, 1024, 320, 1)])
def test_a_tied_choice_in_every_run(B, E, k, d, f, typ):
    tied = torch.zeros(1, E)
    tied[0, E - 3] = 1.0  # the first is alone, the others tie
    for logits in (tied, torch.zeros(1, E), torch.arange(E).float()[None] // 2):
        layer = Layer(B, 1, d, f, E, k, 64, 64, 0, 0, typ, seed=E, logits=logits.cuda().contiguous())
        first = layer.run()
        layer.check(first)
        ws = [torch.empty(B.moe_w4a16_few_workspace_bytes(layer.shape), dtype=torch.uint8, device="cuda") for _ in range(2)]
        outs = [[torch.empty_like(t) for t in first] for _ in range(100)]
        streams = [torch.cuda.Stream() for _ in ws]
        torch.cuda.synchronize()
        for i, (idx, tw, out) in enumerate(outs):  # two streams, so that CTAs of two calls share an SM
            B.moe_w4a16_few(layer.shape, typ, layer.x, layer.logits, layer.dev.gate_up, layer.dev.down, layer.residual,
                            idx, tw, out, ws[i % 2], streams[i % 2])
        torch.cuda.synchronize()
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, first))
