"""How many digits the whole layer for a few tokens keeps before its one rounding to the type.

A second call whose residual is the first one's output with its sign turned gives what that rounding took away, to as
many digits again: first + second is the output before it. Its difference from 64 bits, over its norm, is at most 2^-18.

Derivation. A group's sum is made by up to eight matrix instructions, each of which leaves off at most a step of what
it keeps, 24 bits below its largest product. The sum of the codes with their bias (bf16: 16 + q) or without (fp16) is R =
5.2 or 2 times that of the weights it stands for, for even codes and zero-points near their middle. Half a step on
average, of partial sums that grow as the root of their number, comes to 8 x 2/3 x 2^-24 R: 2^-19.2 of a group's sum
(bf16) and 2^-20.6 (fp16; with up to four leading zeros of a code's place, at random, 2^-19). Group sums of a row add as
their root, so a product is off by as much as its groups; the layer has three, two of them side by side, the activation
passing on 1.13: a factor of 1.8 at random, 2^-18.2 at most. The activation (2^-21) and h (fp16 2^-23, bf16 two roundings of
2^-9, at random 2^-19.8) add as a root: below 2^-18.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_few import B, Layer  # noqa: E402, F401


@pytest.mark.parametrize("case", [
    (1, 2048, 704, 128, 8, 64, 64, 0, 0, 0), (4, 2048, 704, 128, 8, 128, 64, 1, 0, 1), (16, 2048, 704, 128, 8, 64, 64, 0, 0, 0),
    (7, 1152, 448, 60, 3, 32, 64, 2, 1, 1), (8, 2048, 704, 128, 8, 128, 64, 2, 0, 0), (32, 1024, 512, 32, 4, 64, 128, 1, 0, 1),
    (3, 512, 256, 16, 2, 32, 32, 0, 0, 1), (1, 4096, 832, 16, 4, 128, 32, 1, 1, 0)], ids=lambda c: "-".join(map(str, c)))
def test_digits_before_the_rounding(B, case):
    layer = Layer(B, *case, seed=sum(case), residual=False)
    first = layer.run()[2]
    want = layer.want()[2]
    layer.residual = -first
    second = layer.run()[2]
    whole = first.double() + second.double()
    assert float((whole - want).norm() / want.norm()) <= 2.0 ** -18
