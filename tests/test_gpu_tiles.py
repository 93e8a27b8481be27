"""Sizes that take the tile shapes of the shared product which small shapes do not reach, for
the layer with adapters and for the head, against the float64 oracle: the checks and
bounds are those of their own tests.

The shape goes by the rounds that 256 x 256 and 128 x 128 tiles make of the 256 compute units:
128-wide tiles with two stages serve about 257 to 512 of them."""

import pytest

from tests import test_gpu_adapters as adapters
from tests import test_gpu_head as head

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["mixed", "runs", "one"])
@pytest.mark.parametrize("M,N,K,n,r", [(1152, 4096, 64, 3, 16), (1150, 4072, 192, 5, 24), (330, 11008, 128, 2, 8)])
def test_adapters_forward_on_many_128_wide_tiles(M, N, K, n, r, kind):
    c, dY = adapters._case(M, N, K, n, r, seed=M)
    adapters._check(c, dY, adapters._index(kind, M, n, seed=2))


@pytest.mark.parametrize("kind", ["mixed", "runs", "one"])
@pytest.mark.parametrize("M,N,K,n,r", [(1152, 64, 4096, 3, 16), (1150, 200, 4032, 5, 24), (330, 136, 11008, 2, 72)])
def test_adapters_backward_on_many_128_wide_tiles(M, N, K, n, r, kind):
    c, dY = adapters._case(M, N, K, n, r, seed=M)
    adapters._check(c, dY, adapters._index(kind, M, n, seed=3))


@pytest.mark.parametrize("M,V,K", [(600, 8000, 128), (1100, 4100, 192)])
def test_head_on_many_128_wide_tiles(M, V, K):
    """The logits, with and without the gradient."""
    head._check(*head._case(M, V, K, seed=M, whole=True), whole=True)


@pytest.mark.parametrize("M,V,K", [(20, 4136, 4096), (130, 8200, 2112)])
def test_gradient_of_a_wide_head_on_256_wide_tiles(M, V, K):
    head._check(*head._case(M, V, K, seed=M, whole=True), whole=True)
