"""Blocks of the latent attention that many clusters share: few parts (a warp merges an
item of them) and many (eight warps do), at both sides of the bound between the two."""
import pytest

from test_gpu_latent import Case, ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,lens,H,sink", [
    ([1] * 3, [20000] * 3, 128, False),           # 25 or 26 parts a block of 128 rows
    ([1] * 2, [20000] * 2, 128, True),            # 38
    ([1, 1, 1], [30000, 24000, 9000], 16, True),  # of different lengths
    ([2], [20000], 128, False),                   # one block of 256 rows, 36
    ([2, 2], [15000, 20000], 128, True),
])
def test_blocks_of_many_parts(n, lens, H, sink, cuda_lib):
    c = Case(n, lens, H, 64, pad=1, sink=sink, seed=len(n) + H)
    c.run()
    ok()
    c.check()
