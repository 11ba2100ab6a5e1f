"""GPU NVFP4 matrix products at every tile width, one CTA and pairs of CTAs, dense
and grouped, against float64: ragged rows and channels, K in every way that its
scales are read, several turns of scales, with and without a residual."""
import numpy as np
import pytest

from matmul_tiles import DENSE, GROUPED, KS
from test_gpu_matmul import Case

pytestmark = pytest.mark.gpu

BF16 = pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])


def _takes(lib, width, M, N, K, E=1):
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert lib.matmul_tile(M, N, K, E, sms) == width


@BF16
@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("width,M,N", DENSE)
def test_dense_widths(lib, width, M, N, K, bf16):
    _takes(lib, width, M, N, K)
    residual = (M + K // 32) % 2 == 0
    Case(lib, width + K, M, N, K, w_tiles=False, bf16=bf16, residual=residual,
         rpg=0 if residual else 37, act="none" if residual else "gelu",
         pad=N % 8 // 4).run().check(f"{M}x{N}x{K}")


@BF16
@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("width,T,N,E", GROUPED)
def test_grouped_widths(lib, width, T, N, E, K, bf16):
    """A group of one row, an empty one, the others, and rows outside all of them."""
    _takes(lib, width, T, N, K, E)
    rng = np.random.default_rng(T + K)
    offsets = [4, 5, 5, *np.sort(rng.integers(6, T - 9, E - 3)), T - 9]
    residual = (T + K // 32) % 2 == 0
    Case(lib, width + K, T, N, K, w_tiles=N % 16 == 0, bf16=bf16, offsets=[int(o) for o in offsets],
         residual=residual, rpg=1 if residual else 0, act="silu").run().check(f"{T}x{N}x{K}")


@BF16
@pytest.mark.parametrize("K", KS)
def test_pairs_with_both_operands_in_tiles(lib, K, bf16):
    M, N = 704, 4240
    _takes(lib, 192, M, N, K)
    Case(lib, 800 + K, M, N, K, x_tiles=True, bf16=bf16, residual=True).run().check(str(K))
