"""Zero points over their whole range, 0 to 127, in the int4 product.

x (q - z) has at most 2 + 7 bits here and sums of up to 1440 of them times scales of 2^-2 to 2 stay
below 2^24 units of 2^-2: every sum is exact in fp32, and results are equal to those in 64 bits."""

import numpy as np
import pytest
import torch

from test_int4_product import call, moe, product


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K,group", [((1,), 40, 128, 128), ((3, 0, 17), 264, 288, 32), ((40, 9), 48, 1440, 32),
                                              ((8, 5), 72, 576, 64)])
def test_every_zero_point(counts, N, K, group):
    m = moe()
    E, rng = len(counts), np.random.default_rng(11)
    bounds = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    codes = rng.integers(0, 16, (E, N, K)).astype(np.uint8)
    zeros = rng.permutation(np.arange(E * N * (K // group)) % 128).reshape(E, N, K // group).astype(np.uint8)
    scales = 2.0 ** rng.integers(-2, 2, (E, N, K // group))
    x = rng.integers(-2, 3, (bounds[-1], K)).astype(np.float64)
    w = (codes - np.repeat(zeros.astype(np.float64), group, -1)) * np.repeat(scales, group, -1)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    packed = m.pack_weights_int4(cu(codes[..., 0::2] + 16 * codes[..., 1::2]), cu(scales).bfloat16(), cu(zeros),
                                 m.MOE_EPI_NONE)
    args = [cu(x).bfloat16(), cu(bounds), torch.arange(E, dtype=torch.int32, device="cuda"), packed]
    want, _ = product(x, w, bounds, np.arange(E), 0)
    assert zeros.max() == 127 or zeros.size < 128
    assert np.array_equal(call(args, int(bounds[-1])).cpu().numpy(), want)
