"""beam_select where most tokens have a very low logit in place of -inf, and fewer others are left than are wanted: the
low ones are level, as they are in 64 bits, and the lowest w V + v of them follow."""

import numpy as np
import pytest

from tests.test_gpu_beam_select import bf16, check

pytestmark = pytest.mark.gpu

LOWEST = {False: -3.3895313892515355e38, True: -3.4028234663852886e38}


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("low", ["lowest", -1e30, -1e18])
@pytest.mark.parametrize("N,W,V,k,left", [(1, 4, 32, 8, 1), (3, 5, 1000, 16, 2), (2, 8, 9, 30, 3), (5, 2, 50001, 2, 0), (2, 64, 2048, 64, 0),
                                          (40, 3, 2049, 7, 1)])
def test_low_logits_are_level(fp32, low, N, W, V, k, left):
    rng = np.random.default_rng(V + k)
    x = np.full((N, W, V), LOWEST[fp32] if low == "lowest" else float(bf16(np.asarray([low]))[0]), np.float32)
    for n in range(N):
        for w in range(W):
            at = rng.choice(V, left if w else max(left, 1), replace=False)
            x[n, w, at] = bf16(rng.standard_normal(len(at)) * 2 + 3 * w)
    check(x, -10 * rng.random((N, W)), k, fp32=fp32)
    check(x, -10 * rng.random((N, W)), k, rng.random((N, W)) < 0.3, 1, fp32)


def test_scores_count_beside_masks_that_64_bits_hold_them_with():
    rng = np.random.default_rng(0)
    for low in (-100.0, -1e4, -1e6):
        x = np.full((2, 4, 300), low, np.float32)
        x[:, :, 5] = 1.0
        check(bf16(x), -10 * rng.random((2, 4)), 12)
