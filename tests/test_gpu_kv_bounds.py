"""Bounds and windows that the library's 32-bit arguments cannot hold."""

import numpy as np
import pytest

from tests.test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


def test_bounds_past_32_bits_are_all_of_it():
    import affine_bit_matmul_gb300 as mxq

    c = Case([300, 90], [3, 2], 4, 2, 128, 64, 32, seed=8)
    plain = c.run()
    for window in (2 ** 32 + 5, 2 ** 31, 2 ** 63):
        got = c.run(window=window)
        assert np.array_equal(got[0], plain[0]) and got[2] == 0
    plain = c.run(max_q_len=5)  # the rows that there are
    for most in (2 ** 32 + 1, 2 ** 31):
        got = c.run(max_q_len=most)
        assert np.array_equal(got[0], plain[0]) and got[2] == 0
    some = c.run(window=9, sinks=10 ** 9)
    assert np.array_equal(c.run(window=9, sinks=2 ** 32 + 1)[0], some[0])
    for kw in (dict(window=-2 ** 32 + 5), dict(sinks=-2 ** 32 + 5), dict(max_q_len=-2 ** 32 + 5)):
        with pytest.raises((ValueError, mxq.MxqError)):
            c.run(**kw)
    # the workspace for such a bound is the one for all rows
    assert (mxq.kv_attention_workspace_bytes(40, 4, 8, 2, 128, 2 ** 32 + 1) ==
            mxq.kv_attention_workspace_bytes(40, 4, 8, 2, 128, 40))
