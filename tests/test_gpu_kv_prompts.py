"""Attention of many query rows (prompts and chunks of them) over the paged 4-bit
cache against float64, alone and beside single rows in one call."""

import pytest

from tests.test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G,heads,kv_heads", [(64, 64, 8, 1), (128, 32, 10, 2), (128, 128, 4, 4), (256, 64, 4, 1), (256, 32, 3, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_prompts(D, G, heads, kv_heads, window, sinks):
    # whole prompts, chunks after cached tokens, and single rows in one call
    ctx, rows = [1, 17, 129, 300, 333, 40, 64], [1, 17, 129, 70, 20, 40, 1]
    Case(ctx, rows, heads, kv_heads, D, G, 64, seed=D).check(window, sinks)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("ctx,rows", [(257, 257), (640, 129), (1000, 33)])
def test_prompt_page_sizes(page, ctx, rows):
    Case([ctx], [rows], 4, 1, 128, 64, page, seed=page).check()


def test_many_query_heads_in_a_prompt():
    Case([70, 150], [70, 30], 40, 2, 64, 64, 32, seed=3).check()


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 1), (64, 4), (100, 70), (5000, 3)])
def test_sixteen_rows_with_window(window, sinks):
    ctx = [16, 17, 90, 80, 400]
    Case(ctx, [16] * 5, 4, 2, 128, 64, 16, seed=16 + window).check(window, sinks)


def test_queries_of_zeros():
    # every visible key weighs the same, also for the first rows, which see little
    import numpy as np

    for rows in (1, 90):
        c = Case([90], [rows], 2, 1, 128, 64, 16, seed=21)
        c.q[:] = 0
        c.q_d.zero_()
        for window in (0, 5):
            c.check(window=window)
    c = Case([90], [90], 2, 1, 128, 64, 16, seed=22)
    k = np.asarray(c.cache.k[:, :, :], dtype=np.float32) * np.float32(2.0 ** -90)
    c.cache.write(np.arange(c.cache.n_pages * 16), k, np.asarray(c.cache.v, dtype=np.float32))
    import torch

    c.pages_d = torch.from_numpy(c.cache.bytes).cuda()
    c.check()
