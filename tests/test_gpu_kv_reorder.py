"""Reordering of the cache after a selection of beams against a plain restatement: groups, lengths,
layers, steps one after the other; its checks of entries, streams and graphs."""

import numpy as np
import pytest

from tests import kv_util as ku
from tests.test_gpu_kv_cache import SHAPES, i32

pytestmark = pytest.mark.gpu


def plain(pages, table, home, lens, parents, D, G, page):
    """numpy pages [L, P, H, block] (changed), table [S, C], ... -> table, lens."""
    N, W = parents.shape
    new, new_lens = table.copy(), lens.copy()
    per = page * D // 2, page * D // G * 4
    for g in range(N):
        a = g * W
        for i in range(W):
            new_lens[a + i] = lens[a + parents[g, i]]
        for c in range(table.shape[1]):
            keeps = {}
            for i in range(W):
                full = (c + 1) * page <= new_lens[a + i]
                if full or list(parents[g]).index(parents[g, i]) == i:
                    keeps[i] = table[a + parents[g, i], c]
            free = [p for p in home[a:a + W, c] if p not in keeps.values()]
            for i in range(W):
                if i in keeps:
                    new[a + i, c] = keeps[i]
                    continue
                new[a + i, c] = free.pop(0)
                n = new_lens[a + i] - c * page
                if 0 < n < page:
                    n = -(-n // 8) * 8
                    src, dst = table[a + parents[g, i], c], new[a + i, c]
                    at = 0
                    for size, room in ((n * D // 2, per[0]), (n * D // G * 4, per[1])) * 2:
                        pages[:, dst, :, at:at + size] = pages[:, src, :, at:at + size]
                        at += room
    return new, new_lens


class Case:
    def __init__(self, N, W, C, D, G, page, H=2, layers=1, seed=0, lens=None):
        self.rng = np.random.default_rng(seed)
        S = N * W
        self.n_pages = S * C + 3
        self.home = self.rng.permutation(self.n_pages)[:S * C].astype(np.int32).reshape(S, C)
        self.table = self.home.copy()
        self.lens = np.full(S, 0, np.int32) if lens is None else np.asarray(lens, np.int32)
        self.pages = self.rng.integers(0, 256, (layers, self.n_pages, H, ku.block_bytes(D, page, G)), dtype=np.uint8)
        self.N, self.W, self.D, self.G, self.page = N, W, D, G, page

    def parents(self):
        return self.rng.integers(0, self.W, (self.N, self.W)).astype(np.int32)

    def step(self, parents, in_place=False, squeeze=False):
        import torch

        import affine_bit_matmul_gb300 as mxq

        pages = torch.from_numpy(self.pages).cuda()
        table, lens, status = i32(self.table), i32(self.lens), i32([-1])
        kw = dict(table_out=table, lens_out=lens) if in_place else {}
        got = mxq.kv_reorder(pages[0] if squeeze else pages, table, i32(self.home), lens, i32(parents), self.D, group_size=self.G,
                             dev_status=status, **kw)
        if in_place:
            assert got[0] is table and got[1] is lens
        want = plain(self.pages, self.table, self.home, self.lens, parents, self.D, self.G, self.page)
        assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
        assert np.array_equal(pages.cpu().numpy(), self.pages)
        assert int(status.item()) == 0
        self.table, self.lens = want


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_every_shape(D, G, page):
    c = Case(2, 4, 3, D, G, page, layers=2, seed=D + G + page, lens=[page + 5] * 4 + [2 * page + 9] * 4)
    for i in range(3):
        c.step(c.parents(), in_place=i % 2 == 1)
        c.lens += 3


@pytest.mark.parametrize("W", [1, 2, 3, 8, 31, 32, 33, 63, 64])
def test_steps_of_a_search(W):
    """From the first token on, several steps, table and lengths in place or not."""
    c = Case(3, W, 4, 64, 64, 16, H=1, seed=W)
    for i in range(12):
        c.lens += 1 + i % 5
        c.step(c.parents(), in_place=i % 2 == 0, squeeze=i % 3 == 0)
    # every beam from one
    c.step(np.full((3, W), W - 1, np.int32))
    c.step(np.tile(np.arange(W, dtype=np.int32)[::-1], (3, 1)))


@pytest.mark.parametrize("over", [0, 1, 7, 8, 9, 15])
def test_tokens_in_the_page(over):
    c = Case(2, 4, 3, 128, 32, 16, seed=over, lens=[16 + over] * 8)
    c.step(np.asarray([[0, 0, 0, 0], [3, 3, 1, 1]], np.int32))
    c = Case(2, 4, 3, 128, 32, 16, seed=over, lens=[over] * 8)
    c.step(np.asarray([[2, 2, 2, 2], [0, 1, 2, 3]], np.int32))
    c = Case(1, 4, 2, 128, 32, 16, seed=over, lens=[32] * 4)  # no page is left
    c.step(np.asarray([[2, 2, 1, 2]], np.int32))


def test_unlike_lengths():
    rng = np.random.default_rng(0)
    c = Case(6, 5, 6, 64, 32, 16, seed=1)
    for i in range(10):
        c.lens = np.minimum(c.lens + rng.integers(0, 9, c.lens.shape), 90).astype(np.int32)
        # a sequence that grew into a page has it for itself
        c.step(c.parents())


def test_many_groups_and_layers():
    c = Case(50, 4, 3, 64, 64, 16, H=3, layers=5, seed=2, lens=np.repeat(np.arange(50) % 40, 4))
    for _ in range(2):
        c.step(c.parents())


def test_entries_out_of_range():
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case(3, 4, 3, 64, 64, 16, seed=3, lens=[21] * 12)
    parents = np.asarray([[0, 0, 1, 1], [2, 2, 2, 2], [3, 0, 0, 3]], np.int32)
    pages = torch.from_numpy(c.pages.copy()).cuda()
    want_pages = c.pages.copy()
    want = plain(want_pages, c.table, c.home, c.lens, parents, 64, 64, 16)
    per_group = want_pages.copy()

    def run(table=c.table, home=c.home, lens=c.lens, parents=parents):
        status, p = i32([-1]), pages.clone()
        t, n = mxq.kv_reorder(p, i32(table), i32(home), i32(lens), i32(parents), 64, dev_status=status)
        return t.cpu().numpy(), n.cpu().numpy(), p.cpu().numpy(), int(status.item())

    t, n, p, st = run()
    assert st == 0 and np.array_equal(t, want[0]) and np.array_equal(p, want_pages)
    for far in (-1, 4, 2 ** 31 - 1, -2 ** 31):
        bad = parents.copy()
        bad[1, 2] = far
        t, n, p, st = run(parents=bad)
        assert st == mxq.DEV_BAD_SEQUENCE
        assert np.array_equal(t[4:8], c.table[4:8]) and np.array_equal(n, c.lens)
        assert np.array_equal(t[:4], want[0][:4]) and np.array_equal(t[8:], want[0][8:])
    for far in (-1, 49, 2 ** 31 - 1):
        bad = c.lens.copy()
        bad[6] = far
        t, n, p, st = run(lens=bad)
        assert st == mxq.DEV_BAD_SEQUENCE and np.array_equal(t[4:8], c.table[4:8]) and np.array_equal(n[4:8], bad[4:8])
    # a page of another group, or twice the same: the column stays
    for page in (int(c.home[0, 1]), -5, 2 ** 31 - 1):
        bad = c.table.copy()
        bad[6, 1] = page
        t, n, p, st = run(table=bad)
        assert st == mxq.DEV_BAD_PAGE and np.array_equal(t[4:8, 1], bad[4:8, 1]) and np.array_equal(t[8:], want[0][8:])
        assert np.array_equal(p[:, c.home[4:8].reshape(-1)], c.pages[:, c.home[4:8].reshape(-1)])
    # the group's own pages are not in the cache: nothing is copied
    bad = c.home.copy()
    bad[4:8, 1] += 10 ** 6
    t, n, p, st = run(table=bad, home=bad)
    assert st == mxq.DEV_BAD_PAGE and np.array_equal(p[:, c.home[4:8].reshape(-1)], c.pages[:, c.home[4:8].reshape(-1)])
    # columns that nobody has been given
    late = c.home.copy()
    late[:, 2] = -1
    t, n, p, st = run(table=late, home=late)
    assert st == 0 and np.array_equal(t[:, :2], want[0][:, :2]) and (t[:, 2] == -1).all()
    late[:, 1] = -1
    t, n, p, st = run(table=late, home=late)
    assert st == mxq.DEV_BAD_PAGE


def test_refusals():
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case(2, 4, 3, 64, 64, 16, seed=4)
    pages, table, home, lens, parents = (torch.from_numpy(c.pages).cuda(), i32(c.table), i32(c.home), i32(c.lens), i32(c.parents()))
    for bad in (lambda: mxq.kv_reorder(pages, table, home[:, :2].contiguous(), lens, parents, 64), lambda: mxq.kv_reorder(pages, table, home, lens[:7], parents, 64),
                lambda: mxq.kv_reorder(pages, table, home, lens, parents.view(-1), 64), lambda: mxq.kv_reorder(pages, table, home, lens, parents, 128),
                lambda: mxq.kv_reorder(pages, table, home, lens, parents, 64, group_size=48), lambda: mxq.kv_reorder(pages[:0], table, home, lens, parents, 64),
                lambda: mxq.kv_reorder(pages, table, home, lens, parents, 64, table_out=table[:4]),
                lambda: mxq.kv_reorder(pages.cpu(), table, home, lens, parents, 64)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mxq.kv_reorder(pages, table.long(), home, lens, parents, 64)
    for kw in (dict(table_out=home), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(mxq.MxqError):
            mxq.kv_reorder(pages, table, home, lens, parents, 64, **kw)


def test_streams_and_graphs():
    import torch

    import affine_bit_matmul_gb300 as mxq

    c = Case(2, 4, 4, 64, 64, 16, seed=5, lens=[20] * 8)
    parents = c.parents()
    pages, table, home, lens, par = (torch.from_numpy(c.pages).cuda(), i32(c.table), i32(c.home), i32(c.lens), i32(parents))
    first = c.pages.copy()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t, n = mxq.kv_reorder(pages, table, home, lens, par, 64, stream=side)
    side.synchronize()
    ref = first.copy()
    want = plain(ref, c.table, c.home, c.lens, parents, 64, 64, 16)
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(pages.cpu().numpy(), ref)
    pages.copy_(torch.from_numpy(first))
    with torch.cuda.graph(g):
        lens.add_(1)
        mxq.kv_reorder(pages, table, home, lens, par, 64, table_out=table, lens_out=lens)
    ref, tab, ln = first.copy(), c.table, c.lens
    for _ in range(20):
        g.replay()
        tab, ln = plain(ref, tab, c.home, ln + 1, parents, 64, 64, 16)
        assert np.array_equal(table.cpu().numpy(), tab) and np.array_equal(lens.cpu().numpy(), ln)
        assert np.array_equal(pages.cpu().numpy(), ref)
