"""How a call over shared prefixes is cut into pieces, walked on the host (no GPU needed): every query row and head
in one row tile, no row tile without rows, no position past the tokens, every place once."""

import subprocess

import pytest

# kv_shared.cuh's lists as the kernels go over them, one run that holds all units.
SOURCE = r"""
#include <cstdio>
#include <vector>
#include "kv_shared.cuh"
using namespace mxq;

static int wrong(const char* what, const KvSharedParams& p, int rep, int item, int plane, int vh) {
    printf("%s: %d heads, %d a part, tiles of %d, %s %d, plane %d, part %d\n", what, rep, p.part_heads, p.tile_rows,
           p.prefix ? "group" : "sequence", item, plane, vh);
    return 1;
}

// Sequences of `rows` rows and `lens` tokens (or, with a list, groups of them), heads in parts of at most `most`.
static int walk(bool prefix, int rep, int most, int tile_rows, const std::vector<int>& rows, const std::vector<int>& lens,
                const std::vector<int>& groups) {
    std::vector<int> starts(1, 0);
    for (int n : rows) starts.push_back(starts.back() + n);
    KvSharedParams p{};
    p.Hkv = 2;
    p.Hq = 2 * rep;
    p.head_parts = (rep + most - 1) / most;
    p.part_heads = (rep + p.head_parts - 1) / p.head_parts;
    p.tile_rows = tile_rows;
    p.tile_shift = most == 128 ? 7 : 5;
    p.end_units = 3;
    p.page_size = 16;
    p.max_pages = 64;
    p.T = starts.back();
    p.S = (int)rows.size();
    p.q_starts = starts.data();
    p.max_q = p.T;
    p.groups_n = (int)groups.size() - 1;
    p.groups = groups.data();
    p.max_group = p.S;
    p.prefix = prefix;
    p.prefix_lens = p.ctx_lens = lens.data();
    const int items = items_of(p), vheads = p.Hkv * p.head_parts;
    long long units = 0, planes = 0;
    for (int i = 0; i < items; ++i) {
        units += units_of(p, item_of(p, i));
        planes += item_of(p, i).planes;
    }
    if (planes > (long long)p.T * p.part_heads / tile_rows + items) return wrong("more row tiles than places", p, rep, items, 0, 0);
    SharedWalk w{};
    w.load(p, 0);
    w.left = units * vheads;
    // tiles of tokens that each (row of q, query head) has gone over, and the row tiles seen
    std::vector<int> seen((size_t)p.T * p.Hq, 0);
    std::vector<char> taken((size_t)(planes * vheads), 0);
    SharedPiece q;
    while (w.next(p, &q)) {
        find_rows(p, q);
        if (q.rows <= 0 || q.count <= 0) return wrong("no rows", p, rep, q.item, q.plane, q.vh);
        if (q.p1 >= q.it.len) return wrong("a position past the tokens", p, rep, q.item, q.plane, q.vh);
        if (q.tile < 0 || q.tile >= planes * vheads || taken[q.tile]) return wrong("a place twice", p, rep, q.item, q.plane, q.vh);
        taken[q.tile] = 1;
        if (q.k0 || q.count != tiles_of(p, q.it)) return wrong("units", p, rep, q.item, q.plane, q.vh);
        for (int r = q.flat0; r < q.flat0 + q.rows; ++r) {
            const int row = q.it.row0 + r / q.heads, head = q.head0 + r % q.heads;
            if (row >= q.it.row0 + q.it.rows || head / rep != q.h) return wrong("other rows", p, rep, q.item, q.plane, q.vh);
            seen[(size_t)row * p.Hq + head] += q.count;
            const int last = prefix ? q.it.len - 1 : q.it.len - q.it.rows + r / q.heads;
            if (last > q.p1) return wrong("a row that sees more", p, rep, q.item, q.plane, q.vh);
        }
    }
    if (q.count) return wrong("a piece after the last", p, rep, items, 0, 0);
    for (int i = 0; i < items; ++i) {
        const Item it = item_of(p, i);
        for (int r = it.row0; r < it.row0 + it.rows; ++r)
            for (int h = 0; h < p.Hq; ++h)
                if (seen[(size_t)r * p.Hq + h] != (it.len ? tiles_of(p, it) : 0)) return wrong("rows left out", p, rep, i, r, h);
    }
    return 0;
}

int main() {
    const int some[] = {1, 2, 3, 4, 5, 7, 8, 15, 16, 17, 31, 33, 64};
    for (int rep = 1; rep <= 300; ++rep)
        for (int rows : some) {
            // tables that are full, and lengths below the rows; one sequence without rows, one without tokens
            const std::vector<int> many = {rows, 1, 0, rows, 2, rows}, lens = {1024, 5, 40, rows / 2, 0, 1000}, groups = {0, 2, 2, 5, 6};
            for (int tile : {4, 8, 16})
                for (int prefix = 0; prefix < 2; ++prefix)
                    if (walk(prefix, rep, 16, tile, many, prefix ? std::vector<int>{1024, 7, 0, 333} : lens, groups)) return 1;
            for (int tile : {128, 256})
                if (walk(true, rep, 128, tile, many, {1024, 7, 0, 333}, groups)) return 1;
        }
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from affine_bit_matmul_gb300 import build

    folder = tmp_path_factory.mktemp("pieces")
    (folder / "walk.cu").write_text(SOURCE)
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, str(folder / "walk.cu"), "-o", str(folder / "walk")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return str(folder / "walk")


def test_pieces_have_rows_and_stay_within_the_tokens(program):
    r = subprocess.run([program], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
