"""Fork and reserve when pages run out: expected values written out by hand from the
header's rules, for the plain definition (CPU) and the library (GPU).  A row that
needs no page is served whatever the rows before it asked for."""
import numpy as np
import pytest
import torch

import q8_ref as R

P = 16
# name: table, lengths, pages, src, need -> table, lengths, refs, taken
CASES = {
    # row 0 asks for two pages, one is free; rows 1 and 2 need none
    "reserve": (
        [[0, 1, -1, -1], [2, -1, -1, -1], [3, -1, -1, -1]], [32, 16, 16], 5, None, [32, 0, 0],
        [[0, 1, -1, -1], [2, -1, -1, -1], [3, -1, -1, -1]], [32, 16, 16], [1, 1, 1, 1, 0], [-1, 0, 0]),
    # row 2 needs one page: none of the free ones goes to a row behind one that found too few
    "a later row that needs one": (
        [[0, 1, -1, -1], [2, -1, -1, -1], [3, -1, -1, -1], [4, 5, -1, -1]], [32, 16, 16, 20], 7, None, [32, 0, 1, 12],
        [[0, 1, -1, -1], [2, -1, -1, -1], [3, -1, -1, -1], [4, 5, -1, -1]], [32, 16, 16, 20],
        [1, 1, 1, 1, 1, 1, 0], [-1, 0, -1, 0]),
    # row 0 asks for two pages, one is free; row 1 shares row 3's full page, which takes none
    "forks": (
        [[0, -1, -1], [1, -1, -1], [2, 3, -1], [4, -1, -1]], [16, 16, 20, 16], 5, [0, 3, 2, 3], [32, 0, 0, 0],
        [[0, -1, -1], [4, -1, -1], [2, 3, -1], [4, -1, -1]], [16, 16, 20, 16], [1, 0, 1, 1, 2], [-1, 0, 0, 0]),
    # row 0 takes both free pages, 1 and 4; row 2 has to copy row 1's open page and ends at its last full one
    "a fork without its copy": (
        [[0, -1, -1], [2, 3, -1], [4, -1, -1]], [16, 20, 16], 5, [0, 1, 1], [17, 0, 0],
        [[0, 1, 4], [2, 3, -1], [2, -1, -1]], [16, 20, 16], [1, 1, 2, 1, 1], [2, 0, -1]),
    # nothing is free at all
    "none free": (
        [[0, -1], [1, -1]], [16, 16], 2, None, [1, 0],
        [[0, -1], [1, -1]], [16, 16], [1, 1], [-1, 0]),
}
i32 = lambda x: np.asarray(x, np.int32)  # noqa: E731


@pytest.mark.parametrize("name", CASES)
def test_definition(name):
    table, lens, n, src, need, *want = CASES[name]
    got = R.fork(i32(table), i32(lens), n, P, src, need)
    for g, w in zip(got, want):
        assert np.array_equal(g, i32(w)), (g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_library(medusa, name):
    table, lens, n, src, need, *want = CASES[name]
    dev = lambda x: None if x is None else torch.from_numpy(i32(x)).cuda()  # noqa: E731
    codes, scale = torch.zeros(n, 1, P, 64, dtype=torch.uint8, device="cuda"), torch.ones(n, 1, device="cuda")
    r = medusa.kv_pages_fork(codes, codes.clone(), scale, scale.clone(), dev(table), dev(lens), dev(src), dev(need))
    for k, w in zip(("page_table", "kv_len", "refs", "taken"), want):
        assert np.array_equal(r[k].cpu().numpy(), i32(w)), (k, r[k], w)
