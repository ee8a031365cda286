"""A step of drafted tokens on the GPU at the edges of what its calls describe."""
import ctypes

import pytest
import torch

import context_exact_attention_gb300 as cea

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MOST = 2 ** 31 - 1025                       # rows of a step, pages of a pool


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def test_no_limit_on_rows():
    """Starts, lengths and pages only, with the largest number of rows as no limit at all."""
    pool, table = cea.page_pool(9, 3, DEV), torch.full((3, 5), -1, dtype=torch.int32, device=DEV)
    new, lens, cu, kv = ints([5, 0, 9]), ints([0, 3, 0]), ints([7] * 4), ints([7] * 3)
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rc = cea.load_library().paged_reserve(pool._c, ptr(new), ptr(lens), ptr(table), 5, 5, 4, MOST, ptr(cu),
                                          ptr(kv), None, None, None, None, 0, s)
    assert rc == 0 and cea.check_status() == 0 and int(pool.status) == 0
    assert cu.tolist() == [0, 5, 5, 14] and kv.tolist() == [5, 3, 9]
    assert pool.held.tolist() == [2, 1, 3] and int(pool.count) == 3
    assert table.tolist() == [[0, 1, -1, -1, -1], [2, -1, -1, -1, -1], [3, 4, 5, -1, -1]]


def test_as_many_rows_and_pages_as_there_may_be():
    """A step of 2^31 - 1025 tokens on as many pages of one key: indexes run up to the last entry and
    not past it, on the way there and back."""
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 44 GB of device memory")
    pool = cea.page_pool(MOST, 1, DEV)
    table = torch.full((1, MOST), -1, dtype=torch.int32, device=DEV)
    step = cea.PagedStep(ints([0, 0]), ints([0]), torch.full((MOST,), -7, dtype=torch.int32, device=DEV))
    cea.paged_reserve(pool, ints([MOST - 3]), ints([0]), table, 1, step)
    assert cea.check_status() == 0 and int(pool.status) == 0 and int(pool.count) == 3
    assert step.cu_new.tolist() == [0, MOST - 3] and step.kv_lens.tolist() == [MOST - 3]
    up = torch.arange(MOST, dtype=torch.int32, device=DEV)
    assert torch.equal(table[0, :-3], up[:-3]) and table[0, -3:].tolist() == [-1] * 3
    assert torch.equal(step.positions[:-3], up[:-3]) and step.positions[-3:].tolist() == [0] * 3
    del step
    pool.free.fill_(-1)
    cea.paged_release(pool, ints([5]), table, 1)
    assert cea.check_status() == 0 and int(pool.count) == MOST - 5 and pool.held.tolist() == [5]
    # (the three pages that were left lie below them)
    assert torch.equal(pool.free[3:MOST - 5].flip(0), up[5:-3]) and (pool.free[:3] == -1).all()
    assert torch.equal(table[0, :5], up[:5]) and bool((table[0, 5:] == -1).all())
