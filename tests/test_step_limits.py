"""What a step of drafted tokens refuses or reports at the edges of what its calls describe, host
side (no GPU): the library's calls are recorded instead of made."""
import copy
import weakref

import pytest
import torch

import context_exact_attention_gb300 as cea


@pytest.fixture
def calls(monkeypatch):
    """The calls of the library, (name, arguments), made by the binding on CPU tensors."""
    made = []
    monkeypatch.setattr(cea, "_same_device", lambda first, *others: first.get_device())
    monkeypatch.setattr(cea, "_stream_here", lambda device, stream: 0)
    monkeypatch.setattr(cea, "_call_fast", lambda name, *args: made.append((name, args)))
    return made


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def attend(masks, T, n_seqs=3):
    pages = torch.zeros(8, 16, 1, 64, dtype=torch.bfloat16)
    q = torch.zeros(T, 2, 64, dtype=torch.bfloat16)
    cea.paged_attn_fwd(q, pages, pages, ints(n_seqs, 2), ints(n_seqs + 1), ints(n_seqs), masks=masks,
                       out=torch.empty_like(q), lse=torch.empty(T, 2), workspace=ints(1))


def test_masks_of_a_broadcast(calls):
    """One row for all new tokens, as expand makes it, has no memory for a row each."""
    for masks in (ints(1, 1).expand(9, 1), ints(1, 4).expand(9, 4), ints(4).expand(9, 4),
                  ints(12).as_strided((9, 4), (1, 1))):
        with pytest.raises(ValueError):
            attend(masks, 9)
    assert not calls
    for masks, step in ((ints(9, 4), 4), (ints(9, 7)[:, 2:6], 7), (ints(9, 3)[:, :1], 3), (ints(18, 2)[::2], 4)):
        attend(masks, 9)
        assert calls.pop()[1][1:4] == (masks.data_ptr(), masks.shape[1], step)
    attend(ints(5).expand(1, 5), 1)                 # one row is one row, whatever its stride
    assert calls.pop()[1][2:4] == (5, 5)


def keep(kept):
    n = kept.shape[0]
    pages = torch.zeros(8, 16, 1, 64, dtype=torch.bfloat16)
    cea.paged_kv_keep(kept, pages, pages.clone(), ints(n, 2), ints(n + 1), ints(n),
                      lens=ints(n))


def test_kept_paths_of_a_broadcast(calls):
    """One path for all sequences, as expand makes it, has no memory for a path each."""
    for kept in (ints(1, 4).expand(3, 4), ints(4).expand(3, 4), ints(1, 1).expand(3, 1),
                 ints(8).as_strided((3, 4), (2, 1))):
        with pytest.raises(ValueError):
            keep(kept)
    assert not calls
    for kept, step in ((ints(3, 4), 4), (ints(3, 9)[:, 1:5], 9), (ints(6, 4)[::2], 8), (ints(3, 5)[:, :1], 5)):
        keep(kept)
        assert calls.pop()[1][1:4] == (kept.data_ptr(), kept.shape[1], step)
    keep(ints(4).expand(1, 4))
    assert calls.pop()[1][2:4] == (4, 4)


def test_a_pool_keeps_its_tensors():
    """The calls use the addresses that a pool was made with: its tensors are filled, not exchanged."""
    pool = cea.page_pool(6, 2, device="cpu")
    for name in ("free", "held", "state", "count", "status", "num_pages", "n_seqs"):
        with pytest.raises(AttributeError):
            setattr(pool, name, getattr(pool, name))
        with pytest.raises(AttributeError):
            delattr(pool, name)
    with pytest.raises(AttributeError):
        pool.other = 1
    pool.held.copy_(torch.tensor([2, 1]))
    assert pool.held.tolist() == [2, 1]
    assert (pool._desc.free_pages, pool._desc.held, pool._desc.state) == (
        pool.free.data_ptr(), pool.held.data_ptr(), pool.state.data_ptr())
    step = cea.paged_step(2, 5, device="cpu")
    with pytest.raises(AttributeError):
        del step.cu_new


def test_pools_that_no_call_takes():
    """More sequences or pages than the calls know are refused where the pool is made."""
    cea.page_pool(1, 8192, device="cpu")
    with pytest.raises(ValueError):
        cea.page_pool(1, 8193, device="cpu")
    with pytest.raises(ValueError):
        cea.page_pool(2 ** 31 - 1024, 1, device="cpu")


def test_reserve_counts_what_masks_leave_out(calls):
    """The pool has a place for the number of tokens that masks have no bit for, and the call gets it."""
    pool, step = cea.page_pool(6, 2, device="cpu"), cea.paged_step(2, 50, mask_words=1, device="cpu")
    assert pool.unmasked.tolist() == [0]
    cea.paged_reserve(pool, ints(2), ints(2), ints(2, 3), 16, step)
    assert calls[0][1][-3:-1] == (1, pool.unmasked.data_ptr())


def test_unmasked_refusals():
    from test_step_host import INVALID, MISALIGNED, NULL, S, at, off, pool
    lib = cea.load_library()

    def call(unmasked, masks=at(11), words=2):
        return lib.paged_reserve_ex(pool(), at(3), at(5), at(4), 10, 10, 16, 40, at(6), at(7), at(8), at(9),
                                    at(10), masks, words, unmasked, S)

    for i in range(12):                     # (2: state, 11: masks, ...; no array holds the number too)
        assert call(at(i)) == INVALID, i
    assert call(off(12, 2)) == MISALIGNED
    assert call(at(12), masks=NULL) == INVALID


def test_a_rotation_keeps_what_it_was_made_with():
    """As a pool does: a new amplitude or new frequencies would not reach the calls."""
    table = cea.rope_table(8, device="cpu")
    for name in ("phases", "rot_dim", "style", "amplitude"):
        with pytest.raises(AttributeError):
            setattr(table, name, getattr(table, name))
    assert cea.RopeTable(table.phases, 8, "half", 2.0).amplitude == 2.0
    assert copy.copy(table).phases is table.phases and weakref.ref(table)() is table
