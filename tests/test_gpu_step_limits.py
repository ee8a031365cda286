"""A step of drafted tokens on the GPU at the edges of what its calls describe."""
import ctypes

import pytest
import torch

import context_exact_attention_gb300 as cea
from paged_helpers import Cache, assert_attends
from step_helpers import ancestors, random_parents, tree_reference

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


# new tokens, lengths before: a prompt beside trees, a token, and a sequence that brings none
MIXED = [100, 13, 0, 33, 1], [40, 0, 7, 60, 500]


def reserved(words, new=MIXED[0], lens=MIXED[1], chain=True, T=None):
    """A step of prompts (chains) and trees with masks of 32 * words tokens: (step, pool, page table,
    what new tokens see)."""
    g = torch.Generator().manual_seed(words)
    n = len(new)
    pool, step = cea.page_pool(200, n, DEV), cea.paged_step(n, sum(new) + 3 if T is None else T, words, DEV)
    table = torch.full((n, 60), -1, dtype=torch.int32, device=DEV)
    before = cea.paged_step(n, sum(lens), device=DEV)
    cea.paged_reserve(pool, ints(lens), ints([0] * n), table, 16, before)
    trees = [list(range(-1, a - 1)) if a > 64 and chain else random_parents(a, g) for a in new]
    parents = [p for t in trees for p in t]
    pool.unmasked.fill_(77)
    cea.paged_reserve(pool, ints(new), ints(lens), table, 16, step,
                      parents=ints((parents + [-1] * step.positions.shape[0])[:step.positions.shape[0]]))
    assert cea.check_status() == 0
    return step, pool, table, [ancestors(t)[0] for t in trees]


def test_tokens_that_masks_have_no_bit_for():
    """Counted wherever a sequence brings more than 32 * words, and only there."""
    for words, want in ((1, 68 + 1), (2, 36), (3, 4), (4, 0), (0, 0)):
        step, pool, _, _ = reserved(words)
        assert int(pool.status) == 0 and pool.unmasked.tolist() == [want], words
    step, pool, _, _ = reserved(1, T=100)                   # does not fit: no rows
    assert int(pool.status) == 2 and pool.unmasked.tolist() == [0]
    # without parents, and many sequences in one call of several blocks
    pool, step = cea.page_pool(9000, 3000, DEV), cea.paged_step(3000, 90000, 1, DEV)
    table, zero = torch.full((3000, 3), -1, dtype=torch.int32, device=DEV), ints([0] * 3000)
    new = torch.arange(3000, device=DEV).remainder(40).int()
    cea.paged_reserve(pool, new, zero, table, 16, step)
    assert int(pool.status) == 0 and pool.unmasked.tolist() == [75 * sum(i - 32 for i in range(33, 40))]


@pytest.mark.parametrize("dtype,H,K,D", [(torch.bfloat16, 8, 2, 128), (torch.bfloat16, 4, 2, 64),
                                         (torch.float32, 8, 2, 64)])
def test_a_prompt_beside_trees(dtype, H, K, D):
    """Masks wide enough for the prompt: its rows follow the causal rule, the trees' their ancestors."""
    step, pool, table, seen = reserved(4)
    assert pool.unmasked.tolist() == [0]
    seqs = [(a, a + b) for a, b in zip(*MIXED)]
    c = Cache(seqs, H, K, D, 16, dtype, "slots", pad=3, seed=D)
    c.table, c.num_pages = table.cpu(), 200
    used = pool.held.tolist()
    g = torch.Generator().manual_seed(1)
    c.k, c.v = (torch.full((200, 16, K, D), float("nan"), dtype=dtype) for _ in "kv")
    for i, (_, kv) in enumerate(seqs):
        for j in range(used[i]):
            n = max(0, min(16, kv - 16 * j))
            for x in (c.k, c.v):
                x[c.table[i, j], :n] = torch.randn(n, K, D, generator=g).to(dtype)
    assert step.cu_new.cpu().tolist() == c.cu.tolist() and step.kv_lens.cpu().tolist() == c.kv_lens.tolist()
    kp, vp = c.device_pages(DEV)
    out, lse = cea.paged_attn_fwd(c.q.to(DEV), kp, vp, table, step.cu_new, step.kv_lens, masks=step.masks)
    assert cea.check_status() == 0
    assert_attends(out, lse, tree_reference(c, seen))
    causal = c.reference(True)
    rows = slice(0, 100)
    assert_attends(out[rows], lse[rows], tuple(x[rows] for x in causal))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot", [(128, 0), (128, 126), (72, 72), (64, 64)])
def test_heads_that_count_as_infinitely_long(dtype, D, rot):
    """A head whose squares pass fp32's range gives zeros, and zero gradients (u = 0, g over infinity),
    however large the sum of g x is; the heads beside it and the weights' gradients as without it."""
    g = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(1, 6, 3, D, generator=g).to(dtype).to(DEV) for _ in "xy")
    w = torch.randn(D, generator=g).to(dtype).to(DEV)
    rope = cea.rope_table(rot, device=DEV) if rot else None
    x[0, 0, 1], dy[0, 0, 1] = 2.0 ** 124, 8.0
    x[0, 4, 2], dy[0, 4, 2] = -2.0 ** 126, 2.0 ** 20
    long = torch.zeros(1, 6, 3, dtype=torch.bool)
    long[0, 0, 1] = long[0, 4, 2] = True
    y, _ = cea.qk_norm_rope_fwd(x, None, w.abs(), None, rope)
    dx, _, dw, _ = cea.qk_norm_rope_bwd(x, None, w.abs(), None, dy, None, rope)
    assert cea.check_status() == 0
    assert (y[long] == 0).all() and (dx[long] == 0).all()
    x[long.to(DEV)], dy[long.to(DEV)] = 1.0, 0.0            # heads that add nothing
    want, _, want_w, _ = cea.qk_norm_rope_bwd(x, None, w.abs(), None, dy, None, rope)
    assert torch.equal(dx[~long], want[~long]) and torch.equal(dw, want_w)


@pytest.mark.parametrize("dtype,D,layout", [(torch.bfloat16, 128, "slots"), (torch.bfloat16, 80, "by_head"),
                                            (torch.float32, 64, "by_slot")])
@pytest.mark.parametrize("normed", [True, False], ids=["norm", "plain"])
def test_append_writes_its_slots_and_no_others(dtype, D, layout, normed):
    """By bits, keys and values alike, in pages that hold something everywhere."""
    c = Cache([(1, 1), (0, 5), (7, 40), (33, 33), (3, 2)], 4, 2, D, 16, dtype, layout, pad=3, seed=D)
    g = torch.Generator().manual_seed(D)
    c.k, c.v = (torch.randn(c.k.shape, generator=g).to(dtype) for _ in "kv")
    k, v = (torch.randn(c.T, 2, D, generator=g).to(dtype) for _ in "kv")
    kp, vp = c.device_pages(DEV)
    more = dict(k_weight=torch.ones(D, dtype=dtype, device=DEV)) if normed else {}
    cea.paged_kv_append(k.to(DEV), v.to(DEV), kp, vp, c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV), **more)
    assert cea.check_status() == 0
    kp, vp, want_v, mine = kp.cpu(), vp.cpu(), c.v.clone(), torch.zeros(c.k.shape[:2], dtype=torch.bool)
    for s, (n, kv) in enumerate(c.seqs):
        for j in range(max(0, n - kv), n):
            at = kv - n + j
            page, slot, row = int(c.table[s, at // 16]), at % 16, int(c.cu[s]) + j
            want_v[page, slot], mine[page, slot] = v[row], True
            if not normed:
                c.k[page, slot] = k[row]
    bits = lambda x: x.contiguous().view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
    assert torch.equal(bits(vp), bits(want_v))
    assert torch.equal(bits(kp[~mine]), bits(c.k[~mine]))
    assert normed or torch.equal(bits(kp), bits(c.k))
