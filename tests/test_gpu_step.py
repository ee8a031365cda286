"""A step of drafted tokens on the GPU: page bookkeeping against a plain model, normalised heads and
their gradients, trees' attention and the kept tokens against 64-bit arithmetic (bounds:
step_helpers, paged_helpers), and all of them run together as a program does."""
import pytest
import torch

import context_exact_attention_gb300 as cea
from paged_helpers import Cache, assert_attends
from step_helpers import (PoolModel, ancestors, angles64, assert_within, mask_words, norm64, norm_bwd64,
                          random_parents, tree_reference)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


# ------------------------------------------------------------------------- pages --

class Pool:
    """A pool on the device beside its plain model."""

    def __init__(self, num_pages, n_seqs, max_pages, page):
        self.model = PoolModel(num_pages, n_seqs, max_pages, page)
        self.pool = cea.page_pool(num_pages, n_seqs, DEV)
        self.table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=DEV)
        self.page, self.n = page, n_seqs

    def reserve(self, new, lens, T, parents=None, words=0, step=None):
        step = step or cea.paged_step(self.n, T, words, DEV)
        for t in step:
            if t is not None:
                t.fill_(77)
        cea.paged_reserve(self.pool, ints(new), ints(lens), self.table, self.page, step,
                          parents=None if parents is None else ints(parents))
        want = self.model.reserve(new, lens, T, parents)
        got = [step.cu_new.tolist(), step.kv_lens.tolist(), step.positions.tolist(), step.slots.tolist(),
               int(self.pool.status)]
        assert got == list(want)
        self.same()
        if words:
            cu, rows = want[0], []
            for a, b in zip(cu, cu[1:]):
                rows.append(mask_words(ancestors(parents[a:b])[0], words))
            rows.append(torch.zeros(T - cu[-1], words, dtype=torch.int32))
            assert torch.equal(step.masks.cpu(), torch.cat(rows))
        return step

    def release(self, lens):
        cea.paged_release(self.pool, ints(lens), self.table, self.page)
        self.model.release(lens)
        self.same()

    def same(self):
        assert cea.check_status() == 0
        m, count = self.model, int(self.pool.count)
        assert self.pool.held.tolist() == m.held and self.table.tolist() == m.table
        assert self.pool.free[:count].tolist() == m.free and int(self.pool.state[1]) == 0


@pytest.mark.parametrize("n_seqs,page,most", [(1, 16, 1), (1, 1, 40), (3, 8, 700), (64, 64, 1), (300, 16, 9),
                                              (1025, 5, 3), (2000, 16, 40), (8192, 16, 2)])
def test_reserve_and_release(n_seqs, page, most):
    g = torch.Generator().manual_seed(n_seqs + page)
    r = lambda hi: torch.randint(0, hi + 1, (n_seqs,), generator=g).tolist()
    lens = r(60)
    max_pages = -(-(60 + 2 * most) // page)
    p = Pool(n_seqs * max_pages, n_seqs, max_pages, page)
    p.reserve(lens, [0] * n_seqs, sum(lens))
    for i in range(3):
        new = r(most)
        before = list(p.model.free)
        p.reserve(new, lens, sum(new) + (7 if i else 0))
        kept = [a + min(b, c) for a, b, c in zip(lens, new, r(most))] if i else lens
        p.release(kept)
        if i == 0:
            assert p.model.free == before
        lens = [k if j % 3 else 0 for j, k in enumerate(kept)]        # some have ended
        p.release(lens)
    p.release([0] * n_seqs)
    assert int(p.pool.count) == n_seqs * max_pages


@pytest.mark.parametrize("words", [1, 2, 5])
def test_trees_of_parents(words):
    """Depths as positions, ancestors as bits; tokens beyond the words, parents that are none."""
    g = torch.Generator().manual_seed(words)
    new, lens = [0, 1, 32, 33, 64, 100, 170, 0, 3], [5, 0, 7, 16, 3, 900, 31, 2, 64]
    parents = []
    for i, n in enumerate(new):
        parents += random_parents(n, g, wide=i % 2 == 0)
    parents[40] = 1000                                 # behind itself: a root
    parents[50] = -9
    p = Pool(500, len(new), 80, 16)
    p.reserve(lens, [0] * len(new), sum(lens))
    p.reserve(new, lens, sum(new) + 5, parents + [12345] * 5, words)


def test_positions_without_masks():
    p = Pool(10, 2, 4, 16)
    p.reserve([4, 3], [0, 0], 8, parents=[-1, 0, 0, 1, -1, -1, 1, 0])


def test_chains_without_parents_and_steps_without_rows():
    """Masks without parents are the causal rule's; a step of no rows writes lengths and starts."""
    p = Pool(40, 3, 10, 16)
    step = cea.paged_step(3, 110, 3, DEV)
    p.reserve([70, 0, 33], [0, 0, 0], 110, step=step)
    want = [mask_words(torch.ones(n, n).tril().bool(), 3) for n in (70, 33)]
    assert torch.equal(step.masks.cpu(), torch.cat(want + [torch.zeros(7, 3, dtype=torch.int32)]))
    none = cea.paged_step(3, 0, 2, DEV)
    p.reserve([0, 0, 0], [70, 0, 33], 0, step=none)
    p.reserve([1, 0, 0], [70, 0, 33], 0, step=none)
    assert int(p.pool.status) == 2 and none.cu_new.tolist() == [0] * 4


def test_steps_that_do_not_fit():
    p = Pool(6, 2, 4, 16)
    p.reserve([20, 10], [0, 0], 40)
    for new, T in (([1, 1], 1), ([45, 0], 64), ([0, 60], 64), ([40, 40], 90)):
        p.reserve(new, [20, 10], T)
        assert int(p.pool.status) in (1, 2, 3)
    p.reserve([28, 22], [20, 10], 50)
    assert int(p.pool.status) == 0 and int(p.pool.count) == 1
    p.reserve([2 ** 31 - 1, 2 ** 31 - 1], [48, 32], 50)
    assert int(p.pool.status) == 2
    p.reserve([-5, -2 ** 31], [-3, 32], 4)             # negative lengths count as none
    assert int(p.pool.status) == 0


def test_lengths_in_place_and_what_is_left_out():
    p = Pool(20, 3, 6, 4)
    lens = ints([0, 0, 0])
    step = cea.paged_step(3, 12, device=DEV)._replace(kv_lens=lens, slots=None)
    for new in ([4, 1, 0], [1, 1, 8], [0, 0, 3]):
        want = p.model.reserve(new, lens.tolist(), 12)
        cea.paged_reserve(p.pool, ints(new), lens, p.table, 4, step)
        assert lens.tolist() == want[1] and step.positions.tolist() == want[2]
        p.same()
    bare = cea.paged_step(3, 12, device=DEV)._replace(kv_lens=lens, positions=None)
    want = p.model.reserve([1, 1, 1], lens.tolist(), 12)
    cea.paged_reserve(p.pool, ints([1, 1, 1]), lens, p.table, 4, bare)
    assert bare.slots.tolist() == want[3]


def test_a_table_of_a_larger_one():
    """Rows of a strided table; entries that a program has damaged reach nothing else."""
    big = torch.full((4, 11), -5, dtype=torch.int32, device=DEV)
    pool, table = cea.page_pool(12, 4, DEV), big[:, 2:7]
    step = cea.paged_step(4, 30, device=DEV)
    cea.paged_reserve(pool, ints([9, 3, 0, 17]), ints([0, 0, 0, 0]), table, 4, step)
    assert (big[:, :2] == -5).all() and (big[:, 7:] == -5).all()
    assert table.tolist()[3] == [4, 5, 6, 7, 8] and int(pool.count) == 3
    table[0, 1] = 10 ** 6
    pool.held[1] = 99                                   # taken as the table's five
    cea.paged_release(pool, ints([4, 0, 0, 17]), table, 4)
    assert cea.check_status() == 0
    assert pool.held.tolist() == [1, 0, 0, 5] and int(pool.count) <= 12
    assert (big[:, :2] == -5).all() and (big[:, 7:] == -5).all()
    pool.count.fill_(-3)
    cea.paged_reserve(pool, ints([9, 3, 0, 17]), ints([4, 0, 0, 0]), table, 4, step)
    assert int(pool.status) == 1 and cea.check_status() == 0


# ------------------------------------------------------------------- normalised heads --

# B, L, H, H_kv, D, rot (0: no rotation), style, layout, dtype, weights' dtype (None: none), offset
NORM = {
    "one token": (1, 1, 1, 1, 128, 128, "half", "contiguous", BF, BF, 0.0),
    "decode": (64, 1, 32, 8, 128, 128, "half", "given", BF, BF, 0.0),
    "odd tokens": (3, 37, 5, 1, 64, 64, "half", "contiguous", BF, F32, 0.0),
    "zigzag": (2, 48, 8, 2, 128, 128, "half", "zigzag", BF, BF, 1.0),
    "packed": (1, 301, 6, 3, 128, 64, "half", "packed", BF, F32, 0.0),
    "interleaved": (2, 33, 4, 4, 128, 128, "interleaved", "given", BF, BF, 0.0),
    "interleaved part": (1, 70, 3, 1, 96, 62, "interleaved", "contiguous", BF, F32, 1.0),
    "odd half": (1, 45, 10, 2, 128, 126, "half", "contiguous", BF, BF, 0.0),
    "odd half of 80": (2, 19, 4, 2, 80, 20, "half", "given", BF, BF, 0.0),
    "80 dims": (1, 50, 5, 5, 80, 80, "half", "contiguous", BF, BF, 0.0),
    "256 dims": (1, 40, 4, 1, 256, 256, "half", "given", BF, F32, 1.0),
    "256 dims, part": (1, 40, 4, 1, 256, 254, "half", "contiguous", BF, None, 0.0),
    "8 dims": (2, 100, 3, 2, 8, 4, "half", "contiguous", BF, BF, 0.0),
    "no rotation": (1, 77, 7, 2, 128, 0, "half", "contiguous", BF, BF, 0.0),
    "many heads": (1, 5, 300, 2, 64, 64, "half", "contiguous", BF, None, 0.0),
    "fp32": (1, 50, 6, 2, 128, 128, "half", "given", F32, F32, 0.0),
    "fp32 odd half": (1, 31, 3, 1, 128, 126, "half", "contiguous", F32, F32, 0.0),
    "fp32 256": (1, 20, 2, 2, 256, 256, "interleaved", "packed", F32, BF, 1.0),
    "fp32 256, part": (1, 20, 2, 2, 256, 128, "half", "zigzag", F32, F32, 0.0),
    "96 dims": (2, 60, 5, 2, 96, 96, "half", "contiguous", BF, BF, 0.0),
    "96 dims, odd half": (1, 60, 5, 2, 96, 24, "half", "given", BF, F32, 0.0),
    "64 dims, odd half": (1, 70, 9, 2, 64, 62, "half", "contiguous", BF, BF, 0.0),
    "72 dims, odd half": (1, 30, 3, 2, 72, 70, "half", "contiguous", BF, BF, 0.0),
    "interleaved 64": (1, 50, 6, 2, 64, 64, "interleaved", "contiguous", BF, BF, 0.0),
    "interleaved 80": (1, 50, 6, 2, 80, 78, "interleaved", "given", BF, F32, 0.0),
    "interleaved 256": (1, 20, 2, 1, 256, 256, "interleaved", "contiguous", BF, BF, 1.0),
    "interleaved 72": (1, 33, 3, 1, 72, 72, "interleaved", "contiguous", BF, BF, 0.0),
    "fp32 interleaved 96": (1, 33, 3, 1, 96, 94, "interleaved", "contiguous", F32, F32, 0.0),
    "24 dims": (1, 90, 3, 2, 24, 24, "half", "contiguous", BF, BF, 0.0),
    "fp32 80 dims": (1, 40, 4, 2, 80, 40, "half", "contiguous", F32, F32, 0.0),
    "fp32 96 dims": (1, 40, 4, 2, 96, 96, "half", "given", F32, F32, 1.0),
    "fp32 256 odd half": (1, 25, 2, 1, 256, 254, "half", "contiguous", F32, F32, 0.0),
    "fp32 4 dims": (1, 600, 2, 1, 4, 2, "half", "contiguous", F32, F32, 0.0),
    "fp32 100 dims": (1, 90, 4, 2, 100, 50, "half", "contiguous", F32, None, 0.0),
    "more tokens than blocks": (1, 6001, 4, 2, 64, 64, "half", "contiguous", BF, BF, 0.0),
}


class NormCase:
    def __init__(self, name):
        (B, L, H, H_kv, D, rot, style, layout, dtype, wtype, offset) = NORM[name]
        g = torch.Generator().manual_seed(len(name) + D)
        self.layout, self.offset, self.style, self.D = layout, offset, style, D
        lead = (L,) if layout == "packed" else (B, L)
        scale = 2.0 ** torch.randint(-6, 7, (*lead, 1, 1), generator=g)
        rand = lambda h: torch.randn(*lead, h, D, generator=g)
        self.q, self.k = (rand(H) * scale).to(dtype), (rand(H_kv) * scale).to(dtype)
        self.q[..., 0, :].view(-1, D)[0] = 0              # an empty head
        self.dq, self.dk = rand(H).to(dtype), rand(H_kv).to(dtype)
        w = lambda: None if wtype is None else (torch.randn(D, generator=g) + 1 - offset).to(wtype)
        self.wq, self.wk = w(), w()
        self.kw = dict(layout="contiguous" if layout == "given" else layout, weight_offset=offset)
        self.P = 2 if layout == "zigzag" else 1
        self.live = torch.ones(L if layout == "packed" else B * L, dtype=torch.bool)
        row = torch.arange(L)
        if layout == "given":
            pos = torch.randint(-50, 1 << 20, (B, L), generator=g).int()
            self.kw["positions"] = pos.to(DEV)
        elif layout == "zigzag":
            pos = torch.tensor(cea.zigzag_positions(L, 2)).expand(B, L)
        elif layout == "packed":
            cu = [0, 0, L // 3, L // 2, L - 4]              # an empty sequence, rows behind the last
            self.live[L - 4:] = False
            pos = row - torch.tensor(cu)[torch.searchsorted(torch.tensor(cu), row, right=True) - 1]
            self.kw["cu_seqlens"] = ints(cu)
        else:
            pos = row.expand(B, L)
        self.kw["P"] = self.P
        self.rope = self.amp = None
        i = torch.arange(rot // 2, dtype=torch.float64)
        self.angle = angles64(pos, 10000.0 ** (-2 * i / max(rot, 1)))
        self.amp = 1.25 if rot else 1.0
        if rot:
            self.kw["rope"] = cea.rope_table(rot, style=style, amplitude=1.25, device=DEV)

    def weight(self, w):
        # (as the kernel has it: the offset added in fp32)
        return torch.ones(self.D, dtype=torch.float64) if w is None else (w.float() + self.offset).double()

    def dev(self, *names):
        return [getattr(self, n).to(DEV) if getattr(self, n) is not None else None for n in names]


@pytest.mark.parametrize("name", NORM)
def test_norm(name):
    c = NormCase(name)
    outs = cea.qk_norm_rope_fwd(*c.dev("q", "k", "wq", "wk"), **c.kw)
    assert cea.check_status() == 0
    for got, x, w in zip(outs, (c.q, c.k), (c.wq, c.wk)):
        y, tol = norm64(x, c.weight(w), c.angle, c.style, c.amp)
        D = c.D
        live = c.live
        flat = lambda t: t.reshape(live.numel(), -1, D)
        assert_within(flat(got)[live.to(DEV)], flat(y)[live], flat(tol)[live], name)
        assert (flat(got.cpu())[~live] == 0).all()
    # in place, and one of the two: the same bits
    q, k = c.dev("q", "k")
    cea.qk_norm_rope_fwd(q, k, *c.dev("wq", "wk"), q_out=q, k_out=k, **c.kw)
    flat = lambda t: t.reshape(c.live.numel(), -1)[c.live.to(DEV)]
    assert torch.equal(flat(q), flat(outs[0])) and torch.equal(flat(k), flat(outs[1]))
    only, none = cea.qk_norm_rope_fwd(None, *c.dev("k"), None, *c.dev("wk"), **c.kw)[::-1]
    assert none is None and torch.equal(only, outs[1])


@pytest.mark.parametrize("name", NORM)
def test_norm_gradients(name):
    c = NormCase(name)
    ws = cea.qk_norm_workspace(DEV)
    args = c.dev("q", "k", "wq", "wk", "dq", "dk")
    dq, dk, wq, wk = cea.qk_norm_rope_bwd(*args, workspace=ws, **c.kw)
    assert cea.check_status() == 0 and wq.dtype == F32
    live = c.live
    rows = lambda t: t.reshape(live.numel(), -1, t.shape[-1])[live.to(t.device)]
    angle = c.angle.flatten(0, -2)
    for got, got_w, x, w, dy in ((dq, wq, c.q, c.wq, c.dq), (dk, wk, c.k, c.wk, c.dk)):
        dx, tol, dw, tol_w = norm_bwd64(rows(x), c.weight(w), rows(dy), angle[live], c.style, c.amp)
        assert_within(rows(got), dx, tol, name)
        assert_within(got_w, dw, tol_w, name + " weight")
    # over the upstream gradients and over the inputs, on the workspace as it was left: the same bits
    for over in (4, 0):
        again = [t.clone() if t is not None else None for t in args]
        r = cea.qk_norm_rope_bwd(*again, dq=again[over], dk=again[over + 1], workspace=ws, **c.kw)
        assert torch.equal(rows(r[0]), rows(dq)) and torch.equal(rows(r[1]), rows(dk))
        assert torch.equal(r[2], wq) and torch.equal(r[3], wk)
    q, _, dy = args[0], args[1], args[4]
    r = cea.qk_norm_rope_bwd(q, None, args[2], None, dy, None, **c.kw)
    assert torch.equal(rows(r[0]), rows(dq)) and r[1] is None and r[3] is None
    # (the sum over the rows is split otherwise then)
    _, _, dw, tol_w = norm_bwd64(rows(c.q), c.weight(c.wq), rows(c.dq), angle[live], c.style, c.amp)
    assert_within(r[2], dw, tol_w, name + " alone")


def test_norm_gradient_against_differences():
    """A central difference of the plain form in 64 bits along random directions, against the
    kernel's gradients in fp32: the difference is exact to h^2 times the third derivative, 1e-8 of the
    inputs' size 1, and a sum of n products of gradients that are good to 2^-18 is good to
    2^-18 sum |products|."""
    g = torch.Generator().manual_seed(9)
    x, dy = torch.randn(30, 3, 32, generator=g), torch.randn(30, 3, 32, generator=g)
    w = torch.randn(32, generator=g)
    rope = cea.rope_table(24, device=DEV)
    i = torch.arange(12, dtype=torch.float64)
    angle = angles64(torch.arange(30), 10000.0 ** (-2 * i / 24))
    dx, _, dw, _ = cea.qk_norm_rope_bwd(x[None].to(DEV), None, w.to(DEV), None, dy[None].to(DEV), None,
                                        rope=rope)
    f = lambda a, b: (norm64(a, b, angle, "half")[0] * dy.double()).sum()
    for seed in range(5):
        a = torch.randn(x.shape, generator=g, dtype=torch.float64)
        b = torch.randn(w.shape, generator=g, dtype=torch.float64)
        h = 1e-4
        diff = (f(x + h * a, w + h * b) - f(x - h * a, w - h * b)) / (2 * h)
        terms = torch.cat([(dx[0].double().cpu() * a).flatten(), dw.double().cpu() * b])
        assert abs(diff - terms.sum()) <= 2.0 ** -17 * terms.abs().sum() + 1e-5


def test_norm_of_views_and_large_values():
    """Strided tokens of one projection (and of its gradient), heads of 1e18 and of 1e-18."""
    g = torch.Generator().manual_seed(11)
    T, H, K, D = 40, 6, 2, 128
    fused = torch.randn(1, T, H + 2 * K, D, generator=g).to(BF)
    fused[0, 3] *= 1e18
    fused[0, 4] *= 1e-18
    w = torch.randn(D, generator=g).to(BF)
    x = fused.to(DEV)
    q, k = x[:, :, :H], x[:, :, H:H + K]
    rope = cea.rope_table(128, device=DEV)
    oq, ok = cea.qk_norm_rope_fwd(q, k, w.to(DEV), w.to(DEV), rope)
    i = torch.arange(64, dtype=torch.float64)
    angle = angles64(torch.arange(T)[None], 10000.0 ** (-2 * i / 128))
    y, tol = norm64(fused[:, :, :H], w.double(), angle, "half")
    assert_within(oq, y, tol)
    dfused = torch.zeros_like(x)
    dq, dk = dfused[:, :, :H], dfused[:, :, H:H + K]
    cea.qk_norm_rope_bwd(q, k, w.to(DEV), w.to(DEV), oq, ok, rope, dq=dq, dk=dk)
    assert (dfused[:, :, H + K:] == 0).all() and torch.equal(x.cpu(), fused)
    dx, tol, _, _ = norm_bwd64(fused[:, :, :H], w.double(), oq.cpu(), angle, "half")
    assert_within(dq, dx, tol)


def test_norm_without_tokens():
    z = torch.zeros(1, 0, 2, 64, dtype=BF, device=DEV)
    w = torch.ones(64, dtype=BF, device=DEV)
    assert cea.qk_norm_rope_fwd(z, z, w, w)[0].shape == z.shape
    r = cea.qk_norm_rope_bwd(z, None, w, None, z, None)
    assert (r[2] == 0).all()


def test_norm_python_refusals():
    x = torch.zeros(1, 4, 2, 64, dtype=BF, device=DEV)
    w = torch.ones(64, dtype=BF, device=DEV)
    bad = [lambda: cea.qk_norm_rope_fwd(x, x, w[:32], w), lambda: cea.qk_norm_rope_fwd(x, x, w, w.float()),
           lambda: cea.qk_norm_rope_fwd(x, x, w.half(), None), lambda: cea.qk_norm_rope_fwd(x, x, w.cpu(), w),
           lambda: cea.qk_norm_rope_bwd(x, x, w, w, x, None), lambda: cea.qk_norm_rope_bwd(x, None, w, w, x, x),
           lambda: cea.qk_norm_rope_bwd(x, x, w, w, x, x[:, :2]), lambda: cea.qk_norm_rope_bwd(x, x, w, w, x, x.float()),
           lambda: cea.qk_norm_rope_bwd(x, x, w, w, x, x, dq_weight=w), lambda: cea.qk_norm_rope_fwd(x, x, w, w, eps=-1.0)]
    for f in bad:
        with pytest.raises((ValueError, cea.RingAttnError)):
            f()


# ------------------------------------------------------------------------ append --

@pytest.mark.parametrize("dtype,D,rot,style,layout", [
    (BF, 128, 128, "half", "slots"), (BF, 64, 64, "interleaved", "by_slot"), (F32, 128, 62, "half", "heads"),
    (BF, 80, 80, "half", "by_page"), (BF, 128, 0, "half", "by_head"), (F32, 256, 256, "half", "slots")])
@pytest.mark.parametrize("normed", [True, False], ids=["norm", "plain"])
def test_append_at_given_positions(dtype, D, rot, style, layout, normed):
    seqs = [(1, 1), (0, 5), (7, 40), (33, 33), (3, 2)]
    H, K = 6, 2
    c = Cache(seqs, H, K, D, 16, dtype, layout, pad=3, seed=D, garbage=9.0)
    g = torch.Generator().manual_seed(D + rot)
    pos = torch.randint(0, 5000, (c.T,), generator=g).int()
    k, v = (torch.randn(c.T, K, D, generator=g).to(dtype) for _ in "kv")
    wq, wk = (torch.randn(D, generator=g).to(dtype) for _ in "qk")
    kp, vp = c.device_pages(DEV)
    before_k, before_v = kp.cpu().clone(), vp.cpu().clone()
    more = dict(q_weight=wq.to(DEV), k_weight=wk.to(DEV)) if normed else {}
    rope = cea.rope_table(rot, style=style, device=DEV) if rot else None
    q_out = cea.paged_kv_append(k.to(DEV), v.to(DEV), kp, vp, c.table.to(DEV), c.cu.to(DEV),
                                c.kv_lens.to(DEV), rope=rope, q=c.q.to(DEV), positions=pos.to(DEV), **more)
    assert cea.check_status() == 0
    i = torch.arange(rot // 2, dtype=torch.float64)
    angle = angles64(pos, 10000.0 ** (-2 * i / max(rot, 1)))
    n = c.T - 3
    one = torch.ones(D, dtype=torch.float64)
    if normed:
        yq, tq = norm64(c.q, wq.double(), angle, style)
        yk, tk = norm64(k, wk.double(), angle, style)
    else:
        from step_helpers import turn64
        (yq, mq), (yk, mk) = turn64(c.q.double(), angle, style, 1.0), turn64(k.double(), angle, style, 1.0)
        tq, tk = 2.0 ** -20 * mq, 2.0 ** -20 * mk
    assert_within(q_out[:n], yq[:n], tq[:n], "q")
    assert (q_out[n:] == 0).all()
    stored = set()
    kp, vp = kp.cpu(), vp.cpu()
    for s, (a, kv) in enumerate(seqs):
        for j in range(a):
            at = kv - a + j
            if at < 0:
                continue
            page, slot, row = int(c.table[s, at // 16]), at % 16, int(c.cu[s]) + j
            stored.add((page, slot))
            assert torch.equal(vp[page, slot], v[row])
            assert_within(kp[page, slot], yk[row], tk[row], "k")
    for page in range(c.num_pages):
        for slot in range(16):
            if (page, slot) not in stored:
                assert torch.equal(kp[page, slot].view(torch.int16 if dtype == BF else torch.int32),
                                   before_k[page, slot].view(torch.int16 if dtype == BF else torch.int32))
                assert torch.equal(vp[page, slot], before_v[page, slot]) or vp[page, slot].isnan().any()
    if not rot and not normed:
        assert torch.equal(q_out[:n].cpu(), c.q[:n])


def test_append_normalised_without_weights():
    c = Cache([(5, 9)], 2, 1, 64, 4, BF, seed=3)
    k = torch.randn(5, 1, 64, generator=torch.Generator().manual_seed(1)).to(BF)
    kp, vp = c.device_pages(DEV)
    cu, lens, table = c.cu.to(DEV), c.kv_lens.to(DEV), c.table.to(DEV)
    cea.paged_kv_append(k.to(DEV), k.to(DEV), kp, vp, table, cu, lens, normalise=True)
    y, tol = norm64(k, torch.ones(64, dtype=torch.float64), torch.zeros(5, 0, dtype=torch.float64), "half")
    for j in range(5):
        assert_within(kp[c.table[0, (4 + j) // 4], (4 + j) % 4], y[j], tol[j])
    with pytest.raises(ValueError):
        cea.paged_kv_append(k.to(DEV), k.to(DEV), kp, vp, table, cu, lens, k_weight=k[0, 0].to(DEV),
                            normalise=False)
    with pytest.raises(ValueError):
        cea.paged_kv_append(k.to(DEV), k.to(DEV), kp, vp, table, cu, lens, positions=lens)


# -------------------------------------------------------------------------- trees --

# sequences (new tokens, keys), H, H_kv, D, page, dtype, layout, padding rows, words
TREE = {
    "one token": ([(1, 1)], 1, 1, 128, 16, BF, "slots", 0, 1),
    "a small tree": ([(5, 200)], 4, 2, 128, 16, BF, "slots", 0, 1),
    "few rows": ([(3, 90), (4, 300), (1, 7), (0, 9), (2, 2)], 8, 2, 128, 16, BF, "heads", 2, 1),
    "few rows, D 64": ([(4, 77), (2, 1000), (4, 64)], 4, 1, 64, 24, BF, "by_slot", 0, 1),
    "few rows, long": ([(4, 20000)], 4, 1, 128, 64, BF, "slots", 0, 1),
    "many rows": ([(26, 400), (61, 900), (13, 13), (1, 50), (0, 3)], 8, 2, 128, 16, BF, "slots", 3, 2),
    "many rows, D 64": ([(64, 1000), (33, 129)], 16, 4, 64, 32, BF, "by_page", 0, 2),
    "single sub-tiles": ([(20, 2000), (16, 800)], 8, 2, 128, 64, BF, "slots", 0, 1),
    "two hundred nodes": ([(200, 777), (130, 200)], 4, 1, 128, 16, BF, "heads", 1, 7),
    "a wide group": ([(9, 500), (12, 70)], 64, 1, 128, 16, BF, "slots", 0, 1),
    "words too few": ([(50, 300), (10, 20)], 8, 2, 128, 16, BF, "slots", 0, 1),
    "more new than keys": ([(40, 25), (30, 0), (8, 3)], 8, 2, 64, 16, BF, "slots", 2, 2),
    "pages of 3": ([(12, 100), (40, 44)], 8, 2, 64, 3, BF, "slots", 0, 2),
    "long context": ([(60, 9000)], 8, 2, 128, 128, BF, "slots", 0, 2),
    # many tiles
    "many, few rows": ([((i * 3) % 5, 30 * i + 6) for i in range(20)], 8, 4, 128, 16, BF, "slots", 2, 1),
    "many, few rows, D 64": ([(4, 50 + 90 * i) for i in range(12)], 16, 4, 64, 8, BF, "heads", 0, 1),
    "many, long": ([(4, 3000), (3, 100)] + [(1, 500)] * 9, 16, 4, 128, 64, BF, "slots", 0, 1),
    "many, many rows": ([((i * 13) % 62, 40 * i + 62) for i in range(11)], 16, 4, 128, 16, BF, "by_slot", 3, 2),
    "many, single sub-tiles": ([(20 + i % 7, 100 * i + 30) for i in range(10)], 16, 4, 128, 64, BF, "slots", 0, 1),
    "many, D 64": ([((i * 29) % 100, 30 * i + 100) for i in range(10)], 16, 4, 64, 32, BF, "by_page", 1, 4),
    "many, words too few": ([(50, 55 + i) for i in range(10)], 8, 4, 128, 16, BF, "slots", 0, 1),
    "many, more new than keys": ([(30 + i, 20 + 2 * i) for i in range(12)], 8, 4, 64, 16, BF, "slots", 2, 2),
    "a wide group, many": ([(5, 200 + i) for i in range(12)], 128, 4, 64, 16, BF, "slots", 0, 1),
    "pages of 3, many": ([(12, 100 + i) for i in range(12)], 8, 4, 64, 3, BF, "slots", 0, 1),
    "one long context": ([(64, 30000)], 8, 2, 128, 64, BF, "slots", 0, 2),
    "two rows of a tile": ([(3, 700)], 16, 2, 128, 16, BF, "by_head", 0, 1),
    "no keys": ([(5, 0), (0, 0), (3, 1)], 8, 2, 128, 16, BF, "slots", 1, 1),
    "fp32": ([(5, 90), (7, 40), (1, 1), (0, 3)], 6, 2, 128, 16, F32, "slots", 1, 1),
    "fp32 wide": ([(9, 130), (3, 3)], 5, 1, 256, 8, F32, "heads", 0, 1),
    "fp32 rows": ([(64, 300), (90, 777)], 8, 4, 64, 16, F32, "slots", 2, 3),
    "fp32 rows 128": ([(120, 900), (70, 71)], 16, 4, 128, 24, F32, "by_page", 0, 4),
    "fp32 rows 192": ([(150, 400)], 16, 4, 192, 16, F32, "slots", 0, 5),
    "fp32, 16 rows": ([(4, 300), (3, 77)], 8, 2, 128, 16, F32, "heads", 2, 1),
    "fp32, 32 rows": ([(8, 500), (5, 64), (0, 9)], 8, 2, 100, 16, F32, "slots", 0, 1),
    "fp32, narrow": ([(8, 500), (30, 64)], 4, 2, 36, 8, F32, "by_head", 0, 1),
    "fp32, 4 dims": ([(9, 130)], 4, 1, 4, 16, F32, "slots", 0, 1),
    "fp32, many": ([(3, 40 + 30 * i) for i in range(20)], 8, 4, 64, 16, F32, "slots", 1, 1),
    "fp32, many rows of many": ([(40, 50 + 30 * i) for i in range(12)], 16, 4, 128, 16, F32, "slots", 0, 2),
    "fp32, a long context": ([(20, 9000)], 4, 2, 64, 64, F32, "slots", 0, 1),
    "fp32, many of 192": ([(3, 40 + 30 * i) for i in range(30)], 8, 4, 192, 16, F32, "slots", 0, 1),
    "fp32 rows 256": ([(100, 260)], 32, 4, 256, 16, F32, "by_slot", 0, 2),
}


def tree_masks(c, words, kind, seed=0):
    """(what new tokens see, masks) of a cache's sequences: trees, anything, or nothing at all."""
    g = torch.Generator().manual_seed(seed)
    seen = []
    for n, _ in c.seqs:
        if kind == "trees":
            s = ancestors(random_parents(n, g))[0]
        elif kind == "any":
            s = torch.rand(n, n, generator=g) < 0.4
        else:
            s = torch.zeros(n, n, dtype=torch.bool)
        s[:, 32 * words:] = False
        seen.append(s)
    pad = c.T - int(c.cu[-1])
    # padding rows, and bits behind a sequence's tokens, hold anything
    rows = [mask_words(torch.cat([s, torch.ones(len(s), max(0, 32 * words - len(s)), dtype=torch.bool)], 1),
                       words) for s in seen]
    return seen, torch.cat(rows + [torch.full((pad, words), -1, dtype=torch.int32)])


def tree_attend(c, masks, room=0, **kw):
    """room: keys that the page table has columns for, if more than are used.  Calls of few tiles
    whose table is short go to kernels of their own."""
    kp, vp = c.device_pages(DEV)
    table = torch.full((len(c.seqs), max(c.table.shape[1], room // c.page)), -1, dtype=torch.int32)
    table[:, :c.table.shape[1]] = c.table
    r = cea.paged_attn_fwd(c.q.to(DEV), kp, vp, table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV),
                           masks=masks.to(DEV), **kw)
    assert cea.check_status() == 0
    return r


@pytest.mark.parametrize("name", TREE)
@pytest.mark.parametrize("kind", ["trees", "any", "none"])
@pytest.mark.parametrize("room", [0, 1 << 18], ids=["short", "long"])
def test_tree_attention(name, kind, room):
    """Slots that hold no key are NaN throughout, table entries behind a sequence's pages -1."""
    seqs, H, K, D, page, dtype, layout, pad, words = TREE[name]
    c = Cache(seqs, H, K, D, page, dtype, layout, pad, seed=len(name))
    seen, masks = tree_masks(c, words, kind, len(name))
    out = torch.full((c.T, H, D), 3.0, dtype=dtype, device=DEV)
    lse = torch.full((c.T, H), 5.0, device=DEV)
    ws = cea.paged_attn_workspace(D, dtype, DEV)
    tree_attend(c, masks, room, out=out, lse=lse, workspace=ws)
    assert_attends(out, lse, tree_reference(c, seen), name)
    if pad:                                        # rows behind the last sequence stay
        assert (out[-pad:] == 3).all() and (lse[-pad:] == 5).all()
    wide = torch.zeros(c.T, words + 3, dtype=torch.int32)
    wide[:, 1:1 + words] = masks                   # strided masks: the same bits
    again, none = tree_attend(c, wide.to(DEV)[:, 1:1 + words], room, workspace=ws, want_lse=False)
    n = c.T - pad
    assert none is None and torch.equal(again[:n], out[:n])


def test_a_chain_is_the_causal_rule():
    for seqs, dtype in (([(60, 500), (33, 64)], BF), ([(3, 400), (4, 30)], BF), ([(9, 100)], F32),
                        ([(60, 300 + i) for i in range(8)], BF), ([(3, 100)] * 20, BF)):
        c = Cache(seqs, 8, 2, 128, 16, dtype, seed=8)
        masks = torch.cat([mask_words(torch.ones(n, n).tril().bool(), 2) for n, _ in seqs])
        for room in (0, 1 << 18):
            out, lse = tree_attend(c, masks, room)
            assert_attends(out, lse, c.reference(True))


def test_unseen_keys_that_are_not_finite():
    """A drafted token's key that is infinite or NaN reaches the rows that see it, and no others; in
    fp32 its value too."""
    for seqs, H, dtype in (([(4, 100), (3, 50)], 4, BF), ([(40, 300), (20, 90)], 8, BF),
                           ([(4, 100)] + [(3, 50)] * 20, 4, BF), ([(40, 300)] + [(20, 90)] * 12, 8, BF),
                           ([(5, 60), (4, 33)], 4, F32), ([(100, 300)], 8, F32)):
        c = Cache(seqs, H, 2, 64, 16, dtype, seed=9)
        seen, masks = tree_masks(c, 4, "trees", 5)
        ref = tree_reference(c, seen)
        n, kv = seqs[0]
        for j, x in ((n - 1, float("nan")), (n - 2, float("inf"))):
            at = kv - n + j
            c.k[c.table[0, at // 16], at % 16] = x
            if dtype == F32:
                c.v[c.table[0, at // 16], at % 16] = x
        hit = torch.zeros(c.T, dtype=torch.bool)
        hit[:n] = seen[0][:, n - 1] | seen[0][:, n - 2]
        assert hit.any() and not hit.all()
        for room in (0, 1 << 18):
            out, lse = tree_attend(c, masks, room)
            assert out[hit.to(DEV)].isnan().flatten(1).any(1).all()
            assert_attends(out[~hit.to(DEV)], lse[~hit.to(DEV)], tuple(x[~hit] for x in ref))


def test_tree_python_refusals():
    c = Cache([(4, 40)], 2, 1, 64, 16, BF, seed=1)
    for m in (torch.zeros(3, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
              torch.zeros(4, 1, dtype=torch.int64), torch.zeros(4, 0, dtype=torch.int32)):
        with pytest.raises((ValueError, cea.RingAttnError)):
            tree_attend(c, m)


# --------------------------------------------------------------------------- keep --

@pytest.mark.parametrize("dtype,D,layout,layers,page", [
    (BF, 128, "slots", 1, 16), (BF, 64, "heads", 3, 8), (F32, 80, "by_page", 2, 5), (BF, 256, "by_slot", 1, 64),
    (F32, 4, "by_head", 4, 1)])
def test_keep(dtype, D, layout, layers, page):
    seqs = [(26, 100), (1, 1), (0, 30), (70, 75), (5, 3), (40, 40), (12, 12), (8, 90)]
    kept = [[0, 2, 5, 25], [0], [3], [i for i in range(70) if i % 2], [3, 4], [0, 1, 2, 39, 38, 5], [-1],
            [cea.KEEP_ALL, 3]]
    moved = [[0, 2, 5, 25], [0], [], [i for i in range(70) if i % 2], [3, 4], [0, 1, 2, 39], [], list(range(8))]
    width = 40
    caches = [Cache(seqs, 1, 2, D, page, dtype, layout, seed=50 + i, garbage=4.0) for i in range(layers)]
    c = caches[0]
    table = c.table
    pairs = [x.device_pages(DEV) for x in caches]
    if layers > 1:
        both = [torch.stack([p[i] for p in pairs]) for i in (0, 1)]
        if layout == "heads":                       # heads before slots, layers outermost
            both = [b.permute(0, 1, 3, 2, 4).contiguous().permute(0, 1, 3, 2, 4) for b in both]
        k, v = both
    else:
        k, v = pairs[0]
    want = [[x.cpu().clone().reshape(layers, -1, page, 2, D) for x in (k, v)]][0]
    rows = torch.full((len(seqs), width), -1, dtype=torch.int32)
    for i, r in enumerate(kept):
        rows[i, :len(r)] = torch.tensor(r)
    kv_lens = c.kv_lens.to(DEV)
    lens = cea.paged_kv_keep(rows.to(DEV), k, v, table.to(DEV), c.cu.to(DEV), kv_lens)
    assert cea.check_status() == 0
    assert lens.tolist() == [max(kv - n + len(m), 0) for (n, kv), m in zip(seqs, moved)]
    assert torch.equal(kv_lens.cpu(), c.kv_lens)
    for g, ((n, kv), m) in enumerate(zip(seqs, moved)):
        for i, node in enumerate(m):
            a, b = kv - n + node, kv - n + i
            if a < 0 or b < 0:
                continue
            for x in want:
                x[:, table[g, b // page], b % page] = x[:, table[g, a // page], a % page].clone()
    for got, x in zip((k, v), want):
        assert torch.equal(got.cpu().reshape(x.shape), x)


def test_keep_leaves_bad_pages_alone():
    c = Cache([(6, 12)], 1, 1, 64, 4, BF, seed=2, garbage=1.0)
    kp, vp = c.device_pages(DEV)
    table = c.table.clone()
    table[0, 2] = 10 ** 6
    before = kp.clone()
    lens = cea.paged_kv_keep(ints([[1, 2, 5]]), kp, vp, table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV))
    assert cea.check_status() == 0 and lens.tolist() == [9]
    want = before.clone()
    want[table[0, 1], 2] = before[table[0, 1], 3]          # token 1 to place 0; 2 and 5 lie in no page
    assert torch.equal(kp, want)


# -------------------------------------------------------------------- large and apart --

def test_slots_beyond_32_bits():
    p = Pool(6000, 2, 2100, 1 << 20)
    p.reserve([0, 0], [2 ** 31 - 9, 2 ** 31 - 1], 4)          # lengths only: pages for both
    assert int(p.pool.count) == 6000 - 4096
    p.reserve([4, 0], [2 ** 31 - 9, 2 ** 31 - 1], 4)
    p.reserve([9, 0], [2 ** 31 - 9, 0], 12)
    assert int(p.pool.status) == 3


def test_caches_beyond_32_bits():
    """Pages whose elements pass 2^32: appended to, attended to and kept."""
    g = torch.Generator().manual_seed(3)
    page, K, D, H = 16, 8, 128, 16
    pages = (1 << 32) // (page * K * D) + 8
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 18 GB of device memory")
    c = Cache([(20, 45)], H, K, D, page, BF, seed=6)
    kp, vp = (torch.empty(pages, page, K, D, dtype=BF, device=DEV) for _ in "kv")
    table = torch.tensor([[pages - 3, 1, pages - 1]], dtype=torch.int32, device=DEV)
    for j in range(3):
        kp[table[0, j]], vp[table[0, j]] = c.k[c.table[0, j]].to(DEV), c.v[c.table[0, j]].to(DEV)
    x = torch.randn(20, K, D, generator=g).to(BF).to(DEV)
    cu, lens = c.cu.to(DEV), c.kv_lens.to(DEV)
    for j in range(20):                             # the reference's keys: what the append is to store
        at = 25 + j
        c.k[c.table[0, at // page], at % page] = x[j].cpu()
        c.v[c.table[0, at // page], at % page] = x[j].cpu()
    cea.paged_kv_append(x, x, kp, vp, table, cu, lens, positions=torch.zeros(20, dtype=torch.int32, device=DEV))
    seen, masks = tree_masks(c, 1, "trees", 2)
    for room in (3, 4000):                          # (few tiles, and the kernel for many)
        wide = torch.full((1, room), -1, dtype=torch.int32, device=DEV)
        wide[:, :3] = table
        out, lse = cea.paged_attn_fwd(c.q.to(DEV), kp, vp, wide, cu, lens, masks=masks.to(DEV))
        assert_attends(out, lse, tree_reference(c, seen))
    cea.paged_kv_keep(ints([[3, 9, 19]]), kp, vp, table, cu, lens)
    assert cea.check_status() == 0
    for i, node in enumerate((3, 9, 19)):
        at = 25 + i
        assert torch.equal(kp[table[0, at // page], at % page], x[node])
        assert torch.equal(vp[table[0, at // page], at % page], x[node])


def test_on_streams_of_their_own():
    """Every call on a stream that is not the current one, beside work on the current one."""
    s = torch.cuda.Stream()
    c = Cache([(9, 200), (4, 77)], 8, 2, 128, 16, BF, seed=4)
    seen, masks = tree_masks(c, 1, "trees", 3)
    kp, vp = c.device_pages(DEV)
    q, table, cu, lens, m = (t.to(DEV) for t in (c.q, c.table, c.cu, c.kv_lens, masks))
    pool, step = cea.page_pool(30, 2, DEV), cea.paged_step(2, 13, 1, DEV)
    own, new = torch.full((2, 13), -1, dtype=torch.int32, device=DEV), ints([9, 4])
    zero, k2, v2 = ints([0, 0]), kp.clone(), vp.clone()
    kept, w = ints([[0, 2, -1], [1, 3, -1]]), torch.ones(128, dtype=BF, device=DEV)
    x = q[:, :2].contiguous()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = cea.paged_attn_fwd(q, kp, vp, table, cu, lens, masks=m, stream=s)
    cea.paged_reserve(pool, new, zero, own, 16, step, stream=s)
    cea.paged_release(pool, zero, own, 16, stream=s)
    cea.paged_kv_append(x, x, k2, v2, table, cu, lens, k_weight=w, stream=s)
    left = cea.paged_kv_keep(kept, k2, v2, table, cu, lens, stream=s)
    busy = torch.randn(2000, 2000, device=DEV) @ torch.randn(2000, 2000, device=DEV)
    s.synchronize()
    assert busy.isfinite().all() and cea.check_status(s) == 0
    assert_attends(out, lse, tree_reference(c, seen))
    assert step.cu_new.tolist() == [0, 9, 13] and int(pool.count) == 30 and left.tolist() == [193, 75]
    y, tol = norm64(x.cpu(), torch.ones(128, dtype=torch.float64), torch.zeros(13, 0, dtype=torch.float64), "half")
    at = 200 - 9 + 1                                # node 2 went to place 1 of the first sequence's step
    assert_within(k2[table[0, at // 16], at % 16], y[2], tol[2])


# ---------------------------------------------------------------------- together --

def drafting_step(pool, lens, new, parents, kept, qkv, table, k, v, wq, wk, rope, page, step, ws, out):
    """What a program does with a step of drafted trees, one layer: no host reads."""
    cea.paged_reserve(pool, new, lens, table, page, step, parents=parents)
    H = out.shape[1]
    K = k.shape[2]
    q = cea.paged_kv_append(qkv[:, H:H + K], qkv[:, H + K:], k, v, table, step.cu_new, step.kv_lens,
                            rope=rope, q=qkv[:, :H], positions=step.positions, q_weight=wq, k_weight=wk)
    cea.paged_attn_fwd(q, k, v, table, step.cu_new, step.kv_lens, masks=step.masks, out=out, workspace=ws)
    cea.paged_kv_keep(kept, k, v, table, step.cu_new, step.kv_lens, lens=lens)
    cea.paged_release(pool, lens, table, page)


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("dtype,H,K,D", [(BF, 8, 2, 128), (F32, 4, 2, 64)])
def test_steps_of_drafted_trees(captured, dtype, H, K, D):
    """Prompts and then drafted trees, eight steps over the same buffers (in a replayed graph, too),
    against sequences kept as plain lists of normalised keys and values in 64 bits.  A key has been
    rounded to its type once, so the plain form takes the cache's own keys where it has
    checked them (test_append_at_given_positions), and the attention is bounded as there."""
    g = torch.Generator().manual_seed(40 + D)
    n_seqs, page, words, T = 4, 8, 2, 130
    pool = cea.page_pool(60, n_seqs, DEV)
    table = torch.full((n_seqs, 20), -1, dtype=torch.int32, device=DEV)
    k = torch.full((60, page, K, D), float("nan"), dtype=dtype, device=DEV)
    v = k.clone()
    step = cea.paged_step(n_seqs, T, words, DEV)
    lens, new, kept = ints([0] * n_seqs), ints([0] * n_seqs), torch.zeros(n_seqs, 6, dtype=torch.int32, device=DEV)
    parents = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    qkv = torch.zeros(T, H + 2 * K, D, dtype=dtype, device=DEV)
    wq, wk = (torch.randn(D, generator=g).to(dtype).to(DEV) for _ in "qk")
    rope, ws = cea.rope_table(D, device=DEV), cea.paged_attn_workspace(D, dtype, DEV)
    out = torch.zeros(T, H, D, dtype=dtype, device=DEV)
    args = (pool, lens, new, parents, kept, qkv, table, k, v, wq, wk, rope, page, step, ws, out)
    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            drafting_step(*args)                    # no tokens yet: changes nothing
        torch.cuda.current_stream().wait_stream(side)
        assert lens.tolist() == [0] * n_seqs and int(pool.count) == 60
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            drafting_step(*args)
    history = [[] for _ in range(n_seqs)]           # (key, value) of every token, as inputs
    freq = 10000.0 ** (-2 * torch.arange(D // 2, dtype=torch.float64) / D)
    for turn in range(8):
        if turn == 0:
            n = [30, 1, 0, 17]                      # prompts: a chain each, all kept
        elif turn == 5:
            history[1], n = [], [20, 25, 33, 1]     # a sequence has ended, another takes its place
            lens[1] = 0
        else:
            n = torch.randint(0, 33, (n_seqs,), generator=g).tolist()
        chain = turn == 0
        trees = [list(range(-1, a - 1)) if chain else random_parents(a, g) for a in n]
        paths = []
        for a, t in zip(n, trees):
            node, path = (int(torch.randint(0, a, (1,), generator=g)) if a else -1), []
            while node >= 0:
                path.append(node)
                node = t[node]
            paths.append(path[::-1][:6])
        x = torch.randn(T, H + 2 * K, D, generator=g).to(dtype)
        new.copy_(ints(n))
        flat = [p for t in trees for p in t]
        parents.copy_(ints(flat + [-1] * (T - len(flat))))
        rows = [[cea.KEEP_ALL] + [-1] * 5 if chain else p + [-1] * (6 - len(p)) for p in paths]
        kept.copy_(ints(rows))
        qkv.copy_(x.to(DEV))
        if captured:
            graph.replay()
        else:
            drafting_step(*args)
        assert cea.check_status() == 0 and int(pool.status) == 0
        at = 0
        for s in range(n_seqs):
            seen, depth = ancestors(trees[s])
            rowx = x[at:at + n[s]]
            base = len(history[s])
            pos = torch.tensor([base + d for d in depth], dtype=torch.float64)
            kk = norm64(rowx[:, H:H + K], wk.double().cpu(), angles64(pos, freq), "half")[0].to(dtype)
            qq = norm64(rowx[:, :H], wq.double().cpu(), angles64(pos, freq), "half")[0].to(dtype).double()
            vv = rowx[:, H + K:]
            keys = torch.stack([h[0] for h in history[s]] + list(kk)) if base + n[s] else torch.zeros(0, K, D)
            vals = torch.stack([h[1] for h in history[s]] + list(vv)) if base + n[s] else torch.zeros(0, K, D)
            hidden = torch.cat([torch.zeros(n[s], base, dtype=torch.bool), ~seen], 1)
            for h in range(H if n[s] else 0):
                kh, vh = keys[:, h // (H // K)].double(), vals[:, h // (H // K)].double()
                sc = (qq[:, h] @ kh.T / D ** 0.5).masked_fill(hidden, float("-inf"))
                S = qq[:, h].abs() @ kh.T.abs() / D ** 0.5
                w = torch.softmax(sc, -1)
                want, size = w @ vh, w @ vh.abs()
                # A query or key that the kernel rounds the other way is off by one step of its
                # type (2 half steps), so a score by 4 half steps of S, a weight by as much
                # relative to the others, twice that with the sum's; then the attention's own.
                half = torch.finfo(dtype).eps / 2
                rel = 2 * (4 * half * (1 + 2.0 ** -8) + 160 * 2.0 ** -24) * S.amax(-1, keepdim=True) + 2.0 ** -15
                rel = torch.expm1(rel)
                low = 2.0 ** -8 if dtype == BF else 2.0 ** -15
                tol = (rel + low) * size + half * (want.abs() + (rel + low) * size)
                err = (out[at:at + n[s], h].double().cpu() - want).abs()
                assert (err <= tol).all(), (turn, s, h, float((err / tol).max()))
            nodes = range(n[s]) if chain else paths[s]
            history[s] += [(kk[i], vv[i]) for i in nodes]
            at += n[s]
        assert lens.tolist() == [len(h) for h in history]
        held = [-(-len(h) // page) for h in history]
        assert pool.held.tolist() == held and int(pool.count) == 60 - sum(held)
        # the cache holds what was kept, where its sequence has it
        kc, vc, tc = k.cpu(), v.cpu(), table.tolist()
        assert len({p for t, h in zip(tc, held) for p in t[:h]}) == sum(held)
        for s, h in enumerate(history):
            for j, (key, val) in enumerate(h):
                p, o = tc[s][j // page], j % page
                assert torch.equal(vc[p, o], val)
                off = (kc[p, o].double() - key.double()).abs()
                assert (off <= torch.finfo(dtype).eps * 1.01 * key.double().abs() + 1e-6).all()


def test_training_through_normalised_heads():
    """Norm and rotation, ring attention, and back: the weights' gradients against a 64-bit plain form
    on the attention's own gradients (bounded as test_norm_gradients), and of the right sign along a
    step."""
    g = torch.Generator().manual_seed(77)
    B, L, H, D = 1, 1024, 2, 128
    x = [torch.randn(B, L, H, D, generator=g).to(BF).to(DEV) for _ in range(4)]
    w = [torch.randn(D, generator=g).to(BF).to(DEV) for _ in "qk"]
    rope = cea.rope_table(D, device=DEV)
    pos = torch.tensor(cea.zigzag_positions(L, 2))
    kw = dict(rope=rope, layout="zigzag", P=2)
    q, k = cea.qk_norm_rope_fwd(x[0], x[1], *w, **kw)
    out, lse = cea.ring_attn_fwd_zigzag(q, k, x[2], P=2)
    dq, dk, _ = cea.ring_attn_bwd_zigzag(q, k, x[2], out, lse, x[3], P=2)
    gq, gk, wq, wk = cea.qk_norm_rope_bwd(x[0], x[1], *w, dq, dk, **kw)
    assert cea.check_status() == 0
    freq = 10000.0 ** (-2 * torch.arange(D // 2, dtype=torch.float64) / D)
    angle = angles64(pos, freq)[None]
    for a, wt, dy, got, got_w in ((x[0], w[0], dq, gq, wq), (x[1], w[1], dk, gk, wk)):
        dx, tol, dw, tol_w = norm_bwd64(a.cpu(), wt.double().cpu(), dy.cpu(), angle, "half")
        assert_within(got, dx, tol)
        assert_within(got_w, dw, tol_w)


def test_other_streams_and_a_captured_backward():
    """Calls on a stream of their own, and a backward replayed in a graph while the next eager call
    runs on the same tensors."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 300, 4, 128, generator=g).to(BF).to(DEV)
    y = torch.randn(1, 300, 4, 128, generator=g).to(BF).to(DEV)
    w = torch.randn(128, generator=g).to(BF).to(DEV)
    rope = cea.rope_table(128, device=DEV)
    want = cea.qk_norm_rope_bwd(x, None, w, None, y, None, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = cea.qk_norm_rope_bwd(x, None, w, None, y, None, rope, stream=s)
    fwd = cea.qk_norm_rope_fwd(x, None, w, None, rope, stream=s)[0]
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert torch.equal(fwd, cea.qk_norm_rope_fwd(x, None, w, None, rope)[0])
    ws, dx, dw = cea.qk_norm_workspace(DEV), torch.empty_like(x), torch.empty(128, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cea.qk_norm_rope_bwd(x, None, w, None, y, None, rope, dq=dx, dq_weight=dw, workspace=ws)
    for _ in range(3):
        dx.zero_()
        graph.replay()
        cea.qk_norm_rope_bwd(x, None, w, None, y, None, rope, workspace=ws)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[2])
    with pytest.raises(ValueError):
        cea.qk_norm_rope_fwd(x, None, w.cpu(), None, rope)


def test_index_checked_build(monkeypatch):
    """Every entry point in the build that checks its indexes: no check fails, and the same bits."""
    def everything():
        res = []
        for name in ("odd tokens", "packed", "interleaved part", "odd half", "fp32 256, part", "no rotation",
                     "96 dims", "72 dims, odd half", "fp32 256 odd half"):
            c = NormCase(name)
            res += cea.qk_norm_rope_fwd(*c.dev("q", "k", "wq", "wk"), **c.kw)
            c.kw["dq"], c.kw["dk"] = torch.zeros_like(c.q, device=DEV), torch.zeros_like(c.k, device=DEV)
            res += cea.qk_norm_rope_bwd(*c.dev("q", "k", "wq", "wk", "dq", "dk"), **c.kw)
        for name in ("few rows", "many rows", "more new than keys", "many, few rows", "many, many rows",
                     "fp32", "fp32 rows"):
            seqs, H, K, D, page, dtype, layout, pad, words = TREE[name]
            c = Cache(seqs, H, K, D, page, dtype, layout, pad, seed=1)
            for room in (0, 1 << 18):
                res += tree_attend(c, tree_masks(c, words, "trees")[1], room)
            kp, vp = c.device_pages(DEV)
            kept = ints([[0, 2, 3] for _ in seqs])
            res.append(cea.paged_kv_keep(kept, kp, vp, c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV)))
            x = c.q[:, :K].contiguous().to(DEV)
            w = torch.ones(D, dtype=dtype, device=DEV)
            cea.paged_kv_append(x, x, kp, vp, c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV), k_weight=w,
                                positions=torch.arange(c.T, dtype=torch.int32, device=DEV))
            res += [kp, vp]
        pool, table = cea.page_pool(90, 5, DEV), torch.full((5, 9), -1, dtype=torch.int32, device=DEV)
        step = cea.paged_step(5, 400, 3, DEV)
        g = torch.Generator().manual_seed(1)
        parents = ints([p for n in (70, 1, 0, 44, 100) for p in random_parents(n, g)] + [5] * 185)
        cea.paged_reserve(pool, ints([70, 1, 0, 44, 100]), ints([0, 5, 3, 0, 31]), table, 16, step, parents)
        cea.paged_release(pool, ints([0, 5, 3, 20, 31]), table, 16)
        res += [*step, pool.held, pool.state, table, pool.free]
        assert cea.check_status() == 0
        return [t.clone() for t in res if t is not None]
    normal = everything()
    monkeypatch.setattr(cea, "_lib", cea.load_debug_library(build_if_missing=True))
    checked = everything()
    for a, b in zip(normal, checked):
        assert torch.equal(a.nan_to_num(nan=7.0) if a.is_floating_point() else a,
                           b.nan_to_num(nan=7.0) if b.is_floating_point() else b)
