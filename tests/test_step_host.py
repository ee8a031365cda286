"""A step of drafted tokens, host side (no GPU): the descriptors' layouts and every refusal of its
entry points, which come back before anything is launched."""
import ctypes

import pytest
import torch

import context_exact_attention_gb300 as cea
from context_exact_attention_gb300 import _build
from step_helpers import PoolModel, ancestors, mask_words
from test_paged_host import COMMON, INDIVISIBLE, INVALID, MISALIGNED, OK, S, UNSUPPORTED, at, paged, rope

NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return cea.load_library()


def off(i, n):
    return ctypes.c_void_p((i + 1 << 40) + n)


def test_layouts():
    assert ctypes.sizeof(cea.HeadNorm) == 32 and cea.HeadNorm.eps.offset == 20
    assert ctypes.sizeof(cea.PagePoolDesc) == 32 and cea.PagePoolDesc.state.offset == 24
    assert cea._HEAD_NORM.pack(5, 6, 1, 0.5, 1.0) == bytes(cea.HeadNorm(5, 6, 1, 0.5, 1.0))


def desc(**kw):
    d = dict(B=1, L=8, H=4, H_kv=2, D=64, P=1, layout=0, cu_seqlens=None, n_seqs=0, positions=None,
             position_offset=0, dtype=0, q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0)
    d.update(kw)
    return ctypes.byref(cea.RopeDesc(**d))


def norm(q=at(20), k=at(21), dtype=0, eps=1e-6, offset=0.0):
    return ctypes.byref(cea.HeadNorm(q, k, dtype, eps, offset))


BAD_NORMS = [(dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
             (dict(eps=float("inf")), INVALID), (dict(offset=float("inf")), INVALID),
             (dict(dtype=2), UNSUPPORTED), (dict(q=off(20, 1)), MISALIGNED),
             (dict(k=off(21, 2), dtype=1), MISALIGNED)]


def test_norm_refusals(lib):
    def call(d=desc(), r=rope(), n=norm(), q=at(0), k=at(1), qo=at(2), ko=at(3)):
        return lib.qk_norm_rope_fwd(d, r, n, q, k, qo, ko, S)

    assert call(d=None) == INVALID and call(n=None) == INVALID
    for kw, code in BAD_NORMS:
        assert call(n=norm(**kw)) == code, kw
    for kw in (dict(q=NULL), dict(qo=NULL), dict(k=NULL), dict(ko=NULL)):
        assert call(**kw) == INVALID, kw
    assert call(d=desc(D=60)) == UNSUPPORTED and call(d=desc(D=264)) == UNSUPPORTED
    assert call(d=desc(dtype=2)) == UNSUPPORTED and call(r=rope(rot_dim=66)) == INVALID
    assert call(d=desc(layout=1, L=6, P=2)) == INDIVISIBLE
    assert call(qo=at(1)) == INVALID and call(ko=at(0)) == INVALID and call(qo=off(0, 128)) == INVALID
    assert call(d=desc(q_stride=128)) == INVALID and call(d=desc(q_stride=260)) == MISALIGNED
    # outputs on the weights
    assert call(n=norm(q=at(2))) == INVALID and call(n=norm(k=off(3, 64))) == INVALID


def test_norm_backward_refusals(lib):
    need = lib.qk_norm_workspace_bytes()
    assert need > 0

    def call(d=desc(), r=rope(), n=norm(), q=at(0), k=at(1), y=at(2), ys=0, z=at(3), zs=0, dq=at(4),
             dk=at(5), wq=at(6), wk=at(7), ws=at(8), size=need):
        return lib.qk_norm_rope_bwd(d, r, n, q, k, y, ys, z, zs, dq, dk, wq, wk, ws,
                                    ctypes.c_ulonglong(size), S)

    assert call(d=None) == INVALID and call(n=None) == INVALID
    for kw, code in BAD_NORMS:
        assert call(n=norm(**kw)) == code, kw
    for kw in (dict(q=NULL), dict(y=NULL), dict(z=NULL), dict(dq=NULL), dict(ws=NULL), dict(size=need - 1)):
        assert call(**kw) == INVALID, kw
    # gradients of what is not there
    no_k = dict(d=desc(H_kv=0), k=NULL, z=NULL, dk=NULL)
    assert call(**no_k) == INVALID
    assert call(ys=128) == INVALID and call(zs=132) == MISALIGNED
    assert call(y=off(2, 8)) == MISALIGNED and call(wq=off(6, 2)) == MISALIGNED
    assert call(ws=off(8, 128)) == MISALIGNED
    # overlaps: a gradient with the other's upstream one, results with inputs and one another
    assert call(dq=at(3)) == INVALID and call(dk=at(2)) == INVALID and call(dq=off(2, 512)) == INVALID
    assert call(wq=at(0)) == INVALID and call(wk=at(3)) == INVALID and call(wq=at(7)) == INVALID
    assert call(wq=at(4)) == INVALID and call(ws=at(5)) == INVALID and call(ws=at(6)) == INVALID
    assert call(wq=at(20)) == INVALID and call(n=norm(k=at(5))) == INVALID


def test_append_with_norms_refusals(lib):
    def call(d=paged(), r=rope(), n=norm(), pos=at(22), q=at(0), k=at(1), v=at(2), qo=at(3), kp=at(4),
             vp=at(5)):
        return lib.paged_kv_append_ex(d, r, n, pos, q, 0, k, 0, v, 0, qo, 0, kp, vp, S)

    for kw, code in COMMON:
        assert call(d=paged(**kw)) == code, kw
    for kw, code in BAD_NORMS:
        assert call(n=norm(**kw)) == code, kw
    assert call(pos=off(22, 2)) == MISALIGNED
    assert call(pos=at(3)) == INVALID and call(pos=at(4)) == INVALID
    assert call(n=norm(q=at(4))) == INVALID and call(n=norm(k=at(3))) == INVALID
    assert call(d=paged(T=0)) == OK and call(d=paged(T=0), n=None, pos=NULL) == OK


def test_tree_attention_refusals(lib):
    need = lib.paged_attn_workspace_bytes(64, 0)

    def call(d=paged(), m=at(9), words=1, stride=0, out=at(3), lse=at(4), ws=at(5)):
        return lib.paged_attn_tree_fwd(d, m, words, stride, at(0), 0, at(1), at(2), out, lse, ws,
                                       ctypes.c_ulonglong(need), S)

    for kw, code in COMMON:
        assert call(d=paged(**kw)) == code, kw
    assert call(m=NULL) == INVALID and call(words=0) == INVALID and call(words=2, stride=1) == INVALID
    assert call(m=off(9, 2)) == MISALIGNED
    for kw in (dict(out=at(9)), dict(lse=at(9)), dict(ws=at(9))):
        assert call(**kw) == INVALID, kw
    assert call(d=paged(T=0)) == OK


def pool(num_pages=50, n_seqs=3, free=at(0), held=at(1), state=at(2)):
    return ctypes.byref(cea.PagePoolDesc(num_pages, n_seqs, free, held, state))


BAD_POOLS = [(dict(num_pages=0), INVALID), (dict(n_seqs=0), INVALID), (dict(free=NULL), INVALID),
             (dict(held=NULL), INVALID), (dict(state=NULL), INVALID), (dict(n_seqs=8193), UNSUPPORTED),
             (dict(num_pages=2 ** 31 - 1), UNSUPPORTED), (dict(held=off(1, 2)), MISALIGNED),
             (dict(held=at(0)), INVALID), (dict(state=at(1)), INVALID), (dict(free=at(4)), INVALID)]


def test_reserve_refusals(lib):
    def call(p=pool(), new=at(3), lens=at(5), table=at(4), cols=10, stride=10, page=16, T=40, cu=at(6),
             kv=at(7), pos=at(8), slots=at(9), parents=at(10), masks=at(11), words=2):
        return lib.paged_reserve(p, new, lens, table, cols, stride, page, T, cu, kv, pos, slots, parents,
                                 masks, words, S)

    assert call(p=None) == INVALID
    for kw, code in BAD_POOLS:
        assert call(p=pool(**kw)) == code, kw
    for kw in (dict(new=NULL), dict(lens=NULL), dict(table=NULL), dict(cu=NULL), dict(kv=NULL),
               dict(cols=0), dict(stride=9), dict(page=0), dict(T=-1), dict(words=-1), dict(words=0),
               dict(masks=NULL), dict(kv=at(3)), dict(cu=at(5)), dict(pos=at(10)),
               dict(slots=at(11)), dict(masks=at(4)), dict(kv=off(5, 4)), dict(pos=at(9))):
        assert call(**kw) == INVALID, kw
    assert call(T=2 ** 31 - 1, slots=NULL, pos=NULL, parents=NULL, masks=NULL, words=0) == UNSUPPORTED
    for kw in (dict(new=off(3, 1)), dict(slots=off(9, 4)), dict(masks=off(11, 2)), dict(cu=off(6, 3))):
        assert call(**kw) == MISALIGNED, kw


def test_release_refusals(lib):
    def call(p=pool(), lens=at(5), table=at(4), cols=10, stride=10, page=16):
        return lib.paged_release(p, lens, table, cols, stride, page, S)

    for kw, code in BAD_POOLS:
        assert call(p=pool(**kw)) == code, kw
    for kw in (dict(lens=NULL), dict(table=NULL), dict(cols=0), dict(stride=3), dict(page=-1),
               dict(lens=at(1)), dict(table=at(0)), dict(lens=at(4))):
        assert call(**kw) == INVALID, kw
    assert call(lens=off(5, 2)) == MISALIGNED


def test_keep_refusals(lib):
    def call(d=paged(), kept=at(9), width=4, stride=0, layers=1, step=0, kp=at(0), vp=at(1), lens=at(2)):
        return lib.paged_kv_keep(d, kept, width, stride, layers, step, kp, vp, lens, S)

    assert call(d=None) == INVALID
    for kw, code in COMMON:
        if "T" not in kw:
            assert call(d=paged(**kw)) == code, kw
    for kw in (dict(kept=NULL), dict(kp=NULL), dict(vp=NULL), dict(lens=NULL), dict(width=0),
               dict(layers=0), dict(stride=3), dict(vp=at(0)), dict(kp=at(9)), dict(lens=at(9)),
               dict(lens=at(1))):
        assert call(**kw) == INVALID, kw
    # layers on one another, or within a page's stride but no room there
    assert call(layers=2, step=0) == INVALID and call(layers=2, step=64) == INVALID
    assert call(layers=2, step=-8) == INVALID and call(layers=3, step=(1 << 20) + 4) == MISALIGNED
    assert call(kept=off(9, 2)) == MISALIGNED and call(lens=off(2, 1)) == MISALIGNED
    assert call(kp=off(0, 8)) == MISALIGNED
    assert call(lens=ctypes.c_void_p(1 << 20)) in (INVALID, MISALIGNED)
    assert call(d=paged(D=60, token_stride=120, head_stride=60)) != OK


def test_python_refusals():
    """What the binding refuses before it calls the library, without a GPU."""
    with pytest.raises(ValueError):
        cea.page_pool(0, 4, device="cpu")
    with pytest.raises(ValueError):
        cea.qk_norm_rope_fwd(None, None)
    x = torch.zeros(1, 2, 1, 8)
    with pytest.raises(ValueError):
        cea.qk_norm_rope_fwd(x, None)
    with pytest.raises(ValueError):
        cea.qk_norm_rope_bwd(x, None, None, None, x, None)
    p = cea.page_pool(4, 2, device="cpu")
    assert p.free.tolist() == [3, 2, 1, 0] and int(p.count) == 4 and p.held.tolist() == [0, 0]
    step = cea.paged_step(2, 5, mask_words=3, device="cpu")
    assert step.masks.shape == (5, 3) and step.slots.dtype == torch.int64
    cu, lens, positions, slots, masks = step
    assert step._replace(slots=None).slots is None and step._replace(slots=None).masks is masks
    for kw in (dict(positions=None, slots=None, masks=None), dict(cu_new=lens), dict(slots=positions),
               dict(positions=positions[:3]), dict(masks=masks[:, :2]), dict(kv_lens=lens.long())):
        with pytest.raises(ValueError):
            step._replace(**kw)
    with pytest.raises(AttributeError):
        step.masks = masks
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cea.paged_reserve(p, i, i, i[None], 16, step)
    with pytest.raises(ValueError):
        cea.paged_release(p, i, i[None], 16)


def test_the_model_of_the_pool():
    """The plain form that the GPU tests compare with: a release undoes a reserve; depths, masks."""
    m = PoolModel(9, 3, 4, 4)
    first = m.reserve([5, 0, 9], [0, 0, 0], 20)
    assert first[0] == [0, 5, 5, 14] and first[3][:5] == [0, 1, 2, 3, 4] and m.held == [2, 0, 3]
    free, table = list(m.free), [list(r) for r in m.table]
    step = m.reserve([4, 3, 4], [5, 0, 9], 20, parents=[-1, 0, 0, 2] + [-1, -1, 5] + [-1, 0, 1, 2])
    assert step[4] == 0 and step[2][:7] == [5, 6, 6, 7, 0, 0, 0] and m.held == [3, 1, 4]
    m.release([5, 0, 9])
    assert m.free == free and m.table == table
    assert m.reserve([30, 0, 0], [5, 0, 9], 20)[4] == 2 and m.reserve([12, 0, 0], [5, 0, 9], 20)[4] == 3
    assert m.reserve([8, 8, 0], [5, 0, 9], 20)[4] == 0 and m.reserve([0, 8, 0], [13, 8, 9], 20)[4] == 1
    seen, depth = ancestors([-1, 0, 0, 2])
    assert depth == [0, 1, 1, 2] and seen[3].tolist() == [True, False, True, True]
    assert mask_words(seen, 1)[:, 0].tolist() == [1, 3, 5, 13]
