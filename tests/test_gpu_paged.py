"""The paged cache on the GPU: paged_kv_append and paged_attn_fwd against 64-bit arithmetic
(bounds: paged_helpers), at the lengths, head counts, page sizes, strides and lengths' faults
where they can go wrong, and run together as a program does."""
import pytest
import torch

import context_exact_attention_gb300 as cea
from paged_helpers import Cache, assert_attends, assert_rotated, rotate64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def attend(c, causal=True, q=None, **kw):
    kp, vp = c.device_pages(DEV)
    q = (c.q if q is None else q).to(DEV)
    r = cea.paged_attn_fwd(q, kp, vp, c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV),
                           causal=causal, **kw)
    assert cea.check_status() == 0
    return r


# sequences (new tokens, keys), H, H_kv, D, page, dtype, layout, padding rows
ATTEND = {
    "one key": ([(1, 1)], 1, 1, 128, 16, BF, "slots", 0),
    "one key fp32": ([(1, 1)], 1, 1, 4, 1, F32, "slots", 0),
    "single tokens": ([(1, 1), (1, 63), (1, 64), (1, 65), (1, 1000)], 8, 2, 128, 16, BF, "slots", 0),
    "single tokens, D 64": ([(1, 17), (1, 128), (1, 129), (1, 500)], 8, 8, 64, 32, BF, "heads", 3),
    "many heads a group": ([(1, 300), (1, 31)], 32, 1, 128, 8, BF, "by_slot", 0),
    "twenty heads a group": ([(3, 200)], 40, 2, 64, 24, BF, "by_page", 0),
    "odd group": ([(2, 77), (1, 5)], 15, 5, 128, 3, BF, "slots", 1),
    "pages of one slot": ([(1, 50), (4, 33)], 6, 2, 64, 1, BF, "by_head", 0),
    "no new tokens between": ([(0, 40), (1, 90), (0, 0), (5, 5), (0, 7)], 4, 2, 128, 16, BF, "slots", 2),
    "more new than keys": ([(6, 2), (3, 0), (1, 9)], 4, 1, 64, 16, BF, "slots", 0),
    "proposed tokens": ([(5, 333), (5, 64), (5, 5)], 16, 2, 128, 32, BF, "slots", 0),
    "a long context": ([(1, 20000)], 4, 1, 128, 64, BF, "slots", 0),
    "a chunk": ([(300, 1000)], 4, 2, 128, 128, BF, "slots", 0),
    "a whole prompt": ([(257, 257)], 2, 1, 64, 16, BF, "heads", 0),
    "chunks and tokens": ([(130, 130), (1, 700), (65, 300), (1, 1), (2, 256)], 6, 2, 128, 16, BF, "slots", 4),
    "a group of seven, chunks": ([(90, 400), (33, 33)], 14, 2, 128, 64, BF, "heads", 0),
    "big pages": ([(150, 600), (1, 513)], 4, 4, 64, 256, BF, "slots", 0),
    "pages of 24": ([(150, 600), (1, 513)], 4, 2, 128, 24, BF, "slots", 0),
    "pages of 8": ([(140, 140), (40, 777)], 4, 2, 128, 8, BF, "by_page", 0),
    "a hundred heads a group": ([(2, 150), (5, 40)], 100, 1, 64, 16, BF, "slots", 1),
    "chunks, more new than keys": ([(200, 50), (130, 0), (40, 300)], 4, 1, 64, 16, BF, "slots", 2),
    "pages of 384": ([(90, 900), (140, 385)], 4, 2, 128, 384, BF, "slots", 0),
    "chunks by head": ([(70, 300), (33, 40)], 4, 2, 128, 16, BF, "by_head", 0),
    "chunks by slot": ([(70, 300), (33, 40)], 4, 2, 64, 32, BF, "by_slot", 0),
    "a chunk, a long context": ([(40, 12000)], 4, 2, 128, 128, BF, "heads", 0),
    "many short prompts": ([((i * 7) % 60, (i * 7) % 60 + i % 5) for i in range(150)], 8, 2, 64, 8, BF,
                           "slots", 5),
    "more heads than a tile": ([(2, 150), (40, 90)], 160, 1, 64, 16, BF, "slots", 0),
    "fp32": ([(1, 90), (7, 40), (1, 1), (0, 3)], 6, 2, 128, 16, F32, "slots", 1),
    "fp32 wide": ([(2, 130), (1, 3)], 5, 1, 256, 8, F32, "heads", 0),
    "fp32 narrow": ([(3, 70), (2, 1)], 4, 4, 20, 5, F32, "by_slot", 0),
    "fp32 long": ([(1, 9000), (30, 500)], 2, 1, 64, 64, F32, "slots", 0),
    # many rows
    "fp32 prompts": ([(170, 170), (200, 333), (1, 5), (0, 40), (131, 131)], 4, 2, 128, 16, F32, "slots", 3),
    "fp32 chunk": ([(401, 900)], 1, 1, 100, 24, F32, "heads", 0),
    "fp32 chunk, a long context": ([(200, 7000)], 4, 2, 64, 64, F32, "by_page", 0),
    "fp32 prompts wide": ([(130, 200), (260, 260)], 3, 1, 256, 8, F32, "by_slot", 1),
    "fp32 prompts 192": ([(399, 391), (90, 0)], 4, 1, 192, 16, F32, "slots", 0),
    "fp32 prompts narrow": ([(500, 63), (400, 465)], 2, 1, 4, 1, F32, "slots", 2),
    "fp32 group of sixty-four": ([(9, 40), (20, 20)], 64, 1, 36, 16, F32, "by_head", 0),
    "fp32 group of nine": ([(90, 200), (64, 64)], 18, 2, 68, 3, F32, "slots", 0),
    "fp32 group of sixty-four, more keys": ([(9, 400), (20, 20)], 64, 1, 36, 16, F32, "by_head", 0),
    "fp32 group of nine, more keys": ([(90, 500), (64, 64)], 18, 2, 68, 3, F32, "slots", 1),
    "fp32 prompts of few keys": ([(100, 100), (64, 70), (90, 3)], 40, 8, 20, 16, F32, "slots", 0),
}


@pytest.mark.parametrize("name", ATTEND)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
def test_attention(name, causal):
    """Slots and pages that hold no key are NaN throughout, table entries behind a sequence's
    pages -1."""
    seqs, H, H_kv, D, page, dtype, layout, pad = ATTEND[name]
    c = Cache(seqs, H, H_kv, D, page, dtype, layout, pad, seed=len(name))
    out = torch.full((c.T, H, D), 3.0, dtype=dtype, device=DEV)
    lse = torch.full((c.T, H), 5.0, device=DEV)
    ws = cea.paged_attn_workspace(D, dtype, DEV)
    attend(c, causal, out=out, lse=lse, workspace=ws)
    assert_attends(out, lse, c.reference(causal), name)
    if pad:                                        # rows behind the last sequence stay
        assert (out[-pad:] == 3).all() and (lse[-pad:] == 5).all()
    # again, on the workspace as the first call left it, without lse: the same bits
    again, none = attend(c, causal, workspace=ws, want_lse=False)
    n = c.T - pad
    assert none is None and torch.equal(again[:n], out[:n])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_more_sequences_than_threads(dtype):
    seqs = [((i * 5) % 3, (i * 13) % 40 + 2) for i in range(700)]
    c = Cache(seqs, 2, 1, 64, 16, dtype, seed=3)
    out, lse = attend(c)
    assert_attends(out, lse, c.reference())


def test_large_scores():
    """Scores in the hundreds: the running maximum is raised many times."""
    c = Cache([(1, 3000), (20, 800)], 4, 2, 128, 16, seed=4, kv_scale=12.0)
    out, lse = attend(c)
    assert_attends(out, lse, c.reference())


def test_infinite_and_nan_inputs_stay_in_their_rows():
    """A NaN query, an infinite key and a NaN value reach the rows that use them and no
    others; a future key that is not finite never shows."""
    c = Cache([(1, 40), (1, 40), (1, 40), (4, 40)], 2, 1, 64, 16, seed=5)
    c.q[0] = float("nan")
    kp, vp = c.k, c.v
    vp[c.table[1, 1], 3] = float("nan")
    c.k[c.table[3, 2], 7] = float("nan")           # key 39: the last new token's own
    out, lse = attend(c)
    assert out[0].isnan().all() and out[1].isnan().all() and not lse[1].isnan().any()
    assert torch.isfinite(out[2:6]).all() and out[6].isnan().all()
    clean = Cache([(1, 40), (1, 40), (1, 40), (4, 40)], 2, 1, 64, 16, seed=5)
    ref = clean.reference()
    real = slice(2, 6)
    assert_attends(out[real], lse[real], tuple(x[real] for x in ref))


def test_a_key_of_a_later_token_that_is_not_finite():
    """In a chunk: the last tokens' keys are NaN and infinite, earlier rows do not see them."""
    c = Cache([(150, 400)], 4, 2, 128, 16, seed=20)
    clean = c.reference()
    for pos, x in ((398, float("nan")), (399, float("inf"))):
        c.k[c.table[0, pos // 16], pos % 16] = x
    out, lse = attend(c)
    assert out[148:].isnan().all()
    assert_attends(out[:148], lse[:148], tuple(x[:148] for x in clean))


def test_strided_queries():
    c = Cache([(3, 100), (1, 30)], 4, 2, 64, 16, seed=6)
    fused = torch.zeros(c.T, 4 + 4, 64, dtype=BF, device=DEV)
    fused[:, :4] = c.q.to(DEV)
    kp, vp = c.device_pages(DEV)
    out, lse = cea.paged_attn_fwd(fused[:, :4], kp, vp, c.table.to(DEV), c.cu.to(DEV),
                                  c.kv_lens.to(DEV))
    assert_attends(out, lse, c.reference())


def test_shared_pages_and_a_wider_table():
    """Two sequences with a common prefix, the table a view of a wider one."""
    c = Cache([(1, 64), (1, 80)], 4, 2, 128, 16, seed=7)
    c.table[1, :4] = c.table[0, :4]
    wide = torch.full((2, 50), 10 ** 9, dtype=torch.int32)
    wide[:, :c.table.shape[1]] = c.table
    kp, vp = c.device_pages(DEV)
    out, lse = cea.paged_attn_fwd(c.q.to(DEV), kp, vp, wide.to(DEV)[:, :c.table.shape[1]],
                                  c.cu.to(DEV), c.kv_lens.to(DEV))
    assert_attends(out, lse, c.reference())


@pytest.mark.parametrize("dtype,D,n,H", [(BF, 128, 1, 4), (BF, 64, 70, 4), (F32, 32, 3, 4), (F32, 32, 700, 4),
                                           (F32, 32, 700, 32)])
def test_page_indices_outside_the_cache_read_as_zeros(dtype, D, n, H, monkeypatch):
    c = Cache([(n, 200), (1, 90)], H, 2, D, 16, dtype, seed=8)
    for i, (g, j) in enumerate(((0, 0), (0, 5), (1, 2))):
        c.table[g, j] = [-1, c.num_pages, 2 ** 31 - 1][i]
    normal = cea.load_library()
    monkeypatch.setattr(cea, "_lib", cea.load_debug_library(build_if_missing=True))
    out, lse = attend(c)
    assert_attends(out, lse, c.reference())
    monkeypatch.setattr(cea, "_lib", normal)
    out2, lse2 = attend(c)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


BAD_CU = [[0, 50, 3, 60], [-7, 4, 999, 2 ** 31 - 1], [60, 30, 10, 0], [0] * 4]
BAD_KV = [[-5, 100, 30], [2 ** 31 - 1, 1, 33], [-2 ** 31, 0, 10 ** 9], [300, 300, 300]]


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 24), (F32, 8)], ids=["bf16", "bf16-24", "f32"])
@pytest.mark.parametrize("cu", BAD_CU, ids=str)
@pytest.mark.parametrize("kv", BAD_KV, ids=str)
def test_malformed_lengths_stay_in_bounds(dtype, page, cu, kv, monkeypatch):
    c = Cache([(20, 64), (20, 64), (20, 64)], 4, 2, 64, page, dtype, seed=9, garbage=0.0)
    kp, vp = c.device_pages(DEV)
    new = torch.randn(60, 2, 64, device=DEV).to(dtype)
    table = cea.rope_table(64, device=DEV)
    dcu, dkv = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu, kv))
    normal = cea.load_library()
    for lib in (cea.load_debug_library(build_if_missing=True), normal):
        monkeypatch.setattr(cea, "_lib", lib)
        cea.paged_kv_append(new, new, kp, vp, c.table.to(DEV), dcu, dkv, rope=table,
                            q=c.q.to(DEV))
        assert cea.check_status() == 0
        cea.paged_attn_fwd(c.q.to(DEV), kp, vp, c.table.to(DEV), dcu, dkv)
        assert cea.check_status() == 0


@pytest.mark.parametrize("cu", BAD_CU, ids=str)
@pytest.mark.parametrize("kv", BAD_KV, ids=str)
def test_malformed_lengths_of_many_fp32_rows(cu, kv, monkeypatch):
    c = Cache([(400, 464), (400, 64), (400, 500)], 4, 2, 36, 16, F32, seed=9, garbage=0.0)
    kp, vp = c.device_pages(DEV)
    cu = [min(max(20 * x, -2 ** 31), 2 ** 31 - 1) for x in cu]
    dcu, dkv = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu, kv))
    normal = cea.load_library()
    for lib in (cea.load_debug_library(build_if_missing=True), normal):
        monkeypatch.setattr(cea, "_lib", lib)
        cea.paged_attn_fwd(c.q.to(DEV), kp, vp, c.table.to(DEV), dcu, dkv)
        assert cea.check_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_of_later_tokens_stay_out_of_fp32_rows(bad):
    c = Cache([(400, 450)], 4, 1, 64, 16, F32, seed=11)
    want, _ = attend(c)
    c.v[c.table[0, 300 // 16], 300 % 16] = bad            # seen by new tokens 250 and on
    got, _ = attend(c)
    assert torch.equal(got[:250], want[:250])
    assert not got[250:].isfinite().any()


APPEND = {
    "one": ([(1, 1)], 1, 1, 64, 16, BF, "slots", 0, 64, "half"),
    "tokens": ([(1, 5), (1, 16), (1, 17), (1, 300)], 8, 2, 128, 16, BF, "slots", 2, 128, "half"),
    "chunks": ([(30, 100), (0, 9), (65, 65), (1, 64)], 5, 5, 96, 24, BF, "heads", 0, 32, "interleaved"),
    "by page": ([(9, 40), (3, 3)], 4, 2, 80, 8, BF, "by_page", 1, 78, "half"),
    "by slot": ([(9, 40), (3, 3)], 4, 2, 64, 1, BF, "by_slot", 0, 64, "interleaved"),
    "by head": ([(9, 40), (3, 3)], 4, 2, 64, 256, BF, "by_head", 0, 64, "half"),
    "fp32": ([(17, 40), (1, 31)], 3, 1, 100, 16, F32, "slots", 0, 50, "half"),
    "early": ([(6, 2), (3, 0), (1, 9)], 2, 1, 64, 16, BF, "slots", 0, 64, "half"),
    "unrotated": ([(7, 30)], 2, 2, 256, 16, F32, "heads", 0, 0, "half"),
    "interleaved wide": ([(40, 70), (2, 9)], 1, 1, 256, 16, BF, "slots", 1, 254, "interleaved"),
    "interleaved odd": ([(9, 40), (1, 3)], 4, 2, 72, 16, BF, "slots", 0, 62, "interleaved"),
    "half odd wide": ([(9, 40), (1, 3)], 4, 2, 256, 16, BF, "by_page", 0, 250, "half"),
    "half of 8 bytes": ([(9, 40), (1, 3)], 4, 2, 64, 16, BF, "slots", 0, 24, "half"),
}


@pytest.mark.parametrize("name", APPEND)
@pytest.mark.parametrize("fused", [False, True], ids=["apart", "fused"])
def test_append(name, fused):
    """Every slot of the cache: new keys rotated, new values copied, the rest untouched (rows
    at negative positions, which a sequence with fewer keys than new rows has, not stored)."""
    seqs, H, H_kv, D, page, dtype, layout, pad, rot, style = APPEND[name]
    c = Cache(seqs, H, H_kv, D, page, dtype, layout, pad, seed=11, garbage=9.0)
    qkv = torch.randn(c.T, H + 2 * H_kv, D, generator=torch.Generator().manual_seed(12)).to(dtype)
    q, k, v = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
    dev = qkv.to(DEV)
    dq, dk, dv = dev[:, :H], dev[:, H:H + H_kv], dev[:, H + H_kv:]
    if not fused:
        dq, dk, dv = dq.contiguous(), dk.contiguous(), dv.contiguous()
    kp, vp = c.device_pages(DEV)
    table = cea.rope_table(rot, style=style, scaling="yarn", factor=4.0, original_length=64,
                           device=DEV) if rot else None
    q_out = torch.full((c.T, H, D), 2.0, dtype=dtype, device=DEV)
    cea.paged_kv_append(dk, dv, kp, vp, c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV),
                        rope=table, q=dq, q_out=q_out)
    assert cea.check_status() == 0
    if rot:
        two_pi = 2 * torch.pi
        phase = [(int(x) % 2 ** 64) / 2 ** 64 for x in table.phases.tolist()]
        freq = torch.tensor(phase, dtype=torch.float64) * two_pi
    want_k, want_v = c.k.double(), c.v.double()
    mag_k = torch.zeros_like(want_k)
    for i, (n, kv) in enumerate(seqs):
        r0 = int(c.cu[i])
        pos = torch.arange(kv - n, kv)
        rk, mk = k[r0:r0 + n].double(), torch.zeros(n, H_kv, D, dtype=torch.float64)
        rq, mq = q[r0:r0 + n].double(), torch.zeros(n, H, D, dtype=torch.float64)
        if rot:
            angle = pos.double()[:, None] * freq
            rk, mk = rotate64(rk, angle, rot, style, table.amplitude)
            rq, mq = rotate64(rq, angle, rot, style, table.amplitude)
        assert_rotated(q_out[r0:r0 + n], rq, mq, "q")
        for j in range(n):
            p = int(pos[j])
            if p >= 0:
                at = int(c.table[i, p // page]), p % page
                want_k[at], want_v[at], mag_k[at] = rk[j], v[r0 + j].double(), mk[j]
    assert_rotated(kp, want_k, mag_k, "k")
    assert torch.equal(vp.double().cpu(), want_v)
    if pad:
        assert (q_out[-pad:] == 2).all()
    # without q
    kp2, vp2 = c.device_pages(DEV)
    assert cea.paged_kv_append(dk, dv, kp2, vp2, c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV),
                               rope=table) is None
    assert torch.equal(kp2, kp) and torch.equal(vp2, vp)


def test_append_skips_pages_outside_the_cache():
    c = Cache([(40, 40)], 2, 1, 64, 16, seed=13, garbage=9.0)
    c.table[0, 1] = c.num_pages
    kp, vp = c.device_pages(DEV)
    new = torch.ones(40, 1, 64, dtype=BF, device=DEV)
    cea.paged_kv_append(new, new, kp, vp, c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV))
    assert cea.check_status() == 0
    assert int((vp == 1).all(-1).sum()) == 24


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 elements, used at its end."""
    pages, page, H_kv, D = 34000, 128, 8, 128        # 4.46e9 elements
    kp = torch.empty(pages, page, H_kv, D, dtype=BF, device=DEV)
    vp = torch.empty_like(kp)
    c = Cache([(1, 300), (40, 150)], 16, H_kv, D, page, seed=14)
    top = {int(x): pages - 1 - i for i, x in enumerate(c.table.unique()) if x >= 0}
    table = torch.tensor([[top.get(int(x), -1) for x in row] for row in c.table],
                         dtype=torch.int32, device=DEV)
    for old, new in top.items():
        kp[new], vp[new] = c.k[old].to(DEV), c.v[old].to(DEV)
    out, lse = cea.paged_attn_fwd(c.q.to(DEV), kp, vp, table, c.cu.to(DEV), c.kv_lens.to(DEV))
    assert_attends(out, lse, c.reference())
    k = torch.randn(41, H_kv, D, device=DEV).to(BF)
    cea.paged_kv_append(k, k, kp, vp, table, c.cu.to(DEV), c.kv_lens.to(DEV))
    assert cea.check_status() == 0
    assert torch.equal(kp[table[0, 2], 299 - 256], k[0])
    assert torch.equal(vp[table[1, 1], 149 - 128], k[40])


def test_parts_of_a_cache_join_by_their_lse():
    """Attention over two halves of the keys, merged, is attention over all of them."""
    c = Cache([(1, 512)], 8, 2, 128, 16, seed=15)
    whole, lse = attend(c)
    kp, vp = c.device_pages(DEV)
    parts = []
    for lo, hi in ((0, 12), (12, 32)):
        n = torch.tensor([16 * (hi - lo)], dtype=torch.int32, device=DEV)
        parts.append(cea.paged_attn_fwd(c.q.to(DEV), kp, vp, c.table[:, lo:hi].contiguous().to(DEV),
                                        c.cu.to(DEV), n, causal=False))
    (oa, la), (ob, lb) = parts
    joined, ljoined = cea.attn_merge_partials(oa, la, ob, lb)
    r_out, r_lse, tol, tol_lse = c.reference()
    # a partial's rounding to bf16 and the merged one's on top of the direct bound
    extra = 2.0 ** -8 * (oa.double().abs() + ob.double().abs()).cpu() + 2.0 ** -8 * r_out.abs()
    assert ((joined.double().cpu() - r_out).abs() <= tol + extra).all()
    assert ((ljoined.double().cpu() - r_lse).abs() <= 3 * tol_lse).all()


def test_captured_step_follows_the_lengths():
    """Append and attention captured once; the replay decodes the next token when the lengths
    on the device have moved on.  Two graphs share a workspace, replayed in order."""
    c = Cache([(1, 100), (1, 33)], 4, 2, 64, 16, seed=16, garbage=0.0)
    table = torch.arange(2 * 10, dtype=torch.int32, device=DEV).view(2, 10)
    kp = torch.randn(20, 16, 2, 64, device=DEV).to(BF)
    vp = torch.randn_like(kp)
    q, k, v = (torch.randn(2, h, 64, device=DEV).to(BF) for h in (4, 2, 2))
    cu, kv = c.cu.to(DEV), c.kv_lens.to(DEV)
    rope, ws = cea.rope_table(64, device=DEV), cea.paged_attn_workspace(64, BF, DEV)
    qr, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(2, 4, device=DEV)

    def step(o):
        cea.paged_kv_append(k, v, kp, vp, table, cu, kv, rope=rope, q=q, q_out=qr)
        cea.paged_attn_fwd(qr, kp, vp, table, cu, kv, out=o, lse=lse, workspace=ws)

    graphs = []
    outs = [torch.empty_like(q), torch.empty_like(q)]
    step(out)
    torch.cuda.synchronize()
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o)
        graphs.append(g)
    for i in range(5):
        kv.add_(1)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device=DEV).to(BF))
        graphs[i % 2].replay()
        kp2, vp2 = kp.clone(), vp.clone()
        step(out)
        assert torch.equal(out, outs[i % 2]) and torch.equal(kp, kp2) and torch.equal(vp, vp2)
    assert cea.check_status() == 0


def test_two_streams_with_their_own_workspaces():
    c = Cache([(1, 5000), (3, 700)], 8, 2, 128, 16, seed=17)
    want, wl = attend(c)
    kp, vp = c.device_pages(DEV)
    args = (c.q.to(DEV), kp, vp, c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV))
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [cea.paged_attn_workspace(128, BF, DEV) for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            outs[i].append(cea.paged_attn_fwd(*args, workspace=ws[i], stream=s))
    torch.cuda.synchronize()
    for o in outs:
        for out, lse in o:
            assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("G", [1, 4], ids=["mha", "gqa"])
def test_prefill_and_decode_against_dense_ring_attention(G):
    """A sequence prefilled in chunks of odd lengths and decoded token by token, every step
    rope + append + attention over the pages, against rope_fwd and the dense causal
    forward over the whole sequence: both are within their bounds of the same result."""
    H, D, L, page = 4, 128, 384, 32
    H_kv = H // G
    g = torch.Generator().manual_seed(18)
    q, k, v = (torch.randn(L, h, D, generator=g).to(BF).to(DEV) for h in (H, H_kv, H_kv))
    rope = cea.rope_table(D, device=DEV)
    qr, kr = cea.rope_fwd(q[None], k[None], rope)
    dense, dlse = cea.ring_attn_fwd_gqa(qr, kr, v[None].contiguous(), P=1, causal=True)
    pages = L // page
    kp = torch.full((pages, page, H_kv, D), float("nan"), dtype=BF, device=DEV)
    vp = kp.clone()
    table = torch.randperm(pages, generator=g).int().to(DEV)[None]
    ws = cea.paged_attn_workspace(D, BF, DEV)
    outs, lses, at = [], [], 0
    for n in (100, 1, 1, 170, 3, 60, *[1] * 49):
        rows = slice(at, at + n)
        at += n
        cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        kv = torch.tensor([at], dtype=torch.int32, device=DEV)
        x = cea.paged_kv_append(k[rows], v[rows], kp, vp, table, cu, kv, rope=rope, q=q[rows])
        assert torch.equal(x, qr[0, rows])
        o, s = cea.paged_attn_fwd(x, kp, vp, table, cu, kv, workspace=ws)
        outs.append(o)
        lses.append(s)
    assert at == L and cea.check_status() == 0
    c = Cache([(L, L)], H, H_kv, D, page, seed=0)
    for j in range(pages):
        c.k[c.table[0, j]] = kr[0, j * page:(j + 1) * page].cpu()
        c.v[c.table[0, j]] = v[j * page:(j + 1) * page].cpu()
    ref = c.reference(q=qr[0].cpu())
    assert_attends(torch.cat(outs), torch.cat(lses), ref, "paged")
    assert_attends(dense[0], dlse[0], ref, "dense")


def test_debug_build_gives_the_same_bits(monkeypatch):
    cases = ["chunks and tokens", "odd group", "a long context", "fp32", "no new tokens between",
             "fp32 prompts", "fp32 prompts wide", "fp32 group of nine",
             "more heads than a tile", "pages of 24", "twenty heads a group"]
    normal = {}
    for n in cases:
        seqs, H, H_kv, D, page, dtype, layout, pad = ATTEND[n]
        normal[n] = attend(Cache(seqs, H, H_kv, D, page, dtype, layout, pad, seed=1))
    monkeypatch.setattr(cea, "_lib", cea.load_debug_library(build_if_missing=True))
    for n in cases:
        seqs, H, H_kv, D, page, dtype, layout, pad = ATTEND[n]
        out, lse = attend(Cache(seqs, H, H_kv, D, page, dtype, layout, pad, seed=1))
        assert torch.equal(out, normal[n][0]) and torch.equal(lse, normal[n][1])


def test_binding_refusals():
    c = Cache([(2, 40)], 4, 2, 64, 16, seed=19, garbage=0.0)
    kp, vp = c.device_pages(DEV)
    q, t, cu, kv = c.q.to(DEV), c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV)
    k = torch.zeros(2, 2, 64, dtype=BF, device=DEV)
    bad = [
        lambda: cea.paged_attn_fwd(q.float(), kp, vp, t, cu, kv),
        lambda: cea.paged_attn_fwd(q[None], kp, vp, t, cu, kv),
        lambda: cea.paged_attn_fwd(q, kp, vp[:, :8], t, cu, kv),
        lambda: cea.paged_attn_fwd(q, kp, vp, t.long(), cu, kv),
        lambda: cea.paged_attn_fwd(q, kp, vp, t, cu[:1], kv),
        lambda: cea.paged_attn_fwd(q, kp, vp, t.cpu(), cu, kv),
        lambda: cea.paged_attn_fwd(q, kp, vp, t[:0], cu, kv),
        lambda: cea.paged_attn_fwd(q, kp, vp, t, cu, kv, out=q.float()),
        lambda: cea.paged_attn_fwd(q, kp, vp, t, cu, kv, lse=torch.zeros(2, 4, dtype=BF, device=DEV)),
        lambda: cea.paged_kv_append(k[:1], k, kp, vp, t, cu, kv),
        lambda: cea.paged_kv_append(k.float(), k.float(), kp, vp, t, cu, kv),
        lambda: cea.paged_kv_append(k, k, kp, vp, t, cu, kv, q=q[:1]),
        lambda: cea.paged_kv_append(k, k, kp, vp, t, cu, kv, q_out=q),
        lambda: cea.paged_attn_fwd(q[:1].expand(2, 4, 64), kp, vp, t, cu, kv),
        lambda: cea.paged_attn_fwd(q, kp, vp, t, cu, kv, workspace=cea.paged_attn_workspace(
            64, BF, DEV).view(-1, 2)[:, 0]),
        lambda: cea.paged_kv_append(k[:1].expand(2, 2, 64), k, kp, vp, t, cu, kv),
        lambda: cea.paged_kv_append(k, k[:, :1].expand(2, 2, 64), kp, vp, t, cu, kv),
        lambda: cea.paged_attn_workspace(96), lambda: cea.paged_attn_workspace(64, torch.half),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    short = torch.zeros(1024, dtype=torch.uint8, device=DEV)
    same = kp[:1].expand(kp.shape)                 # every page the same memory
    for f in (lambda: cea.paged_attn_fwd(q, kp, vp, t, cu, kv, workspace=short),
              lambda: cea.paged_kv_append(k, k, kp, kp, t, cu, kv),
              lambda: cea.paged_kv_append(k, k, same, same, t, cu, kv)):
        with pytest.raises(cea.RingAttnError):
            f()
    none = torch.zeros(0, 4, 64, dtype=BF, device=DEV)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    assert cea.paged_attn_fwd(none, kp, vp, t, zero, kv)[0].shape == (0, 4, 64)
    assert cea.paged_kv_append(k[:0], k[:0], kp, vp, t, zero, kv) is None
