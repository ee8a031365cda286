"""paged_attn_fwd with values that are not finite, with values whose weighted sum nearly
cancels, which shows what the weights were rounded to, and with huge scores (bounds:
paged_helpers)."""
import math

import pytest
import torch

import context_exact_attention_gb300 as cea
from paged_helpers import Cache, U, assert_attends, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def attend(c, causal=True):
    kp, vp = c.device_pages(DEV)
    r = cea.paged_attn_fwd(c.q.to(DEV), kp, vp, c.table.to(DEV), c.cu.to(DEV), c.kv_lens.to(DEV),
                           causal=causal)
    assert cea.check_status() == 0
    return r


# sequences (new tokens, keys), H, H_kv, D, page, dtype
SEEN = {
    "one key": ([(1, 1)], 4, 1, 128, 16, BF),
    "single tokens": ([(1, 5), (1, 64), (1, 70), (1, 1000)], 8, 2, 128, 16, BF),
    "single tokens, D 64": ([(1, 2), (1, 129), (1, 500)], 4, 4, 64, 8, BF),
    "a long context": ([(1, 20000)], 4, 1, 128, 64, BF),
    "few tokens": ([(3, 90), (2, 2), (4, 700)], 6, 2, 64, 32, BF),
    "a chunk on odd pages": ([(70, 200)], 4, 2, 128, 3, BF),
    "chunks": ([(300, 1000), (40, 44)], 4, 2, 128, 64, BF),
    "chunks, D 64": ([(140, 900), (33, 33)], 4, 1, 64, 16, BF),
    "a chunk, a long context": ([(40, 12000)], 4, 2, 128, 128, BF),
    "fp32": ([(1, 90), (7, 40), (1, 3000)], 6, 2, 128, 16, F32),
    "fp32 prompts": ([(170, 333), (200, 400)], 4, 2, 64, 16, F32),
}


@pytest.mark.parametrize("name", SEEN)
def test_infinite_values_that_every_row_sees(name):
    """A key before the new tokens has an infinite value in one column and minus infinity in
    another: positive weights make the sums of those columns the same infinities, and the
    other columns stay what they are."""
    seqs, H, H_kv, D, page, dtype = SEEN[name]
    ref = Cache(seqs, H, H_kv, D, page, dtype, seed=len(name)).reference()
    for part in (0.0, 0.37, 1.0):                  # first, some, and the first new token's key
        c = Cache(seqs, H, H_kv, D, page, dtype, seed=len(name))
        for i, (n, kv) in enumerate(seqs):
            at = int(part * (kv - n))
            c.v[c.table[i, at // page], at % page, :, 3] = math.inf
            c.v[c.table[i, at // page], at % page, :, 5] = -math.inf
        out, lse = attend(c)
        assert (out[..., 3] == math.inf).all(), f"{part}: {out[..., 3].isnan().sum()} NaN"
        assert (out[..., 5] == -math.inf).all(), part
        rest = [x for x in range(D) if x not in (3, 5)]
        assert_attends(out[..., rest], lse, (ref[0][..., rest], ref[1], ref[2][..., rest], ref[3]), name)


@pytest.mark.parametrize("name", SEEN)
def test_rows_whose_scores_are_all_minus_infinity(name):
    """Such a row is as one that sees no key; the other heads and sequences are as ever."""
    seqs, H, H_kv, D, page, dtype = SEEN[name]
    c = Cache(seqs, H, H_kv, D, page, dtype, seed=len(name))
    c.q[:, 0, 0] = 1.0
    ref = c.reference()
    for pg in c.table[0, :-(-seqs[0][1] // page)]:
        c.k[pg, :, 0, 0] = -math.inf               # the first sequence's keys for the first head
    out, lse = attend(c)
    n, G = seqs[0][0], H // H_kv
    assert (out[:n, 0] == 0).all() and (lse[:n, 0] == -math.inf).all()
    if G < H:
        assert_attends(out[:, G:], lse[:, G:], tuple(x[:, G:] for x in ref), name)
    if len(seqs) > 1:
        assert_attends(out[n:], lse[n:], tuple(x[n:] for x in ref), name)


# (new tokens, keys) of every sequence, H, H_kv, D, page: calls of the kernel for few rows
TWO_PARTS = {
    "one token": ([(1, 2)], 32, 4, 128, 16),
    "single tokens, D 64": ([(1, 70), (1, 500)] * 4, 16, 2, 64, 16),
    "a long context": ([(1, 20000)], 16, 1, 128, 64),
    "proposed tokens": ([(4, 300), (2, 30)] * 4, 16, 4, 64, 8),
    "a chunk on odd pages": ([(70, 200)], 4, 2, 128, 3),
}


@pytest.mark.parametrize("name", TWO_PARTS)
def test_weights_of_few_rows_go_in_as_two_parts(name):
    """Half of the keys score 0 and have the values c, 1/2 to 1 over the columns; the others
    score below 0, all the same in a row, and have the values -1.  Where c is near the weight w
    of those, the output nearly cancels, and neither its own rounding nor the average hides how
    w was rounded.  The bound: w is off by 2^-16 (two bf16 parts: the first cut off, the rest,
    up to 2^-7 of a power of two, rounded to half a step, 2^-16 of that) and by e = (D + 8) u
    |score| + 2^-21 (see paged_helpers), which the numerator feels as that times A = (sum of w
    |v|) / sum of w.  The denominator's error is one of the quotient: e + (n / 16 + 64) u +
    2^-20.  A matrix product of 16 keys is off by 17 2^-23 of the larger of its sum so far and
    its terms; keys alternate, so sums grow as the result does: n / 32 products, 17 n / 32 2^-23
    of |out| and (their terms, which are 1) 2^-21 A.  One part would be off by 2^-9 at weights
    of 1/2 to 1."""
    seqs, H, H_kv, D, page = TWO_PARTS[name]
    c = Cache(seqs, H, H_kv, D, page, BF, seed=len(name), garbage=0.0)
    columns = (0.5 + torch.arange(D) / (2 * D)).to(BF)
    c.q.zero_()
    # scores of 0 down to -0.7: weights of 1 down to 1/2
    c.q[..., 0] = torch.rand(c.T, H, generator=torch.Generator().manual_seed(1)).mul(0.7).to(BF)
    low = torch.tensor(-math.sqrt(D)).to(BF)
    for i, (n, kv) in enumerate(seqs):
        for j in range(kv):
            at = int(c.table[i, j // page]), j % page
            c.k[at], c.v[at] = 0, columns
            if j % 2:
                c.k[at][:, 0], c.v[at] = low, -1
    out, _ = attend(c, causal=False)
    got = out.double().cpu()

    worst, one_part = 0.0, 0.0
    for i, (n, kv) in enumerate(seqs):
        rows = slice(int(c.cu[i]), int(c.cu[i]) + n)
        score = c.q[rows, :, 0].double() * float(low) / math.sqrt(D)
        w = torch.exp(score)[..., None]
        a, b = (kv + 1) // 2, kv // 2              # keys that score 0, and below
        total = a + b * w
        ref, A = (a * columns.double() - b * w) / total, (a * columns.double() + b * w) / total
        e = (D + 8) * U * score.abs()[..., None] + 2.0 ** -21
        tol = ((2.0 ** -16 + e + 2.0 ** -21) * A
               + (e + (kv / 16 + 64) * U + 2.0 ** -20 + 17 * kv / 32 * 2.0 ** -23) * ref.abs())
        tol = tol + half_step(BF) * (ref.abs() + tol)
        worst = max(worst, float(((got[rows] - ref).abs() / tol).max()))
        # the same with weights of one part: the bound has to tell them apart
        planted = (a * columns.double() - b * w.to(BF).double()) / total
        one_part = max(one_part, float(((planted - ref).abs() / tol).max()))
    assert one_part > 4, one_part
    assert worst <= 1, f"{worst:.2f} bounds off"


# sequences (new tokens, keys), H, H_kv, D, page, dtype
HUGE = {
    "single tokens": ([(1, 5), (1, 64), (1, 70), (1, 1000)], 8, 2, 128, 16, BF),
    "single tokens, D 64": ([(1, 9), (1, 129), (1, 500)], 4, 4, 64, 8, BF),
    "a long context": ([(1, 20000)], 4, 1, 128, 64, BF),
    "chunks": ([(300, 1000), (40, 44)], 4, 2, 128, 64, BF),
    "chunks, D 64": ([(140, 900), (33, 53)], 4, 1, 64, 16, BF),
    "a chunk, a long context": ([(40, 12000)], 4, 2, 128, 128, BF),
    "fp32": ([(1, 90), (7, 40), (1, 3000)], 6, 2, 128, 16, F32),
    "fp32 prompts": ([(170, 333), (200, 400)], 4, 2, 64, 16, F32),
}


@pytest.mark.parametrize("top", [26, 31, 32, 33, 38, 60, 120])
@pytest.mark.parametrize("name", HUGE)
def test_huge_scores_pick_their_keys(name, top):
    """Scores up to 2^top / sqrt(D) of either sign, so far apart that a row's result is the value
    of its largest key, which every row sees: that key's weight is 1, however the maximum was
    rounded.  (Products of one column, exact in fp32; the value's rounding as a weight of one
    bf16 part and to the output, half a step each; lse a few roundings of fp32.)"""
    seqs, H, H_kv, D, page, dtype = HUGE[name]
    c = Cache(seqs, H, H_kv, D, page, dtype, seed=len(name))
    g = torch.Generator().manual_seed(2)
    a, b = 2.0 ** (top // 2), 2.0 ** (top - top // 2)
    c.q.zero_()
    c.q[..., 0] = (torch.randint(65, 128, c.q.shape[:2], generator=g) * (a / 128)).to(dtype)
    c.q[:, ::2] *= -1
    for i, (n, kv) in enumerate(seqs):
        for j in range(kv):
            at = int(c.table[i, j // page]), j % page
            # the first for the positive queries, the second for the negative ones
            x = {int(0.4 * (kv - n)): 1.0, int(0.8 * (kv - n)): 0.25}.get(j, 0.5)
            c.k[at] = 0
            c.k[at][:, 0] = x * b
    r_out, r_lse, _, _ = c.reference()
    out, lse = attend(c)
    err = (out.double().cpu() - r_out).abs() / r_out.abs()
    assert err.max() <= 2.02 * half_step(dtype), f"{err.max()} of the value"
    err = (lse.double().cpu() / r_lse - 1).abs()
    assert err.max() <= 4 * U, err.max()
