"""paged_attn_fwd with infinite values that the rows see (bounds: paged_helpers)."""
import math

import pytest
import torch

import context_exact_attention_gb300 as cea
from paged_helpers import Cache, assert_attends

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
