"""Inputs and plain 64-bit forms for the tests of rotary positions and the paged cache.

The error bounds follow from the operations' roundings (u = 2^-24 for fp32, half a step of
the result's type for the final rounding):

rotation: a cosine or sine comes from an angle known to pi 2^-25 + 2^-29 and a function good
  to two units in the last place, times the amplitude A: less than 4e-7 A off.  Two products
  and a sum in fp32 add 3u (|x_a| + |x_b|) A.  Together less than 2^-20 A (|x_a| + |x_b|).

attention: a score is a sum of D exact (bf16) or rounded (fp32) products, off by at most
  (D + 4) u S, S = sum |q_d k_d| / sqrt(D) of the key; the exponential adds 2^-22 relative
  and the rounding of its argument u |score| (below S u): a weight is off by a relative
  e = (D + 8) u S + 2^-21.  Summing n weights adds at most (n / 16 + 64) u (no thread adds
  more than n / 16 of them in a row).  The quotient is off by twice that times the average
  of |v| under the weights, A_v; in fp32, where a thread may add the weighted values of all n
  keys one after the other (n - 1 roundings, each below u times a partial sum of at most the
  weights' sum times A_v), by n u A_v more.  The kernel for bf16 calls with many rows also
  rounds the weights to bf16, 2^-8 A_v, which is allowed in every bf16 call here; that few rows
  keep them to 2^-16 is shown by values whose sum nearly cancels (test_gpu_paged_values).
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rotate64(x, angle, rot, style, amplitude=1.0):
    """x [..., H, D] fp64 rotated by angle [..., rot/2] fp64, and the bound's |x_a| + |x_b|."""
    y, mag = x.clone(), torch.zeros_like(x)
    h = rot // 2
    ia = torch.arange(h) if style == "half" else 2 * torch.arange(h)
    ib = ia + h if style == "half" else ia + 1
    c, s = torch.cos(angle)[..., None, :] * amplitude, torch.sin(angle)[..., None, :] * amplitude
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * abs(amplitude)
    return y, mag


def assert_rotated(got, ref, mag, what=""):
    err = (got.double().cpu() - ref).abs()
    bound = half_step(got.dtype) * ref.abs() * (1 + 2 ** -7) + 2.0 ** -20 * mag + 1e-30
    bad = err > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {(err / bound).max():.2f} bounds"


class Cache:
    """A cache with its lengths on the CPU: seqs is a list of (new tokens, keys)."""

    def __init__(self, seqs, H, H_kv, D, page, dtype=torch.bfloat16, layout="slots", pad=0, seed=0,
                 spare=2, garbage=float("nan"), kv_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.H, self.H_kv, self.D, self.page, self.dtype = seqs, H, H_kv, D, page, dtype
        held = [max(0, -(-kv // page)) for _, kv in seqs]
        used = sum(held)
        self.num_pages = used + spare
        cols = max(1, max(held))
        perm = torch.randperm(self.num_pages, generator=g)[:used].tolist()
        table = torch.full((len(seqs), cols), -1, dtype=torch.int32)
        for i, n in enumerate(held):
            for j in range(n):
                table[i, j] = perm.pop()
        self.table = table
        starts = [0]
        for n, _ in seqs:
            starts.append(starts[-1] + n)
        self.cu = torch.tensor(starts, dtype=torch.int32)
        self.kv_lens = torch.tensor([kv for _, kv in seqs], dtype=torch.int32)
        self.T = starts[-1] + pad
        shape = (self.num_pages, page, H_kv, D)
        def pages():
            x = torch.full(shape, garbage, dtype=dtype)
            for i, (_, kv) in enumerate(seqs):
                for j in range(held[i]):
                    n = min(page, kv - j * page)
                    x[table[i, j], :n] = (torch.randn(n, H_kv, D, generator=g) * kv_scale).to(dtype)
            return x
        self.k, self.v = pages(), pages()
        self.q = torch.randn(self.T, H, D, generator=g).to(dtype)
        self.layout = layout

    def device_pages(self, device):
        """The pages on the device with the strides of `layout`: slots before heads, heads
        before slots, or keys and values alternating by page, slot or head."""
        k, v = self.k.to(device), self.v.to(device)
        if self.layout == "slots":
            return k, v
        if self.layout == "heads":
            return tuple(x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (k, v))
        dim = {"by_page": 1, "by_slot": 2, "by_head": 3}[self.layout]
        both = torch.stack([k, v], dim=dim)
        return both.select(dim, 0), both.select(dim, 1)

    def keys(self, i, pages):
        """Sequence i's [kv, H_kv, D] in fp64, zeros where the page index names no page."""
        kv = self.seqs[i][1]
        out = torch.zeros(kv, self.H_kv, self.D, dtype=torch.float64)
        for j in range(kv):
            pg = int(self.table[i, j // self.page])
            if 0 <= pg < self.num_pages:
                out[j] = pages[pg, j % self.page].double()
        return out

    def reference(self, causal=True, q=None):
        """(out, lse, bound of out, bound of lse) in fp64; rows of no sequence are NaN."""
        q = (self.q if q is None else q).double()
        H, D, G = self.H, self.D, self.H // self.H_kv
        out = torch.full((self.T, H, D), math.nan, dtype=torch.float64)
        lse = torch.full((self.T, H), math.nan, dtype=torch.float64)
        tol, tol_lse = out.clone(), lse.clone()
        for i, (n, kv) in enumerate(self.seqs):
            r0 = int(self.cu[i])
            k, v = self.keys(i, self.k), self.keys(i, self.v)
            for h in range(H):
                qh = q[r0:r0 + n, h]
                s = qh @ k[:, h // G].T / math.sqrt(D)
                S = (qh.abs() @ k[:, h // G].T.abs()) / math.sqrt(D)
                if causal:
                    hidden = torch.arange(kv)[None] > (kv - n + torch.arange(n))[:, None]
                    s, S = s.masked_fill(hidden, -math.inf), S.masked_fill(hidden, 0.0)
                top = s.amax(-1, keepdim=True) if kv else torch.full((n, 1), -math.inf)
                p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
                total = p.sum(-1, keepdim=True)
                w = torch.where(total > 0, p / total, 0.0)
                out[r0:r0 + n, h] = w @ v[:, h // G]
                lse[r0:r0 + n, h] = (top + torch.log(total))[:, 0]
                Av = w @ v[:, h // G].abs()
                Smax = S.amax(-1) if kv else torch.zeros(n, dtype=torch.float64)
                e = (D + 8) * U * Smax + 2.0 ** -21 + (kv / 16 + 64) * U
                low = 2.0 ** -8 if self.dtype == torch.bfloat16 else kv * U
                o = out[r0:r0 + n, h]
                tol[r0:r0 + n, h] = ((2 * e + low * (1 + 2.0 ** -7))[:, None] * Av
                                     + half_step(self.dtype) * (o.abs() + (2 * e + low)[:, None] * Av)
                                     + 1e-30)
                # the logarithm of the sum: its relative error, and fp32's on the result
                tol_lse[r0:r0 + n, h] = e + 4 * U * (lse[r0:r0 + n, h].abs() + Smax + 1)
        return out, lse, tol, tol_lse


def assert_attends(out, lse, ref, what=""):
    r_out, r_lse, tol, tol_lse = ref
    real = ~r_lse.isnan()
    got, got_lse = out.double().cpu()[real], lse.double().cpu()[real]
    empty = r_lse[real] == -math.inf
    assert (got_lse[empty] == -math.inf).all() and (got[empty] == 0).all(), f"{what}: empty rows"
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    err = (got - r_out[real]).abs() / tol[real]
    assert err.numel() == 0 or err.max() <= 1, f"{what}: out {err.max():.2f} bounds off"
    some = ~empty
    err = (got_lse[some] - r_lse[real][some]).abs() / tol_lse[real][some]
    assert err.numel() == 0 or err.max() <= 1, f"{what}: lse {err.max():.2f} bounds off"
