"""Plain 64-bit forms for the tests of a step of drafted tokens: page bookkeeping, normalised
heads, trees' attention.

Error bounds (u = 2^-24; the rotation's and the attention's are paged_helpers'):

norm: a head's squares are summed 16 to a lane one after the other and over at most 32 lanes
  by halving, 16 + 5 roundings and one for the product with 1/D, which is itself rounded; eps
  adds one more: the mean is off by 24u, its reciprocal root by half of that and 2 units in the
  last place (2^-22 = 4u): 16u.  The products with x and with the weight (and the sum with the
  weight's offset) add 3u: an element of w x r is off by 20u < 2^-19 of itself.  Rotating it
  adds 2^-20 (|v_a| + |v_b|) A and passes its own error on, 2^-19 (|v_a| + |v_b|) A.

its gradients: z = R^T dy is off by ez = 2^-20 A (|dy_a| + |dy_b|) (0 behind rot); g = w z by
  |w| ez + 2u |g|; u_i = x r by 17u |u_i|.  The dot product sum g x of D terms has 24 roundings
  of at most S = sum |g x|, and the errors of g: |w| ez |x| summed.  c = r dot / D is off by
  r / D sum |w| ez |x| + (24 + 16 + 5) u C, C = r S / D.  dx = r (g - u_i c) is off by
  r (|w| ez + 2u |g| + |u_i| err_c + 18u |u_i| C + u (|g| + |u_i| C)) + 20u r (|g| + |u_i| C),
  then the rounding to its type.  dw sums n terms z u_i, each off by |u_i| ez + 19u |z u_i|, with at
  most n roundings of at most the sum of |z u_i|.
"""
import math

import torch

from paged_helpers import U, half_step


def angles64(pos, freq):
    return pos.double()[..., None] * freq.double()


def turn64(x, angle, style, amplitude, sign=1.0):
    """x [..., H, D] fp64 rotated by angle [..., rot/2]; and the |x_a| + |x_b| of the pairs."""
    y, mag = x.clone(), torch.zeros_like(x)
    h = angle.shape[-1]
    if h == 0:
        return y, mag
    i = torch.arange(h)
    ia, ib = (i, i + h) if style == "half" else (2 * i, 2 * i + 1)
    c = torch.cos(angle)[..., None, :] * amplitude
    s = torch.sin(angle)[..., None, :] * amplitude * sign
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * abs(amplitude)
    return y, mag


def norm64(x, w, angle, style, amplitude=1.0, eps=1e-6):
    """(R(w x r), bound without the last rounding) of x [..., H, D], w [D] fp64 (with its offset)."""
    x = x.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    v = w * x * r
    y, mag = turn64(v, angle, style, amplitude)
    passed = mag == 0
    return y, torch.where(passed, 2.0 ** -19 * v.abs(), 3 * 2.0 ** -20 * mag)


def norm_bwd64(x, w, dy, angle, style, amplitude=1.0, eps=1e-6):
    """(dx, bound without the last rounding, dw, bound) in fp64; rows are all but the last dim."""
    x, dy = x.double(), dy.double()
    D = x.shape[-1]
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    z, mag = turn64(dy, angle, style, amplitude, sign=-1.0)
    ez = 2.0 ** -20 * mag
    g, un = w * z, x * r
    c = (g * un).mean(-1, keepdim=True)
    C = (g * un).abs().mean(-1, keepdim=True)
    dx = r * (g - un * c)
    err_c = (w.abs() * ez * un.abs()).mean(-1, keepdim=True) + 45 * U * C
    both = g.abs() + un.abs() * C
    tol = r * (w.abs() * ez + 2 * U * g.abs() + un.abs() * (err_c + 18 * U * C) + 21 * U * both)
    dw = (z * un).flatten(0, -2).sum(0)
    n = x.numel() // D
    size = (z * un).abs().flatten(0, -2).sum(0)
    tol_w = (un.abs() * ez).flatten(0, -2).sum(0) + (19 + n) * U * size + 1e-30
    return dx, tol, dw, tol_w


def assert_within(got, ref, tol, what=""):
    """|got - ref| within tol and one rounding to got's type."""
    err = (got.double().cpu() - ref).abs()
    bound = tol + half_step(got.dtype) * (ref.abs() + tol) + 1e-30
    assert not got.isnan().any(), f"{what}: NaN"
    bad = err > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {(err / bound).max():.2f} bounds"


def tree_reference(c, seen):
    """Cache.reference for a tree: seen[i] is a bool [n, n] of which new tokens see which.  New
    token j of n stands at key kv - n + j."""
    H, D, G = c.H, c.D, c.H // c.H_kv
    out = torch.full((c.T, H, D), math.nan, dtype=torch.float64)
    lse = torch.full((c.T, H), math.nan, dtype=torch.float64)
    tol, tol_lse = out.clone(), lse.clone()
    q = c.q.double()
    for i, (n, kv) in enumerate(c.seqs):
        r0 = int(c.cu[i])
        k, v = c.keys(i, c.k), c.keys(i, c.v)
        hidden = torch.zeros(n, kv, dtype=torch.bool)
        for j in range(n):
            if kv - n + j >= 0:
                hidden[:, kv - n + j] = ~seen[i][:, j]
        for h in range(H):
            qh, kh, vh = q[r0:r0 + n, h], k[:, h // G], v[:, h // G]
            # a key or value that no row sees may be anything
            unseen = hidden.all(0)
            kh, vh = kh.masked_fill(unseen[:, None], 0.0), vh.masked_fill(unseen[:, None], 0.0)
            s = (qh @ kh.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            S = (qh.abs() @ kh.T.abs() / math.sqrt(D)).masked_fill(hidden, 0.0)
            top = s.amax(-1, keepdim=True) if kv else torch.full((n, 1), -math.inf, dtype=torch.float64)
            p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
            total = p.sum(-1, keepdim=True)
            w = torch.where(total > 0, p / total, 0.0)
            o, Av = w @ vh, w @ vh.abs()
            Smax = S.amax(-1) if kv else torch.zeros(n, dtype=torch.float64)
            e = (D + 8) * U * Smax + 2.0 ** -21 + (kv / 16 + 64) * U
            low = 2.0 ** -8 if c.dtype == torch.bfloat16 else kv * U
            out[r0:r0 + n, h], lse[r0:r0 + n, h] = o, (top + torch.log(total))[:, 0]
            tol[r0:r0 + n, h] = ((2 * e + low * (1 + 2.0 ** -7))[:, None] * Av
                                 + half_step(c.dtype) * (o.abs() + (2 * e + low)[:, None] * Av) + 1e-30)
            tol_lse[r0:r0 + n, h] = e + 4 * U * (lse[r0:r0 + n, h].abs() + Smax + 1)
    return out, lse, tol, tol_lse


def random_parents(n, g, wide=False):
    """Parents of n drafted tokens: mostly recent ones, or with `wide` any earlier one; some roots."""
    out = []
    for i in range(n):
        lo = 0 if wide else max(0, i - 4)
        p = int(torch.randint(lo, i + 1, (1,), generator=g)) - 1 if i else -1
        out.append(p if p >= 0 or i == 0 or torch.rand(1, generator=g) < 0.1 else i - 1)
    return out


def ancestors(parents):
    """(bool [n, n] of which tokens a token follows or is, depths)."""
    n = len(parents)
    seen, depth = torch.zeros(n, n, dtype=torch.bool), [0] * n
    for i, p in enumerate(parents):
        if 0 <= p < i:
            seen[i] = seen[p]
            depth[i] = depth[p] + 1
        seen[i, i] = True
    return seen, depth


def mask_words(seen, words):
    """int32 [n, words] bits of a bool [n, n]; tokens beyond 32 words are left out."""
    n = seen.shape[0]
    out = torch.zeros(n, words, dtype=torch.int64)
    for j in range(min(seen.shape[1], 32 * words)):
        out[:, j // 32] |= seen[:, j].long() << (j % 32)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


class PoolModel:
    """paged_reserve and paged_release in plain Python."""

    def __init__(self, num_pages, n_seqs, max_pages, page):
        self.free, self.table = list(range(num_pages - 1, -1, -1)), [[-1] * max_pages for _ in range(n_seqs)]
        self.held, self.page, self.max_pages = [0] * n_seqs, page, max_pages

    def reserve(self, new, lens, T, parents=None):
        new, lens = [max(x, 0) for x in new], [max(x, 0) for x in lens]
        need = [max(0, -(-(a + b) // self.page) - h) for a, b, h in zip(new, lens, self.held)]
        status = 0
        if sum(need) > len(self.free):
            status = 1
        if any(a + b > min(self.max_pages * self.page, 2 ** 31 - 1) for a, b in zip(new, lens)):
            status = 3
        if sum(new) > T:
            status = 2
        if status:
            new, need = [0] * len(new), [0] * len(new)
        cu, positions, slots, rows = [0], [], [], []
        for g, (a, b) in enumerate(zip(new, lens)):
            for _ in range(need[g]):
                self.table[g][self.held[g]] = self.free.pop()
                self.held[g] += 1
            depth = [0] * a
            for i in range(a):
                p = parents[cu[-1] + i] if parents is not None else i - 1
                if 0 <= p < i:
                    depth[i] = depth[p] + 1
                positions.append(b + depth[i])
                slots.append(self.table[g][(b + i) // self.page] * self.page + (b + i) % self.page)
            rows.append(a)
            cu.append(cu[-1] + a)
        pad = T - cu[-1]
        return (cu, [a + b for a, b in zip(new, lens)], positions + [0] * pad, slots + [-1] * pad, status)

    def release(self, lens):
        back = []
        for g, n in enumerate(lens):
            left = min(-(-max(n, 0) // self.page), self.held[g])
            back += self.table[g][left:self.held[g]]
            for j in range(left, self.held[g]):
                self.table[g][j] = -1
            self.held[g] = left
        self.free += back[::-1]
