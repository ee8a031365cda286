"""rope_fwd and rope_bwd on the GPU against 64-bit arithmetic (bounds: paged_helpers)."""
import ctypes
import math

import pytest
import torch

import context_exact_attention_gb300 as cea
from paged_helpers import assert_rotated, half_step, rotate64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def freqs(rot, base=1e4):
    return base ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)


def positions_of(layout, B, L, P, cu):
    if layout == "zigzag":
        pos = torch.tensor(cea.zigzag_positions(L, P))
    elif layout == "packed":
        pos = torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])])
    else:
        pos = torch.arange(L)
    return pos.double() if layout == "packed" else pos.double().expand(B, L)


CASES = [
    # B, L, H, H_kv, D, rot, style, layout, P, dtype
    (1, 1, 1, 1, 64, 64, "half", "contiguous", 1, torch.bfloat16),
    (2, 37, 5, 1, 128, 128, "half", "contiguous", 1, torch.bfloat16),
    (2, 37, 4, 4, 128, 128, "interleaved", "contiguous", 1, torch.bfloat16),
    (1, 48, 3, 2, 96, 32, "half", "zigzag", 3, torch.bfloat16),
    (3, 16, 2, 0, 80, 40, "half", "zigzag", 2, torch.bfloat16),      # 20 a half
    (1, 101, 0, 3, 72, 70, "interleaved", "packed", 1, torch.bfloat16),
    (1, 101, 6, 2, 256, 64, "interleaved", "packed", 1, torch.bfloat16),
    (1, 101, 3, 2, 128, 2, "interleaved", "packed", 1, torch.bfloat16),
    (2, 9, 3, 1, 64, 24, "half", "contiguous", 1, torch.bfloat16),   # 12 a half
    (2, 9, 3, 1, 80, 20, "half", "contiguous", 1, torch.bfloat16),   # 10
    (2, 9, 3, 1, 128, 126, "half", "contiguous", 1, torch.bfloat16), # 63
    (2, 9, 3, 1, 128, 122, "interleaved", "contiguous", 1, torch.float32),
    (1, 60, 2, 2, 256, 2, "half", "contiguous", 1, torch.bfloat16),  # one pair, 254 passing
    (2, 33, 3, 1, 64, 48, "half", "contiguous", 1, torch.float32),
    (1, 101, 3, 1, 100, 100, "half", "packed", 1, torch.float32),    # 50 a half
    (1, 40, 3, 1, 4, 4, "interleaved", "zigzag", 2, torch.float32),
    (1, 2500, 7, 3, 128, 64, "half", "contiguous", 1, torch.float32),
    # halves that end inside a vector: every remainder, rows of one to 32 vectors, no full warp
    (1, 33, 1, 1, 8, 2, "half", "contiguous", 1, torch.bfloat16),
    (1, 33, 1, 1, 8, 6, "half", "contiguous", 1, torch.bfloat16),
    (2, 19, 5, 2, 24, 20, "half", "contiguous", 1, torch.bfloat16),
    (1, 37, 3, 1, 256, 254, "half", "contiguous", 1, torch.bfloat16),
    (1, 37, 3, 1, 256, 246, "half", "contiguous", 1, torch.bfloat16),
    (1, 3000, 5, 3, 96, 90, "half", "packed", 1, torch.bfloat16),
    (1, 33, 2, 1, 4, 2, "half", "contiguous", 1, torch.float32),
    (1, 33, 3, 1, 128, 122, "half", "contiguous", 1, torch.float32),
    (1, 34, 3, 1, 128, 124, "half", "contiguous", 1, torch.float32),
    (1, 33, 3, 1, 132, 130, "half", "contiguous", 1, torch.float32),  # more than 32 vectors
    (1, 33, 3, 1, 256, 252, "half", "contiguous", 1, torch.float32),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:9]))
@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
def test_rotation(case, back):
    B, L, H, H_kv, D, rot, style, layout, P, dtype = case
    g = torch.Generator().manual_seed(1)
    lead = (L,) if layout == "packed" else (B, L)
    q = torch.randn(*lead, H, D, generator=g).to(dtype) if H else None
    k = torch.randn(*lead, H_kv, D, generator=g).to(dtype) if H_kv else None
    cu = [0, 1, 40, 40, L] if layout == "packed" else None
    table = cea.rope_table(rot, style=style, amplitude=1.25, device=DEV)
    kw = dict(layout=layout, P=P, offset=1000)
    if cu:
        kw["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    to = lambda t: None if t is None else t.to(DEV)
    f = cea.rope_bwd if back else cea.rope_fwd
    got = f(to(q), to(k), table, **kw)
    assert cea.check_status() == 0
    angle = (positions_of(layout, B, L, P, cu) + 1000)[..., None] * freqs(rot)
    for x, y in zip((q, k), got):
        if x is None:
            assert y is None
            continue
        ref, mag = rotate64(x.double(), -angle if back else angle, rot, style, 1.25)
        assert_rotated(y, ref, mag)
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])          # passed through, same bits
        inplace = x.to(DEV)
        f(inplace if x is q else None, inplace if x is k else None, table, **kw,
          **({"q_out": inplace} if x is q else {"k_out": inplace}))
        assert torch.equal(inplace, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_given_positions_near_and_far(dtype):
    """Any int32 position, the angle as exact as at position 0."""
    pos = torch.tensor([[0, 1, -1, 4095, 131071, 1 << 20, 10 ** 9, 2 ** 31 - 1, -2 ** 31]])
    x = torch.randn(1, pos.shape[1], 2, 128, generator=torch.Generator().manual_seed(2)).to(dtype)
    table = cea.rope_table(128, device=DEV)
    got, _ = cea.rope_fwd(x.to(DEV), None, table, positions=pos.int().to(DEV))
    assert cea.check_status() == 0
    # the reference's own angle has to be known: position times frequency in 64 bits is off by
    # |p| 2^-53 radians, 2.4e-7 at 2^31, which the tables' own rounding doubles
    ref, mag = rotate64(x.double(), pos.double()[..., None] * freqs(128), 128, "half")
    assert_rotated(got[:, :6], ref[:, :6], mag[:, :6])
    assert_rotated(got[:, 6:], ref[:, 6:], mag[:, 6:] * 2)


def test_backward_is_the_transpose_and_matches_differences():
    """<dy, R x> = <R^T dy, x>, and the gradient of a scalar against central differences of
    the forward (linear, so differences have no error but rounding)."""
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(1, 9, 2, 64, generator=g) for _ in range(2))
    table = cea.rope_table(48, style="interleaved", amplitude=0.9, device=DEV)
    y, _ = cea.rope_fwd(x.to(DEV), None, table, offset=77)
    dx, _ = cea.rope_bwd(dy.to(DEV), None, table, offset=77)
    a, b = (dy.double() * y.double().cpu()).sum(), (dx.double().cpu() * x.double()).sum()
    # a rotated value is off by at most 2^-20 0.9 times its pair's magnitudes
    assert abs(a - b) <= 2.0 ** -19 * (dy.abs().double().sum() * x.abs().max()
                                       + x.abs().double().sum() * dy.abs().max())
    h = 0.5
    for i, hd, c in ((0, 0, 0), (4, 1, 17), (8, 1, 47), (8, 0, 63)):
        e = torch.zeros_like(x)
        e[0, i, hd, c] = h
        up, _ = cea.rope_fwd((x + e).to(DEV), None, table, offset=77)
        dn, _ = cea.rope_fwd((x - e).to(DEV), None, table, offset=77)
        diff = ((up.double() - dn.double()).cpu() * dy.double()).sum() / (2 * h)
        # two evaluations of the pair's two values, each off by (2^-20 + 2^-24) of at most
        # |x_a| + |x_b| + h, and the gradient's own 2^-20 (|dy_a| + |dy_b|)
        bound = (4.2 * 2.0 ** -20 * (2 * x.abs().max() + h) + 2.0 ** -19) * dy.abs().max()
        assert abs(diff - dx[0, i, hd, c].double().cpu()) <= bound


def test_views_of_a_fused_projection():
    """q and k as strided views of one [B, L, H + 2 H_kv, D] buffer, rotated in place: the
    values in between stay."""
    H, H_kv, D = 6, 2, 64
    qkv = torch.randn(2, 19, H + 2 * H_kv, D, generator=torch.Generator().manual_seed(4)).to(
        torch.bfloat16)
    dev = qkv.to(DEV)
    q, k = dev[:, :, :H], dev[:, :, H:H + H_kv]
    table = cea.rope_table(64, device=DEV)
    want = cea.rope_fwd(q.contiguous(), k.contiguous(), table)
    cea.rope_fwd(q, k, table, q_out=q, k_out=k)
    assert cea.check_status() == 0
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(dev[:, :, H + H_kv:].cpu(), qkv[:, :, H + H_kv:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_dims_behind_the_rotation_pass_whatever_they_are(dtype, style):
    """NaN and infinities behind `rot`, in the vector that the rotation ends in too."""
    x = torch.randn(1, 6, 2, 64, generator=torch.Generator().manual_seed(9)).to(dtype)
    x[..., 54:] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 1e30] * 2).to(dtype)
    got, _ = cea.rope_fwd(x.to(DEV), None, cea.rope_table(54, style=style, amplitude=3.0, device=DEV),
                          offset=5)
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(got[..., 54:].cpu().view(bits), x[..., 54:].view(bits))
    assert torch.isfinite(got[..., :54]).all()


def test_rows_of_no_sequence_are_left():
    """Packed rows in front of the first and behind the last boundary."""
    x = torch.randn(20, 2, 64, generator=torch.Generator().manual_seed(5)).to(DEV)
    out = torch.full_like(x, 7.0)
    cu = torch.tensor([3, 8, 15], dtype=torch.int32, device=DEV)
    cea.rope_fwd(x, None, cea.rope_table(64, device=DEV), layout="packed", cu_seqlens=cu, q_out=out)
    assert cea.check_status() == 0
    assert (out[:3] == 7).all() and (out[15:] == 7).all()
    assert torch.equal(out[3], x[3]) and torch.equal(out[8], x[8])    # position 0 of each


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
def test_rows_of_no_sequence_are_zero_in_outputs_allocated_here(back, dtype):
    """The same rows where the call makes its outputs, in memory that held NaN before: a
    gradient with anything else there would reach the projection's weights."""
    g = torch.Generator().manual_seed(10)
    q, k = (torch.randn(2000, h, 64, generator=g).to(dtype).to(DEV) for h in (4, 2))
    cu = torch.tensor([3, 800, 800, 1500], dtype=torch.int32, device=DEV)
    table = cea.rope_table(64, device=DEV)
    f = cea.rope_bwd if back else cea.rope_fwd
    want = [torch.zeros_like(x) for x in (q, k)]
    f(q, k, table, layout="packed", cu_seqlens=cu, q_out=want[0], k_out=want[1])
    for _ in range(3):
        used = [torch.full((2000, h, 64), float("nan"), dtype=dtype, device=DEV)
                for h in (4, 2) * 8]
        del used
        got = f(q, k, table, layout="packed", cu_seqlens=cu)
        assert cea.check_status() == 0
        for x, y in zip(got, want):
            assert (x[:3] == 0).all() and (x[1500:] == 0).all()
            assert torch.equal(x, y)


def test_many_boundaries():
    """The 32-wide search over more sequences than one or two of its steps hold."""
    lens = [(i * 7) % 5 for i in range(2500)]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    L = cu[-1]
    x = torch.ones(L, 1, 64, device=DEV)
    got, _ = cea.rope_fwd(x, None, cea.rope_table(64, device=DEV), layout="packed",
                          cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
    pos = torch.cat([torch.arange(n) for n in lens]).double()
    ref, mag = rotate64(x.double().cpu(), pos[:, None] * freqs(64), 64, "half")
    assert_rotated(got, ref, mag)


@pytest.mark.parametrize("cu", [[0, 9, 3, 20], [-5, 4, 40, 2 ** 31 - 1], [20, 10, 5, 0], [0] * 4])
def test_malformed_boundaries_stay_in_bounds(cu, monkeypatch):
    x = torch.randn(20, 2, 64, device=DEV)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    table = cea.rope_table(64, device=DEV)
    normal = cea.load_library()
    monkeypatch.setattr(cea, "_lib", cea.load_debug_library(build_if_missing=True))
    cea.rope_fwd(x, None, table, layout="packed", cu_seqlens=c)
    assert cea.check_status() == 0
    monkeypatch.setattr(cea, "_lib", normal)
    cea.rope_fwd(x, None, table, layout="packed", cu_seqlens=c)
    assert cea.check_status() == 0


@pytest.mark.parametrize("rot,D,style,dtype", [
    (126, 128, "half", torch.bfloat16), (20, 80, "half", torch.bfloat16), (2, 8, "half", torch.bfloat16),
    (24, 64, "half", torch.bfloat16), (122, 128, "half", torch.float32), (130, 132, "half", torch.float32),
    (62, 72, "interleaved", torch.bfloat16), (46, 100, "interleaved", torch.float32)])
def test_in_place_and_checked_indices(rot, D, style, dtype, monkeypatch):
    """Rows of a fused buffer, more than a wave of blocks of them, rotated in place and by the
    index-checked build: the same bits, and nothing outside q and k changes."""
    g = torch.Generator().manual_seed(rot)
    H, H_kv, L = 3, 2, 3001
    buf = torch.randn(1, L, H + 2 * H_kv, D, generator=g).to(dtype).to(DEV)
    was = buf.clone()
    table = cea.rope_table(rot, style=style, device=DEV)
    q, k = buf[:, :, :H], buf[:, :, H:H + H_kv]
    want = cea.rope_fwd(q, k, table, offset=-7)
    angle = torch.arange(-7, L - 7, dtype=torch.float64)[:, None] * freqs(rot)
    for x, y in zip((q, k), want):
        ref, mag = rotate64(x[0].double().cpu(), angle, rot, style)
        assert_rotated(y[0], ref, mag)
    normal = cea.load_library()
    monkeypatch.setattr(cea, "_lib", cea.load_debug_library(build_if_missing=True))
    for x, y in zip(cea.rope_fwd(q, k, table, offset=-7), want):
        assert torch.equal(x, y)
    assert cea.check_status() == 0
    monkeypatch.setattr(cea, "_lib", normal)
    cea.rope_fwd(q, k, table, offset=-7, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, :, H + H_kv:], was[:, :, H + H_kv:])
    with pytest.raises(ValueError):
        cea.rope_fwd(q, k, table, offset=2 ** 31)


def test_captured_and_other_stream():
    x = torch.randn(2, 50, 4, 128, generator=torch.Generator().manual_seed(6)).to(
        torch.bfloat16).to(DEV)
    pos = torch.randint(0, 9999, (2, 50), dtype=torch.int32).to(DEV)
    table = cea.rope_table(128, device=DEV)
    want, _ = cea.rope_fwd(x, None, table, positions=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = cea.rope_fwd(x, None, table, positions=pos, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cea.rope_fwd(x, None, table, positions=pos, q_out=out)
    pos.add_(3)                                   # the replay reads what the array now holds
    graph.replay()
    assert torch.equal(out, cea.rope_fwd(x, None, table, positions=pos)[0])


def test_binding_refusals():
    x = torch.zeros(1, 4, 2, 64, device=DEV)
    t = cea.rope_table(64, device=DEV)
    bad = [
        lambda: cea.rope_fwd(None, None, t),
        lambda: cea.rope_fwd(x.cpu(), None, t),
        lambda: cea.rope_fwd(x.half(), None, t),
        lambda: cea.rope_fwd(x[0], None, t),
        lambda: cea.rope_fwd(x, None, t, layout="packed"),
        lambda: cea.rope_fwd(x, None, t, layout="striped"),
        lambda: cea.rope_fwd(x, x[:, :2], t),
        lambda: cea.rope_fwd(x, None, t, positions=torch.zeros(4, dtype=torch.int32, device=DEV)),
        lambda: cea.rope_fwd(x, None, t, positions=torch.zeros(1, 4, device=DEV)),
        lambda: cea.rope_fwd(x, None, t, q_out=x.bfloat16()),
        lambda: cea.rope_fwd(x, None, t, k_out=x),
        lambda: cea.rope_fwd(x.transpose(2, 3), None, t),
        lambda: cea.rope_fwd(x[:, :1].expand(1, 4, 2, 64), None, t),         # broadcast tokens
        lambda: cea.rope_fwd(x[:, :, :1].expand(1, 4, 2, 64), None, t),      # broadcast heads
        lambda: cea.rope_fwd(x, None, t, q_out=x[:, :1].expand(1, 4, 2, 64)),
        lambda: cea.rope_bwd(x[:1].expand(2, 4, 2, 64), None, t),            # broadcast batch
        lambda: cea.rope_table(63), lambda: cea.rope_table(64, style="third"),
        lambda: cea.rope_table(64, scaling="more"),
        lambda: cea.rope_table(64, inv_freq=[1.0]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(cea.RingAttnError):
        cea.rope_fwd(x, None, cea.rope_table(66, device=DEV))
    assert cea.rope_fwd(x[:, :0], None, t)[0].shape == (1, 0, 2, 64)


def test_custom_angles_and_amplitude():
    f = torch.tensor([1.0, 0.5, 3e-3, 0.0], dtype=torch.float64)
    x = torch.randn(1, 30, 1, 8, generator=torch.Generator().manual_seed(8))
    got, _ = cea.rope_fwd(x.to(DEV), None, cea.rope_table(8, inv_freq=f, amplitude=2.0, device=DEV))
    ref, mag = rotate64(x.double(), torch.arange(30).double()[None, :, None] * f, 8, "half", 2.0)
    assert_rotated(got, ref, mag)
    assert half_step(torch.bfloat16) == 2 ** -8 and math.isclose(half_step(torch.float32), 2 ** -24)
