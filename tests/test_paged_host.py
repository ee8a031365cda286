"""Rotary positions and the paged cache, host side (no GPU): the descriptors' layouts, the
frequency tables against 64-bit arithmetic, and every refusal of the new entry points, which
come back before anything is launched."""
import ctypes
import math

import numpy as np
import pytest

import context_exact_attention_gb300 as cea
from context_exact_attention_gb300 import _build

OK, INVALID, UNSUPPORTED, MISALIGNED, INDIVISIBLE = 0, 1, 2, 3, 4
S = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return cea.load_library()


def at(i):
    """A fake device address, 1 TiB apart, never dereferenced."""
    return ctypes.c_void_p((i + 1) << 40)


def test_descriptor_layouts():
    assert ctypes.sizeof(cea.Rope) == 24 and cea.Rope.amplitude.offset == 16
    assert ctypes.sizeof(cea.RopeConfig) == 48 and cea.RopeConfig.base.offset == 8
    assert ctypes.sizeof(cea.RopeDesc) == 96
    assert cea.RopeDesc.cu_seqlens.offset == 32 and cea.RopeDesc.positions.offset == 48
    assert cea.RopeDesc.q_stride.offset == 64
    assert ctypes.sizeof(cea.PagedDesc) == 96
    assert cea.PagedDesc.page_stride.offset == 32 and cea.PagedDesc.page_table.offset == 64
    assert cea.PagedDesc.dtype.offset == 88


def phases(lib, **kw):
    c = cea.RopeConfig(rot_dim=128, scaling=0, base=1e4, factor=1.0, original_length=0.0,
                       beta_fast=32.0, beta_slow=1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    out = (ctypes.c_ulonglong * (c.rot_dim // 2))()
    amp = ctypes.c_float(0)
    rc = lib.ra_rope_phases(ctypes.byref(c), out, ctypes.byref(amp))
    return rc, np.array(out, dtype=np.uint64), amp.value


def turns(freq):
    """2^64 of the fraction of a turn of angles in radians, as Python integers."""
    from fractions import Fraction
    two_pi = Fraction(math.pi) * 2 + Fraction(2.4492935982947064e-16)   # 2 pi to 107 bits
    return [int(Fraction(f) / two_pi % 1 * 2 ** 64) for f in freq]


def near(got, ref):
    """Fixed-point phases within the rounding of the 64-bit frequency (a few 2^-52)."""
    for g, r in zip(got, ref):
        d = abs(int(g) - r)
        assert min(d, 2 ** 64 - d) <= max(4, r >> 50), (g, r)


def test_frequencies_of_every_scaling(lib):
    i = np.arange(64, dtype=np.float64)
    plain = 1e4 ** (-2 * i / 128)
    rc, ph, amp = phases(lib)
    assert rc == OK and amp == 1.0
    near(ph, turns(plain))
    rc, ph, amp = phases(lib, scaling=1, factor=4.0)
    assert rc == OK and amp == 1.0
    near(ph, turns(plain / 4))
    rc, ph, amp = phases(lib, scaling=2, factor=8.0)
    assert rc == OK and amp == 1.0
    near(ph, turns((1e4 * 8.0 ** (128 / 126)) ** (-2 * i / 128)))
    rc, ph, amp = phases(lib, scaling=3, factor=16.0, original_length=4096.0)
    assert rc == OK and amp == np.float32(0.1 * math.log(16) + 1)
    # pairs with 32 turns and more over 4096 positions keep their frequency, those with less
    # than one are 16 times slower; the ramp is monotone in between
    n_turns = 4096 * plain / (2 * math.pi)
    ratio = np.array([int(p) for p in ph], dtype=np.float64) / np.array(turns(plain), dtype=np.float64)
    assert np.allclose(ratio[n_turns >= 33], 1) and np.allclose(ratio[n_turns < 0.9], 1 / 16)
    assert (np.diff(ratio) <= 1e-12).all()


def test_phases_of_given_angles(lib):
    f = np.array([0.0, 1.0, 2 * math.pi, 7.0, -0.25, 1e-9, -1e-30], dtype=np.float64)
    out = (ctypes.c_ulonglong * len(f))()
    assert lib.ra_rope_phases_of(f.ctypes.data_as(ctypes.c_void_p), len(f), out) == OK
    got = [int(x) for x in out]
    for g, r in zip(got, turns(f.tolist())):
        d = abs(g - r)
        assert min(d, 2 ** 64 - d) <= 2 ** 13
    # position times phase, modulo 2^64, is the angle modulo a turn at any position
    for p in (1, 131071, 10 ** 9):
        frac = (p * got[1] % 2 ** 64) / 2 ** 64
        exact = (p / (2 * math.pi)) % 1
        assert abs((frac - exact + 0.5) % 1 - 0.5) < p * 2.0 ** -50


def test_phase_refusals(lib):
    assert phases(lib, base=0.0)[0] == INVALID
    assert phases(lib, base=math.nan)[0] == INVALID
    assert phases(lib, scaling=1, factor=0.0)[0] == INVALID
    assert phases(lib, scaling=2, factor=math.inf)[0] == INVALID
    assert phases(lib, scaling=4)[0] == INVALID
    assert phases(lib, scaling=3, factor=2.0)[0] == INVALID                   # no original length
    assert phases(lib, scaling=3, factor=2.0, original_length=1e3, beta_fast=1.0)[0] == INVALID
    amp, out = ctypes.c_float(0), (ctypes.c_ulonglong * 1)()
    c = cea.RopeConfig(rot_dim=3, scaling=0, base=1e4)
    assert lib.ra_rope_phases(ctypes.byref(c), out, ctypes.byref(amp)) == INVALID
    assert lib.ra_rope_phases(None, out, ctypes.byref(amp)) == INVALID
    bad = (ctypes.c_double * 1)(math.inf)
    assert lib.ra_rope_phases_of(bad, 1, out) == INVALID
    assert lib.ra_rope_phases_of(bad, 0, out) == INVALID
    assert lib.ra_rope_phases_of(None, 1, out) == INVALID


def rope(**kw):
    d = dict(phases=1 << 20, rot_dim=64, style=0, amplitude=1.0)
    d.update(kw)
    return ctypes.byref(cea.Rope(**d))


def test_rope_refusals(lib):
    def call(r=None, q=at(0), k=at(1), qo=at(2), ko=at(3), **kw):
        d = dict(B=1, L=64, H=4, H_kv=2, D=64, P=1, layout=0, dtype=0)
        d.update(kw)
        return [f(ctypes.byref(cea.RopeDesc(**d)), r or rope(), q, k, qo, ko, S)
                for f in (lib.rope_fwd, lib.rope_bwd)]

    both = lambda code: [code, code]
    null = ctypes.c_void_p(0)
    assert lib.rope_fwd(None, rope(), at(0), at(1), at(2), at(3), S) == INVALID
    assert lib.rope_fwd(ctypes.byref(cea.RopeDesc(B=1, L=1, H=1, H_kv=1, D=64, P=1)), None, at(0),
                        at(1), at(2), at(3), S) == INVALID
    for kw in (dict(B=0), dict(L=0), dict(H=-1), dict(P=0), dict(H=0, H_kv=0)):
        assert call(**kw) == both(INVALID), kw
    assert call(dtype=2) == both(UNSUPPORTED)
    assert call(D=60) == both(UNSUPPORTED) and call(D=264) == both(UNSUPPORTED)
    for kw in (dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=66), dict(style=2),
               dict(phases=0), dict(amplitude=math.inf)):
        assert call(rope(**kw)) == both(INVALID), kw
    assert call(rope(phases=(1 << 20) + 4)) == both(MISALIGNED)
    # pointers and head counts agree
    assert call(q=null) == both(INVALID) and call(ko=null) == both(INVALID)
    assert call(H=0) == both(INVALID)
    # layouts and positions
    assert call(layout=3) == both(INVALID)
    assert call(layout=1, P=5) == both(INDIVISIBLE)
    assert call(layout=0, P=5) == both(INDIVISIBLE)
    assert call(layout=2) == both(INVALID)                                     # no boundaries
    assert call(layout=2, cu_seqlens=1 << 20, n_seqs=2, B=2) == both(INVALID)
    assert call(layout=2, cu_seqlens=(1 << 20) + 2, n_seqs=2) == both(MISALIGNED)
    assert call(layout=0, cu_seqlens=1 << 20, n_seqs=2) == both(INVALID)
    assert call(layout=1, P=2, positions=1 << 20) == both(INVALID)
    assert call(positions=(1 << 20) + 1) == both(MISALIGNED)
    # strides: shorter than a row, not whole 16-byte pieces
    assert call(q_stride=128) == both(INVALID) and call(q_stride=260) == both(MISALIGNED)
    assert call(k_out_stride=-256) == both(INVALID)
    odd = ctypes.c_void_p((5 << 40) + 8)
    assert call(q=odd) == both(MISALIGNED) and call(ko=odd) == both(MISALIGNED)
    # overlap: shifted in place, output on the other input, outputs on one another
    assert call(qo=ctypes.c_void_p((1 << 40) + 16)) == both(INVALID)
    assert call(qo=at(0), q_out_stride=512) == both(INVALID)
    assert call(qo=at(1)) == both(INVALID) and call(ko=at(0)) == both(INVALID)
    assert call(qo=at(2), ko=at(2)) == both(INVALID)
    assert call(qo=ctypes.c_void_p(1 << 20)) == both(INVALID)                  # on the phases
    assert call(positions=3 << 40, qo=at(2)) == both(INVALID)
    # interleaved rows that do collide: k starts inside q's row
    fused = dict(q_stride=512, k_stride=512, q_out_stride=512, k_out_stride=512)
    assert call(qo=at(0), k=ctypes.c_void_p((1 << 40) + 256), ko=at(3), **fused) == both(INVALID)
    # too many elements
    assert call(B=2 ** 20, L=2 ** 20) == both(INVALID)


def paged(**kw):
    d = dict(T=8, n_seqs=2, H=4, H_kv=2, D=64, num_pages=10, page_size=16, max_pages=4,
             page_stride=16 * 2 * 64, token_stride=128, head_stride=64, table_stride=4,
             page_table=1 << 20, cu_new=2 << 20, kv_lens=3 << 20, dtype=0, causal=1)
    d.update(kw)
    return ctypes.byref(cea.PagedDesc(**d))


COMMON = [
    (dict(T=-1), INVALID), (dict(n_seqs=0), INVALID), (dict(H_kv=0), INVALID),
    (dict(D=0), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(page_table=0), INVALID),
    (dict(cu_new=0), INVALID), (dict(kv_lens=0), INVALID),
    (dict(page_table=(1 << 20) + 2), MISALIGNED), (dict(cu_new=(2 << 20) + 1), MISALIGNED),
    (dict(kv_lens=(3 << 20) + 3), MISALIGNED), (dict(table_stride=3), INVALID),
    (dict(page_stride=-2048), INVALID), (dict(token_stride=64), INVALID),     # slots on heads
    (dict(head_stride=32), INVALID), (dict(page_stride=1024), INVALID),       # pages on slots
    (dict(token_stride=132), MISALIGNED), (dict(page_stride=1 << 41), INVALID),
]


def test_append_refusals(lib):
    def call(d, r=rope(), q=at(0), qs=0, k=at(1), ks=0, v=at(2), vs=0, qo=at(3), qos=0, kp=at(4),
             vp=at(5)):
        return lib.paged_kv_append(d, r, q, qs, k, ks, v, vs, qo, qos, kp, vp, S)

    null = ctypes.c_void_p(0)
    assert call(None) == INVALID
    for kw, code in COMMON:
        assert call(paged(**kw)) == code, kw
    assert call(paged(D=60, token_stride=120, head_stride=60)) != OK
    assert call(paged(D=264, head_stride=264, token_stride=528, page_stride=16 * 528)) == UNSUPPORTED
    assert call(paged(), r=rope(rot_dim=66)) == INVALID
    for kw in (dict(k=null), dict(v=null), dict(kp=null), dict(vp=null), dict(q=null),
               dict(qo=null)):
        assert call(paged(), **kw) == INVALID, kw
    assert call(paged(H=0)) == INVALID
    assert call(paged(), qs=128) == INVALID and call(paged(), vs=132) == MISALIGNED
    assert call(paged(), kp=ctypes.c_void_p((5 << 40) + 8)) == MISALIGNED
    # overlap: pages on inputs, on tables, on one another (alternating views are fine)
    assert call(paged(), kp=at(1)) == INVALID and call(paged(), vp=at(3)) == INVALID
    assert call(paged(), kp=at(4), vp=at(4)) == INVALID
    assert call(paged(), vp=ctypes.c_void_p((5 << 40) + 2048)) == INVALID
    assert call(paged(), kp=ctypes.c_void_p((1 << 20) - 1024)) == INVALID
    assert call(paged(), qo=at(1)) == INVALID
    assert call(paged(), qo=ctypes.c_void_p((1 << 40) + 128)) == INVALID
    # no tokens: nothing to do, and no CUDA call is made
    assert call(paged(T=0)) == OK
    two = dict(T=0, page_stride=2 * 2048)
    assert call(paged(**two), vp=ctypes.c_void_p((5 << 40) + 4096)) == OK       # [pages, 2, ...]
    assert call(paged(**two), vp=ctypes.c_void_p((5 << 40) + 2048)) == INVALID
    two = dict(T=0, page_stride=4096, token_stride=256)
    assert call(paged(**two), vp=ctypes.c_void_p((5 << 40) + 256)) == OK        # [.., 2, H, D]
    assert call(paged(**two), vp=ctypes.c_void_p((5 << 40) + 128)) == INVALID
    two = dict(T=0, page_stride=4096, token_stride=256, head_stride=128)
    assert call(paged(**two), vp=ctypes.c_void_p((5 << 40) + 128)) == OK        # [.., H, 2, D]
    assert call(paged(**two), vp=ctypes.c_void_p((5 << 40) + 64)) == INVALID


def test_attention_refusals(lib):
    need = lib.paged_attn_workspace_bytes(64, 0)
    assert need > 0 and need % 4 == 0

    def call(d, q=at(0), qs=0, kp=at(1), vp=at(2), out=at(3), lse=at(4), ws=at(5), n=None):
        return lib.paged_attn_fwd(d, q, qs, kp, vp, out, lse, ws,
                                  ctypes.c_ulonglong(need if n is None else n), S)

    null = ctypes.c_void_p(0)
    assert call(None) == INVALID
    for kw, code in COMMON:
        assert call(paged(**kw)) == code, kw
    assert call(paged(D=96, head_stride=96, token_stride=192, page_stride=16 * 192)) == UNSUPPORTED
    assert call(paged(D=258, dtype=1, head_stride=260, token_stride=520, page_stride=16 * 520)) == UNSUPPORTED
    for kw in (dict(q=null), dict(kp=null), dict(vp=null), dict(out=null), dict(ws=null)):
        assert call(paged(), **kw) == INVALID, kw
    assert call(paged(H=0)) == INVALID and call(paged(H=5)) == INDIVISIBLE
    assert call(paged(), qs=128) == INVALID and call(paged(), qs=260) == MISALIGNED
    assert call(paged(), n=need - 1) == INVALID
    assert call(paged(), ws=ctypes.c_void_p((6 << 40) + 128)) == MISALIGNED
    assert call(paged(), out=ctypes.c_void_p((4 << 40) + 8)) == MISALIGNED
    assert call(paged(), lse=ctypes.c_void_p((5 << 40) + 2)) == MISALIGNED
    for i in (0, 1, 2):
        assert call(paged(), out=at(i)) == INVALID and call(paged(), lse=at(i)) == INVALID
        assert call(paged(), ws=at(i)) == INVALID
    assert call(paged(), lse=at(3)) == INVALID and call(paged(), ws=at(3)) == INVALID
    assert call(paged(page_table=4 << 40)) == INVALID                          # out on the table
    assert call(paged(T=2 ** 30, H=4)) == INVALID                              # T * H
    assert call(paged(T=0)) == OK and call(paged(T=0), lse=null) == OK


def test_workspace_sizes(lib):
    f = lib.paged_attn_workspace_bytes
    assert f(64, 0) > 0 and f(128, 0) > f(64, 0)
    assert f(96, 0) == 0 and f(256, 0) == 0 and f(64, 2) == 0
    assert f(4, 1) > 0 and f(256, 1) > 0 and f(6, 1) == 0 and f(260, 1) == 0 and f(0, 1) == 0


def test_packed_descriptors_are_the_structures():
    """The byte formats that the binding packs are the structures' layouts."""
    rope_fields = [f[0] for f in cea.RopeDesc._fields_]
    values = list(range(1, len(rope_fields) + 1))
    packed = cea._ROPE_DESC.pack(*values)
    assert len(packed) == ctypes.sizeof(cea.RopeDesc)
    d = cea.RopeDesc.from_buffer_copy(packed)
    assert [getattr(d, f) for f in rope_fields] == values
    paged_fields = [f[0] for f in cea.PagedDesc._fields_]
    values = list(range(1, len(paged_fields) + 1))
    packed = cea._PAGED_DESC.pack(*values)
    assert len(packed) == ctypes.sizeof(cea.PagedDesc)
    d = cea.PagedDesc.from_buffer_copy(packed)
    assert [getattr(d, f) for f in paged_fields] == values
