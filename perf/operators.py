"""Rotary positions, appending to a paged key/value cache, and attention over that cache.

What a serving or training program does around ring attention, as cases to be measured:
`rope` rotates queries and keys (or their gradients) in place of a layer's projection
output, `append` writes a step's new keys and values into the pages of a cache (rotating
queries and keys on the way), and `attend` lets the step's queries attend to the pages.
With `own` false everything is computed in elementary torch operations in 32 bits (angles
in 64); with `own` true the library's entry points are called.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------- cases --

def listed():
    return [
        # One decoding step of 64 sequences far into their contexts: launch latency.
        dict(name="rope decode step", op="rope", dtype="bf16", direction="fwd", layout="given",
             B=64, L=1, P=1, H=32, H_kv=8, D=128, rot=128, style="half", scaling="yarn",
             factor=4.0, original=32768, top=131072),
        # The causal language-model workload, its rows in zigzag shard order.
        dict(name="rope zigzag prompt", op="rope", dtype="bf16", direction="fwd", layout="zigzag",
             B=1, L=32768, P=8, H=32, H_kv=32, D=128, rot=128, style="half", scaling="none",
             factor=1.0, original=0, top=32768),
        # Gradients of packed training samples, fp32, only part of an odd head rotated.
        dict(name="rope packed gradients", op="rope", dtype="f32", direction="bwd",
             layout="packed", B=1, L=8191, P=1, H=12, H_kv=4, D=96, rot=64, style="interleaved",
             scaling="linear", factor=2.0, original=4096, top=8191, n_seqs=7),
        # One new token of each of 128 sequences into pages of 16.
        dict(name="append decode step", op="append", dtype="bf16", n_seqs=128, new="one",
             new_max=1, kv_max=512, H=32, H_kv=8, D=128, page=16, rot=128, style="half",
             scaling="none", factor=1.0, original=0, fused=True, pad=0),
        # Prompts of six sequences, straight out of a fused projection, into pages of 64.
        dict(name="append prompts", op="append", dtype="bf16", n_seqs=6, new="ragged",
             new_max=4096, kv_max=6000, H=32, H_kv=8, D=128, page=64, rot=128, style="half",
             scaling="ntk", factor=8.0, original=8192, fused=True, pad=0),
        # A single conversation: the smallest attention call.
        dict(name="attend one token", op="attend", dtype="bf16", n_seqs=1, new="one", new_max=1,
             kv_min=1000, kv_max=1000, H=32, H_kv=8, D=128, page=16, causal=True, pad=0),
        # A full decoding batch with contexts of very different lengths.
        dict(name="attend decode batch", op="attend", dtype="bf16", n_seqs=64, new="one",
             new_max=1, kv_min=1000, kv_max=16384, H=32, H_kv=8, D=128, page=64, causal=True,
             pad=0),
        # One token over the long-context workload's 131072 keys, a key head for every head.
        dict(name="attend long context", op="attend", dtype="bf16", n_seqs=1, new="one",
             new_max=1, kv_min=131072, kv_max=131072, H=8, H_kv=8, D=128, page=128, causal=True,
             pad=0),
        # A few proposed tokens per sequence checked at once, 40 query rows per key head.
        dict(name="attend proposed tokens", op="attend", dtype="bf16", n_seqs=32, new="all",
             new_max=5, kv_min=500, kv_max=8192, H=32, H_kv=4, D=128, page=32, causal=True,
             pad=0),
        # A chunk of a long prompt: 2048 tokens that end at position 32768.
        dict(name="attend prompt chunk", op="attend", dtype="bf16", n_seqs=1, new="all",
             new_max=2048, kv_min=32768, kv_max=32768, H=32, H_kv=8, D=128, page=128,
             causal=True, pad=0),
        # Decoding and prompt chunks of odd lengths mixed in one call, head dim 64, padded.
        dict(name="attend mixed batch", op="attend", dtype="bf16", n_seqs=24, new="mixed",
             new_max=700, kv_min=1, kv_max=5000, H=12, H_kv=4, D=64, page=16, causal=True,
             pad=13),
        # fp32, as used for checks.
        dict(name="attend fp32 decode", op="attend", dtype="f32", n_seqs=16, new="one", new_max=1,
             kv_min=100, kv_max=4000, H=8, H_kv=2, D=128, page=16, causal=True, pad=0),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _scaling(rng):
    kind = rng.choice(["none", "linear", "ntk", "yarn"])
    return dict(scaling=kind, factor=1.0 if kind == "none" else rng.choice([2.0, 4.0, 8.5]),
                original=0 if kind == "none" else rng.choice([4096, 8192, 32768]))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if H_kv * group > 40:
        group = max(1, 40 // H_kv)
    H = H_kv * group
    if op == "rope":
        layout = rng.choice(["given", "contiguous", "zigzag", "packed"])
        D = rng.choice([64, 80, 96, 128, 256])
        c = dict(op="rope", dtype=dtype, direction=rng.choice(["fwd", "bwd"]), layout=layout,
                 B=1 if layout == "packed" else rng.choice([1, 2, 3]),
                 L=_log_uniform(rng, 1, 16384), P=1, H=H, H_kv=H_kv, D=D,
                 rot=rng.choice([D, D // 2, D // 4, D - 2]), style=rng.choice(["half", "interleaved"]),
                 top=_log_uniform(rng, 1, 1 << 20), **_scaling(rng))
        if layout == "zigzag":
            c["P"] = rng.choice([1, 2, 4])
            c["L"] = max(1, c["L"] // (2 * c["P"])) * 2 * c["P"]
        if layout == "packed":
            c["n_seqs"] = rng.randint(1, min(12, c["L"]))
        return c
    page = rng.choice([8, 16, 24, 32, 64, 128, 256])
    n_seqs = _log_uniform(rng, 1, 100)
    if op == "append":
        D = rng.choice([64, 80, 96, 128, 256])
        new = rng.choice(["one", "ragged", "mixed"])
        return dict(op="append", dtype=dtype, n_seqs=n_seqs, new=new,
                    new_max=1 if new == "one" else _log_uniform(rng, 2, max(2, 12000 // n_seqs)),
                    kv_max=_log_uniform(rng, 1, max(1, 40000 // n_seqs)), H=H, H_kv=H_kv, D=D,
                    page=page, rot=rng.choice([D, D // 2, D - 2]),
                    style=rng.choice(["half", "interleaved"]), fused=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 5]), **_scaling(rng))
    # attend: sizes bounded by the padded score matrix and the cache of the plain form
    D = rng.choice([64, 128])
    new = rng.choice(["one", "one", "all", "ragged", "mixed"])
    kv_max = _log_uniform(rng, 1, 65536 if dtype == "bf16" else 8192)
    while n_seqs > 1 and n_seqs * kv_max * H_kv * D > (1 << 28 if dtype == "bf16" else 1 << 25):
        n_seqs = (n_seqs + 1) // 2
    budget = (1 << 31) if dtype == "bf16" else (1 << 27)
    new_max = 1 if new == "one" else _log_uniform(rng, 2, 2048)
    new_max = max(1, min(new_max, kv_max, budget // (n_seqs * kv_max * H)))
    return dict(op="attend", dtype=dtype, n_seqs=n_seqs, new=new if new_max > 1 else "one",
                new_max=new_max, kv_min=rng.choice([1, max(1, kv_max // 2), kv_max]),
                kv_max=kv_max, H=H, H_kv=H_kv, D=D, page=page, causal=rng.random() < 0.8,
                pad=rng.choice([0, 0, 3]))


def _lengths(case):
    """(new tokens, keys including them) of every sequence: fixed by the case's sizes."""
    rng = random.Random("%(new)s %(new_max)d %(kv_max)d %(n_seqs)d" % case)
    n, top = case["n_seqs"], case["new_max"]
    if case["new"] in ("one", "all"):
        new = [top] * n
    elif case["new"] == "ragged":
        new = [rng.randint(1, top) for _ in range(n)]
        new[0] = top
    else:                                    # some sequences decode, the others bring a chunk
        new = [1 if rng.random() < 0.6 else rng.randint(1, top) for _ in range(n)]
        new[-1] = top
    lo = case.get("kv_min", 1)
    kv = [max(t, rng.randint(lo, case["kv_max"])) for t in new]
    kv[0] = max(new[0], case["kv_max"])
    return new, kv


def _packed_starts(case):
    rng = random.Random("%(L)d %(n_seqs)d" % case)
    cuts = sorted(rng.sample(range(1, case["L"]), case["n_seqs"] - 1))
    return [0] + cuts + [case["L"]]


# ------------------------------------------------------------------------- state --

def _randn(shape, dtype, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _frequencies(case):
    """Angle per position of each rotated pair, in 64 bits, and the factor on the result."""
    rot, base, s = case["rot"], 10000.0, case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * s ** (rot / (rot - 2.0)) if rot > 2 else base
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / s
    amplitude = 1.0
    if case["scaling"] == "yarn":
        def pair_of(turns):                  # pair that makes `turns` turns in the original length
            return rot * math.log(case["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0.0, math.floor(pair_of(32.0))), min(rot - 1.0, math.ceil(pair_of(1.0)))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / s * ramp
        amplitude = 0.1 * math.log(s) + 1.0
    return f.cuda(), amplitude


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    H, H_kv, D = case["H"], case["H_kv"], case["D"]
    st = dict(case=case)
    if "rot" in case:
        st["freq"], st["amplitude"] = _frequencies(case)
        if own:                              # the handle that a program makes once per model
            import context_exact_attention_gb300 as cea
            st["rope"] = cea.rope_table(case["rot"], style=case["style"], scaling=case["scaling"],
                                        factor=case["factor"], original_length=case["original"])
    if case["op"] == "rope":
        B, L = case["B"], case["L"]
        lead = (L,) if case["layout"] == "packed" else (B, L)
        st["q"] = _randn((*lead, H, D), dtype, gen)
        st["k"] = _randn((*lead, H_kv, D), dtype, gen)
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        if case["layout"] == "given":
            st["positions"] = torch.randint(0, case["top"], (B, L), generator=gen, device="cuda",
                                            dtype=torch.int32)
        if case["layout"] == "packed":
            st["cu"] = torch.tensor(_packed_starts(case), dtype=torch.int32, device="cuda")
        return st
    new, kv = _lengths(case)
    page = case["page"]
    T = sum(new) + case["pad"]
    cols = -(-max(kv) // page)
    used = sum(-(-x // page) for x in kv)
    st["pages"] = used + 3                   # a pool a little larger than what is in use
    order = torch.randperm(st["pages"], generator=gen, device="cuda")[:used].to(torch.int32)
    table = torch.zeros((len(kv), cols), dtype=torch.int32)
    held = torch.tensor([-(-x // page) for x in kv])
    table = table.cuda()
    table[(torch.arange(cols)[None] < held[:, None]).cuda()] = order
    st["table"] = table
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    st["cu"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    st["max_new"], st["max_kv"], st["T"] = max(new), max(kv), T
    head_scale = torch.rand(H_kv, generator=gen, device="cuda")[:, None] * 1.5 + 0.5
    st["k_pages"] = _randn((st["pages"], page, H_kv, D), dtype, gen)
    st["v_pages"] = _randn((st["pages"], page, H_kv, D), dtype, gen)
    if case["op"] == "append":
        if case["fused"]:                    # views of one projection's output
            qkv = _randn((T, H + 2 * H_kv, D), dtype, gen)
            st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
        else:
            st["q"] = _randn((T, H, D), dtype, gen)
            st["k"], st["v"] = _randn((T, H_kv, D), dtype, gen), _randn((T, H_kv, D), dtype, gen)
        st["q_out"] = torch.zeros((T, H, D), dtype=dtype, device="cuda")
        return st
    st["k_pages"].mul_(head_scale.to(dtype))  # heads differ in how sharply they attend
    st["q"] = _randn((T, H, D), dtype, gen)
    st["out"] = torch.zeros((T, H, D), dtype=dtype, device="cuda")
    st["lse"] = torch.zeros((T, H), dtype=torch.float32, device="cuda")
    if own:                                  # scratch that a program keeps for all its layers
        import context_exact_attention_gb300 as cea
        st["workspace"] = cea.paged_attn_workspace(D, dtype)
    return st


# ------------------------------------------------------------------------ passes --

def _rotate(x, pos, st, sign):
    """x [..., H, D] rotated by the angles of pos [...]; sign -1 is the transpose."""
    rot, D = st["case"]["rot"], x.shape[-1]
    angle = pos.double()[..., None] * st["freq"]
    cos = (torch.cos(angle) * st["amplitude"]).float()[..., None, :]
    sin = (torch.sin(angle) * (st["amplitude"] * sign)).float()[..., None, :]
    xf = x[..., :rot].float()
    if st["case"]["style"] == "half":
        a, b = xf[..., :rot // 2], xf[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = xf[..., 0::2], xf[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    y = y.to(x.dtype)
    return y if rot == D else torch.cat([y, x[..., rot:]], dim=-1)


def _rope_positions(st):
    c = st["case"]
    row = torch.arange(c["L"], device="cuda")
    if c["layout"] == "given":
        return st["positions"]
    if c["layout"] == "zigzag":              # shard r holds chunks r and 2P-1-r of 2P
        chunk = c["L"] // (2 * c["P"])
        piece, i = row // chunk, row % chunk
        shard = piece // 2
        row = torch.where(piece % 2 == 0, shard, 2 * c["P"] - 1 - shard) * chunk + i
    if c["layout"] == "packed":
        seq = torch.searchsorted(st["cu"], row.int(), right=True) - 1
        return row - st["cu"][seq]
    return row.expand(c["B"], c["L"])


def _plain_rope(st):
    sign = 1.0 if st["case"]["direction"] == "fwd" else -1.0
    pos = _rope_positions(st)
    return _rotate(st["q"], pos, st, sign), _rotate(st["k"], pos, st, sign)


def _token_positions(st):
    """(sequence, position in it) of each new token, the padding rows left out."""
    cu, lens = st["cu"].long(), st["kv_lens"].long()
    row = torch.arange(st["T"] - st["case"]["pad"], device="cuda")
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq, lens[seq] - (cu[seq + 1] - cu[seq]) + row - cu[seq]


def _plain_append(st):
    seq, pos = _token_positions(st)
    n, page = seq.numel(), st["case"]["page"]
    where = st["table"][seq, pos // page].long(), pos % page
    st["q_out"][:n] = _rotate(st["q"][:n], pos, st, 1.0)
    st["k_pages"][where] = _rotate(st["k"][:n], pos, st, 1.0)
    st["v_pages"][where] = st["v"][:n]
    return st["q_out"], st["k_pages"], st["v_pages"]


def _plain_attend(st):
    c = st["case"]
    n, H, H_kv, D = c["n_seqs"], c["H"], c["H_kv"], c["D"]
    G, page, mq, mk = H // H_kv, c["page"], st["max_new"], st["max_kv"]
    cu, lens = st["cu"].long(), st["kv_lens"].long()
    new = cu[1:] - cu[:-1]
    key = torch.arange(mk, device="cuda")
    held = key[None] < lens[:, None]                                        # [n, mk]
    at = st["table"][:, key // page].long(), (key % page).expand(n, mk)
    k = torch.where(held[..., None, None], st["k_pages"][at].float(), 0.0).permute(0, 2, 3, 1)
    v = torch.where(held[..., None, None], st["v_pages"][at].float(), 0.0).permute(0, 2, 1, 3)
    i = torch.arange(mq, device="cuda")
    real = i[None] < new[:, None]                                           # [n, mq]
    rows = torch.where(real, cu[:-1, None] + i, 0)
    q = st["q"][rows].float().view(n, mq, H_kv, G, D).permute(0, 2, 1, 3, 4)
    s = (q.reshape(n, H_kv, mq * G, D) @ k).view(n, H_kv, mq, G, mk) * (1 / math.sqrt(D))
    last = (lens - new)[:, None] + i if c["causal"] else (lens - 1)[:, None].expand(n, mq)
    seen = held[:, None, :] & (key <= last[..., None])                      # [n, mq, mk]
    s = torch.where(seen[:, None, :, None, :], s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -torch.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, H_kv, mq * G, mk) @ v).view(n, H_kv, mq, G, D) / total
    lse = (m + torch.log(total))[..., 0]
    st["out"][rows[real]] = o.permute(0, 2, 1, 3, 4).reshape(n, mq, H, D)[real].to(st["out"].dtype)
    st["lse"][rows[real]] = lse.permute(0, 2, 1, 3).reshape(n, mq, H)[real]
    return st["out"], st["lse"]


def run(st):
    c = st["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[c["op"]](st)
    import context_exact_attention_gb300 as cea
    if c["op"] == "rope":
        f = cea.rope_fwd if c["direction"] == "fwd" else cea.rope_bwd
        layout = "contiguous" if c["layout"] == "given" else c["layout"]
        return f(st["q"], st["k"], st["rope"], positions=st.get("positions"), layout=layout,
                 P=c["P"], cu_seqlens=st.get("cu"), q_out=st["q_out"], k_out=st["k_out"])
    if c["op"] == "append":
        cea.paged_kv_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["cu"],
                            st["kv_lens"], rope=st["rope"], q=st["q"], q_out=st["q_out"])
        return st["q_out"], st["k_pages"], st["v_pages"]
    return cea.paged_attn_fwd(st["q"], st["k_pages"], st["v_pages"], st["table"], st["cu"],
                              st["kv_lens"], causal=c["causal"], out=st["out"], lse=st["lse"],
                              workspace=st["workspace"])


# ------------------------------------------------------------------ floor and 64 bits --

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    H, H_kv, D = case["H"], case["H_kv"], case["D"]
    if case["op"] == "rope":
        rows = case["B"] * case["L"]
        n = rows * (H + H_kv)
        extra = rows * 4 if case["layout"] == "given" else 0
        return {"bytes": 2 * n * D * e + extra, "flops": 3 * n * case["rot"]}
    new, kv = _lengths(case)
    T, tables = sum(new), 8 * len(new) + 4 * sum(-(-x // case["page"]) for x in kv)
    if case["op"] == "append":
        return {"bytes": 2 * T * (H + 2 * H_kv) * D * e + tables,
                "flops": 3 * T * (H + H_kv) * case["rot"]}
    if case["causal"]:
        pairs = sum(t * (x - t) + t * (t + 1) // 2 for t, x in zip(new, kv))
    else:
        pairs = sum(t * x for t, x in zip(new, kv))
    return {"bytes": 2 * T * H * D * e + 4 * T * H + 2 * sum(kv) * H_kv * D * e + tables,
            "flops": 4 * D * H * pairs}


def _exact_angles(case, positions):
    """cos and sin, with the factor on them, of every position (a 64-bit tensor) and pair."""
    rot, s, kind = case["rot"], case["factor"], case["scaling"]
    freq = []
    for j in range(rot // 2):
        base = 1e4 * (s ** (rot / (rot - 2)) if kind == "ntk" and rot > 2 else 1.0)
        f = base ** (-2 * j / rot)
        if kind == "linear":
            f /= s
        if kind == "yarn":
            # pairs that turn 32 times or more in the original length keep their frequency,
            # those that turn less than once are slowed by the factor, the rest in between
            index = [rot * math.log(case["original"] / (2 * math.pi * b)) / (2 * math.log(base))
                     for b in (32.0, 1.0)]
            a, b = max(math.floor(index[0]), 0), min(math.ceil(index[1]), rot - 1)
            slow = min(max((j - a) / max(b - a, 0.001), 0.0), 1.0)
            f *= 1 - slow + slow / s
        freq.append(f)
    ang = torch.outer(positions, torch.tensor(freq, dtype=torch.float64, device="cuda"))
    amp = 0.1 * math.log(s) + 1 if kind == "yarn" else 1.0
    return amp * ang.cos(), amp * ang.sin()


def _exact_rotation(x, case, positions, backwards=False):
    """x [rows, H, D] as complex pairs times e^(i angle)."""
    half, y = case["rot"] // 2, x.double().clone()
    cos, sin = _exact_angles(case, positions)
    turn = torch.complex(cos, -sin if backwards else sin)[:, None, :]
    if case["style"] == "half":
        z = torch.complex(y[:, :, :half].clone(), y[:, :, half:2 * half].clone()) * turn
        y[:, :, :half], y[:, :, half:2 * half] = z.real, z.imag
    else:
        z = torch.complex(y[:, :, 0:2 * half:2].clone(), y[:, :, 1:2 * half:2].clone()) * turn
        y[:, :, 0:2 * half:2], y[:, :, 1:2 * half:2] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    H, H_kv, D = case["H"], case["H_kv"], case["D"]
    if case["op"] == "rope":
        B, L, P = case["B"], case["L"], case["P"]
        if case["layout"] == "given":
            pos = st["positions"].reshape(-1).tolist()
        elif case["layout"] == "packed":
            cu = _packed_starts(case)
            pos = [i for a, b in zip(cu, cu[1:]) for i in range(b - a)]
        elif case["layout"] == "zigzag":
            c = L // (2 * P)
            pos = [x * c + i for r in range(P) for x in (r, 2 * P - 1 - r) for i in range(c)] * B
        else:
            pos = list(range(L)) * B
        pos = torch.tensor(pos, dtype=torch.float64, device="cuda")
        back = case["direction"] == "bwd"
        return tuple(_exact_rotation(st[n].reshape(-1, st[n].shape[-2], D), case, pos, back)
                     .reshape(st[n].shape) for n in ("q", "k"))
    new, kv = _lengths(case)
    page = case["page"]
    if case["op"] == "append":
        q, kp, vp = (st[n].double() for n in ("q_out", "k_pages", "v_pages"))
        at = 0
        for g, (t, x) in enumerate(zip(new, kv)):
            pos = torch.arange(x - t, x, device="cuda")
            q[at:at + t] = _exact_rotation(st["q"][at:at + t], case, pos.double())
            flat = st["table"][g].long()[pos // page] * page + pos % page
            kp.view(-1, H_kv, D)[flat] = _exact_rotation(st["k"][at:at + t], case, pos.double())
            vp.view(-1, H_kv, D)[flat] = st["v"][at:at + t].double()
            at += t
        return q, kp, vp
    out, lse = st["out"].double(), st["lse"].double()
    at = 0
    for g, (t, x) in enumerate(zip(new, kv)):
        slots = (st["table"][g, :-(-x // page)].long()[:, None] * page
                 + torch.arange(page, device="cuda")).reshape(-1)[:x]
        for h in range(H_kv):
            k = st["k_pages"].view(-1, H_kv, D)[slots, h].double()
            v = st["v_pages"].view(-1, H_kv, D)[slots, h].double()
            for f in range(h * (H // H_kv), (h + 1) * (H // H_kv)):
                s = st["q"][at:at + t, f].double() @ k.T / D ** 0.5
                if case["causal"] and t > 1:
                    s += torch.full((t, x), -math.inf, dtype=torch.float64,
                                    device="cuda").triu(x - t + 1)
                lse[at:at + t, f] = torch.logsumexp(s, -1)
                out[at:at + t, f] = torch.softmax(s, -1) @ v
        at += t
    return out, lse
