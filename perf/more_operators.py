"""A step of drafted tokens: pages, normalised heads, a tree's attention, what is kept of it.

What a serving program does around paged attention when it checks a tree of drafted tokens for
every sequence, and a training program around ring attention when queries and keys are
normalised per head, as cases to be measured: `reserve` finds the step's rows, positions, masks
and page slots on the GPU (and gives pages back), `norm` normalises and rotates query and key
heads or computes the gradients of that, `append` does it on the way into the pages, `tree`
lets every drafted token attend to the cache and its ancestors, `keep` moves what was accepted
to its place.  With `own` false everything is computed in elementary torch operations in 32
bits (angles and long sums in 64); with `own` true the library's entry points are called.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------- cases --

def listed():
    return [
        # The bookkeeping of one decoding step of 64 sequences: launch latency.
        dict(name="reserve decode step", op="reserve", n_seqs=64, new="one", new_max=1,
             kv_max=16384, page=64, words=0, pad=0),
        # Every sequence of a large server brings a tree of up to 61 drafted tokens.
        dict(name="reserve drafted trees", op="reserve", n_seqs=1024, new="ragged", new_max=61,
             kv_max=4000, page=16, words=2, pad=100),
        # One decoding step of 64 sequences far into their contexts, heads normalised.
        dict(name="norm decode step", op="norm", direction="fwd", dtype="bf16", layout="given",
             B=64, L=1, P=1, H=32, H_kv=8, D=128, rot=128, style="half", base=1e6, weight="bf16",
             plus=0.0, top=131072),
        # The causal language-model workload's length in zigzag shard order, grouped heads.
        dict(name="norm zigzag prompt", op="norm", direction="fwd", dtype="bf16", layout="zigzag",
             B=1, L=32768, P=8, H=32, H_kv=8, D=128, rot=128, style="half", base=1e6,
             weight="bf16", plus=0.0, top=32768),
        # Gradients of packed training samples, of the heads and of both weights.
        dict(name="norm packed gradients", op="norm", direction="bwd", dtype="bf16",
             layout="packed", B=1, L=16381, P=1, H=32, H_kv=8, D=128, rot=128, style="half",
             base=1e6, weight="f32", plus=0.0, top=16381, n_seqs=7),
        # The drafted trees of 32 sequences enter the cache at their depths' positions.
        dict(name="append drafted trees", op="append", dtype="bf16", n_seqs=32, new="ragged",
             new_max=64, kv_max=8192, H=32, H_kv=8, D=128, page=64, rot=128, style="half",
             base=1e6, weight="bf16", plus=0.0, tree=True, pad=3),
        # Prompt chunks of four sequences, views of one projection's output.
        dict(name="append prompt chunks", op="append", dtype="bf16", n_seqs=4, new="all",
             new_max=2048, kv_max=8192, H=32, H_kv=8, D=128, page=64, rot=128, style="half",
             base=1e6, weight="bf16", plus=0.0, tree=False, pad=0),
        # One user's tree of 26 drafted tokens over a short context: latency.
        dict(name="tree one sequence", op="tree", dtype="bf16", n_seqs=1, new="all", new_max=26,
             kv_min=2000, kv_max=2000, H=32, H_kv=8, D=128, page=16, words=1, pad=0),
        # Trees of up to 64 drafted tokens of a full batch, contexts of different lengths.
        dict(name="tree batch", op="tree", dtype="bf16", n_seqs=32, new="ragged", new_max=64,
             kv_min=500, kv_max=8192, H=32, H_kv=8, D=128, page=64, words=2, pad=0),
        # fp32, as used for checks.
        dict(name="tree fp32", op="tree", dtype="f32", n_seqs=4, new="ragged", new_max=13,
             kv_min=100, kv_max=1500, H=8, H_kv=2, D=128, page=16, words=1, pad=2),
        # What 16 sequences accepted of small trees, in one layer's cache: launch latency.
        dict(name="keep one layer", op="keep", dtype="bf16", n_seqs=16, nodes=26, path=5,
             kv_max=1000, layers=1, H_kv=8, D=128, page=16),
        # A full batch's accepted tokens in the caches of all layers at once.
        dict(name="keep all layers", op="keep", dtype="bf16", n_seqs=64, nodes=61, path=8,
             kv_max=500, layers=12, H_kv=8, D=128, page=64),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["reserve", "norm", "norm", "append", "tree", "tree", "keep"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([8, 16, 24, 32, 64, 128, 256])
    if op == "reserve":
        n = _log_uniform(rng, 1, 1024)
        words = rng.choice([0, 0, 1, 2, 4])
        new = rng.choice(["one", "ragged", "mixed"])
        most = max(2, 62000 // n)
        new_max = 1 if new == "one" else _log_uniform(rng, 2, min(most, 32 * words or 20000))
        return dict(op=op, n_seqs=n, new=new, new_max=new_max, kv_max=_log_uniform(rng, 1, 20000),
                    page=page, words=words, pad=rng.choice([0, 0, 7, 100]))
    H_kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if H_kv * group > 40:
        group = max(1, 40 // H_kv)
    H = H_kv * group
    if op in ("norm", "append"):
        D = rng.choice([64, 80, 96, 128, 256])
        heads = dict(H=H, H_kv=H_kv, D=D, rot=rng.choice([D, D, D // 2, D // 4, D - 2]),
                     style=rng.choice(["half", "half", "interleaved"]),
                     base=rng.choice([1e4, 5e5, 1e6]),
                     weight=rng.choice([dtype, "f32"]), plus=rng.choice([0.0, 0.0, 1.0]))
    if op == "norm":
        layout, B = rng.choice(["given", "contiguous", "zigzag", "packed"]), rng.choice([1, 2, 3])
        B = 1 if layout == "packed" else B
        most = (1 << 26) // (B * (H + H_kv) * heads["D"])
        c = dict(op=op, direction=rng.choice(["fwd", "bwd"]), dtype=dtype, layout=layout, B=B,
                 L=_log_uniform(rng, 1, min(16384, most)), P=1, top=_log_uniform(rng, 1, 1 << 20),
                 **heads)
        if layout == "zigzag":
            c["P"] = rng.choice([1, 2, 4])
            c["L"] = max(1, c["L"] // (2 * c["P"])) * 2 * c["P"]
        if layout == "packed":
            c["n_seqs"] = rng.randint(1, min(12, c["L"]))
        return c
    if op == "append":
        n = _log_uniform(rng, 1, 100)
        tree = rng.random() < 0.6
        new = rng.choice(["one", "ragged", "mixed"])
        most = (1 << 26) // (n * (H + 2 * H_kv) * heads["D"])
        most = min(most, 12000 // n, 128 if tree else 12000)
        return dict(op=op, dtype=dtype, n_seqs=n, new=new,
                    new_max=1 if new == "one" else _log_uniform(rng, 2, max(2, most)),
                    kv_max=_log_uniform(rng, 1, max(1, 40000 // n)), page=page, tree=tree,
                    pad=rng.choice([0, 0, 5]), **heads)
    if op == "tree":
        D = rng.choice([64, 128])
        n, kv_max = _log_uniform(rng, 1, 64), _log_uniform(rng, 1, 20000 if dtype == "bf16" else 4000)
        while n > 1 and n * kv_max * H_kv * D > (1 << 27 if dtype == "bf16" else 1 << 24):
            n = (n + 1) // 2
        words = rng.choice([1, 1, 2, 4, 8])
        budget = (1 << 27) if dtype == "bf16" else (1 << 24)
        new_max = max(1, min(_log_uniform(rng, 1, 32 * words), kv_max, budget // (n * kv_max * H)))
        return dict(op=op, dtype=dtype, n_seqs=n, new=rng.choice(["all", "ragged", "mixed"]),
                    new_max=new_max, kv_min=rng.choice([1, max(1, kv_max // 2), kv_max]),
                    kv_max=kv_max, H=H, H_kv=H_kv, D=D, page=page, words=words,
                    pad=rng.choice([0, 0, 3]))
    n, D = _log_uniform(rng, 1, 64), rng.choice([64, 80, 96, 128, 256])
    nodes = _log_uniform(rng, 1, 64)
    layers = rng.choice([1, 1, 2, 5, 8])
    kv_max = _log_uniform(rng, nodes, max(nodes, min(2000, (1 << 27) // (n * layers * H_kv * D))))
    return dict(op="keep", dtype=dtype, n_seqs=n, nodes=nodes, path=rng.randint(1, max(1, nodes // 3)),
                kv_max=kv_max, layers=layers, H_kv=H_kv, D=D, page=page)


def _lengths(case):
    """(new tokens, keys including them) of every sequence: fixed by the case's sizes."""
    n = case["n_seqs"]
    if case["op"] == "keep":
        rng = random.Random("%(nodes)d %(kv_max)d %(n_seqs)d" % case)
        new = [case["nodes"]] * n
    else:
        rng = random.Random("%(new)s %(new_max)d %(kv_max)d %(n_seqs)d" % case)
        top = case["new_max"]
        if case["new"] in ("one", "all"):
            new = [top] * n
        elif case["new"] == "ragged":
            new = [rng.randint(1, top) for _ in range(n)]
        else:                                # some sequences bring one token or rest, others many
            new = [rng.randint(0, 1) if rng.random() < 0.6 else rng.randint(1, top)
                   for _ in range(n)]
        new[-1] = top
    lo = case.get("kv_min", 1)
    kv = [max(t, rng.randint(lo, case["kv_max"])) for t in new]
    kv[0] = max(new[0], case["kv_max"])
    return new, kv


def _parents(new, seed):
    """Drafted trees, sequence after sequence: the parent of every node within its sequence's
    new tokens (-1: it follows the sequence itself), the node it extends being a recent one."""
    rng = random.Random(seed)
    out = []
    for n in new:
        out += [-1 if i == 0 or rng.random() < 0.02 else max(0, i - 1 - int(rng.expovariate(0.25)))
                for i in range(n)]
    return out


def _paths(case):
    """Accepted nodes of every sequence.  Levels of a drafted tree are wider than it is deep, so
    that all but the first lie behind the place that they move to and the others'."""
    rng = random.Random("%(nodes)d %(path)d %(n_seqs)d" % case)
    paths = []
    for _ in range(case["n_seqs"]):
        k = rng.randint(1, case["path"])
        paths.append([0] + sorted(rng.sample(range(k, case["nodes"]), k - 1)) if k > 1 else [0])
    return paths


def _packed_starts(case):
    rng = random.Random("%(L)d %(n_seqs)d" % case)
    return [0] + sorted(rng.sample(range(1, case["L"]), case["n_seqs"] - 1)) + [case["L"]]


# ------------------------------------------------------------------------- state --

def _randn(shape, dtype, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(case):
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    return torch.pow(torch.tensor(case["base"], dtype=torch.float64), -2.0 * i / case["rot"]).cuda()


def _weights(case, gen):
    """What training leaves of a norm's weights: spread around one (less `plus`)."""
    return [(1.0 - case["plus"] + 0.3 * torch.randn(case["D"], generator=gen, device="cuda"))
            .to(DTYPES[case["weight"]]) for _ in "qk"]


def _rope(case):
    import context_exact_attention_gb300 as cea
    return cea.rope_table(case["rot"], base=case["base"], style=case["style"])


def _tables(case, kv, gen, spare=3):
    """A page table with pages in random order (-1 behind them) and the pages left over."""
    page = case["page"]
    held = torch.tensor([-(-x // page) for x in kv])
    cols, used = int(held.max()), int(held.sum())
    order = torch.randperm(used + spare, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(kv), cols), -1, dtype=torch.int32, device="cuda")
    table[(torch.arange(cols)[None] < held[:, None]).cuda()] = order[:used]
    return table, held.to(torch.int32).cuda(), order[used:]


def _starts(new):
    out = [0]
    for x in new:
        out.append(out[-1] + x)
    return out


def _masks_of(parents, new, words):
    """Ancestors of every node, itself among them, as bits of `words` 32-bit words, and depths."""
    rows, depths, at = [], [], 0
    for n in new:
        own_bits = []
        for i in range(n):
            p = parents[at + i]
            own_bits.append((own_bits[p] if p >= 0 else 0) | 1 << i)
            depths.append(depths[at + p] + 1 if p >= 0 else 0)
        rows += own_bits
        at += n
    signed = [[((b >> 32 * w & 0xffffffff) ^ 0x80000000) - 0x80000000 for w in range(words)]
              for b in rows]
    return signed, depths


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    if own:
        import context_exact_attention_gb300 as cea
    if case["op"] == "norm":
        dtype, (B, L) = DTYPES[case["dtype"]], (case["B"], case["L"])
        lead = (L,) if case["layout"] == "packed" else (B, L)
        # a projection's output: heads of different sizes, a token's scale on all of them
        token = 2.0 ** (2 * torch.rand((*lead, 1, 1), generator=gen, device="cuda") - 1)
        for n, h in (("q", case["H"]), ("k", case["H_kv"])):
            st[n] = (_randn((*lead, h, case["D"]), torch.float32, gen) * token).to(dtype)
            if case["direction"] == "bwd":
                st["d" + n + "_out"] = _randn((*lead, h, case["D"]), dtype, gen)
            st[n + "_res"] = torch.empty_like(st[n])
        st["wq"], st["wk"] = _weights(case, gen)
        if case["layout"] == "given":
            st["positions"] = torch.randint(0, case["top"], (B, L), generator=gen, device="cuda",
                                            dtype=torch.int32)
        if case["layout"] == "packed":
            st["cu"] = _ints(_packed_starts(case))
        st["freq"] = _frequencies(case)
        if own:
            st["rope"] = _rope(case)
            if case["direction"] == "bwd":   # scratch that a program keeps for all its layers
                st["workspace"] = cea.qk_norm_workspace()
        return st
    new, kv = _lengths(case)
    n, page = len(new), case["page"]
    st["cu"], st["kv_lens"] = _ints(_starts(new)), _ints(kv)
    if case["op"] == "reserve":
        lens = [x - t for t, x in zip(new, kv)]
        st["new"], st["lens"] = _ints(new), _ints(lens)
        T, cols = sum(new) + case["pad"], -(-max(kv) // page)
        more = sum(-(-x // page) - -(-y // page) for x, y in zip(kv, lens))
        table, held, free = _tables(case, lens, gen, more + 5)
        st["table"] = torch.full((n, cols), -1, dtype=torch.int32, device="cuda")
        st["table"][:, :table.shape[1]] = table
        st["T"], pages = T, int(held.sum()) + free.numel()
        stack = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        stack[:free.numel()] = free
        if case["words"]:
            st["parents"] = _ints(_parents(new, seed) + [-1] * case["pad"])
        if own:
            st["pool"] = cea.page_pool(pages, n)
            st["pool"].free.copy_(stack)
            st["pool"].held.copy_(held)
            st["pool"].count.fill_(free.numel())
            st["step"] = cea.paged_step(n, T, mask_words=case["words"])
        else:
            st["free"], st["held"], st["count"] = stack, held, _ints([free.numel()])
        return st
    dtype, D, H_kv = DTYPES[case["dtype"]], case["D"], case["H_kv"]
    st["table"], held, free = _tables(case, kv, gen)
    pages = int(held.sum()) + free.numel()
    if case["op"] == "keep":
        shape = (case["layers"], pages, page, H_kv, D)
        st["k_pages"], st["v_pages"] = _randn(shape, dtype, gen), _randn(shape, dtype, gen)
        paths = _paths(case)
        st["kept"] = _ints([p + [-1] * (case["path"] - len(p)) for p in paths])
        st["lens"] = torch.empty(n, dtype=torch.int32, device="cuda")
        return st
    H, T = case["H"], sum(new) + case["pad"]
    st["T"], st["max_new"], st["max_kv"] = T, max(new), max(kv)
    shape = (pages, page, H_kv, D)
    st["k_pages"], st["v_pages"] = _randn(shape, dtype, gen), _randn(shape, dtype, gen)
    if case["op"] == "append":
        qkv = _randn((T, H + 2 * H_kv, D), dtype, gen)   # views of one projection's output
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
        st["q_out"] = torch.zeros((T, H, D), dtype=dtype, device="cuda")
        st["wq"], st["wk"] = _weights(case, gen)
        st["freq"] = _frequencies(case)
        if case["tree"]:
            depths = _masks_of(_parents(new, seed), new, 1)[1]
            first = [x - t for t, x in zip(new, kv) for _ in range(t)]
            st["positions"] = _ints([a + d for a, d in zip(first, depths)] + [0] * case["pad"])
        if own:
            st["rope"] = _rope(case)
        return st
    head_scale = torch.rand(H_kv, generator=gen, device="cuda")[:, None] * 1.5 + 0.5
    st["k_pages"].mul_(head_scale.to(dtype))  # heads differ in how sharply they attend
    st["q"] = _randn((T, H, D), dtype, gen)
    masks = _masks_of(_parents(new, _tree_seed(case)), new, case["words"])[0]
    st["masks"] = _ints(masks + [[0] * case["words"]] * case["pad"])
    st["out"] = torch.zeros((T, H, D), dtype=dtype, device="cuda")
    st["lse"] = torch.zeros((T, H), dtype=torch.float32, device="cuda")
    if own:                                  # scratch that a program keeps for all its layers
        st["workspace"] = cea.paged_attn_workspace(D, dtype)
    return st


def _tree_seed(case):
    return "%(new_max)d %(n_seqs)d %(kv_max)d" % case


# ------------------------------------------------------------------------ passes --

def _plain_reserve(st):
    c, T = st["case"], st["T"]
    page, table, held = c["page"], st["table"], st["held"]
    new, old = st["new"].long().clamp(min=0), st["lens"].long().clamp(min=0)
    n, cols = table.shape
    total = old + new
    need = (-(-total // page) - held).clamp(min=0)
    end, taken = torch.cumsum(new, 0), torch.cumsum(need, 0)
    fits = (end[-1] <= T) & (taken[-1] <= st["count"][0]) & (total <= cols * page).all()
    new, need = torch.where(fits, new, 0), torch.where(fits, need, 0)
    end, taken = torch.cumsum(new, 0), torch.cumsum(need, 0)
    cu = torch.cat([torch.zeros_like(end[:1]), end])
    kv_lens = (old + new).int()
    # pages from the top of the stack, sequence by sequence, column by column
    col = torch.arange(cols, device="cuda")
    nth = (taken - need)[:, None] + col - held[:, None]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    at = (st["count"].long() - 1 - nth).clamp(0, st["free"].numel() - 1)
    reserved = torch.where(fresh, st["free"][at], table)
    row = torch.arange(T, device="cuda")
    seq = torch.searchsorted(end, row, right=True).clamp(max=n - 1)
    i = row - cu[seq]
    real = row < end[-1]
    place = torch.where(real, old[seq] + i, 0)
    slots = torch.where(real, reserved[seq, place // page].long() * page + place % page, -1)
    if c["words"]:
        # ancestors: every node takes over what the one 1, 2, 4, ... steps up has gathered
        bits = torch.where(i[:, None] // 32 == torch.arange(c["words"], device="cuda"),
                           1 << (i % 32)[:, None], 0) * real[:, None]
        up = torch.where(real, st["parents"].long(), -1)
        up = torch.where(up >= 0, row - i + up, -1)
        depth = torch.where(up >= 0, 1, 0)
        for _ in range((c["new_max"] - 1).bit_length()):
            on, at = up >= 0, up.clamp(min=0)
            bits |= bits[at] * on[:, None]
            depth = depth + depth[at] * on
            up = torch.where(on, up[at], -1)
        masks = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
        place = old[seq] + depth
    positions = torch.where(real, place, 0).int()
    table.copy_(reserved)
    held += need.int()
    st["count"] -= taken[-1:].int()
    return (cu.int(), kv_lens, positions, slots) + ((masks,) if c["words"] else ())


def _plain_release(st):
    page, table, held = st["case"]["page"], st["table"], st["held"]
    left = torch.minimum(-(-st["lens"].long().clamp(min=0) // page), held)
    gone = held - left
    taken = torch.cumsum(gone, 0)
    col = torch.arange(table.shape[1], device="cuda")
    back = (col >= left[:, None]) & (col < held[:, None])
    nth = (taken - gone)[:, None] + col - left[:, None]      # the first one ends on top
    at = (st["count"].long() + taken[-1:])[:, None] - 1 - nth
    size = st["free"].numel()                # entries that stay go to a place behind the stack
    grown = torch.cat([st["free"], st["free"][:1]])
    grown.scatter_(0, torch.where(back, at, size).flatten(), table.flatten())
    st["free"].copy_(grown[:size])
    table.masked_fill_(back, -1)
    held.copy_(left)
    st["count"] += taken[-1:].int()


def _rotate(x, pos, st, sign):
    """x [..., H, D] in fp32 rotated by the angles of pos [...]; sign -1 is the transpose."""
    rot, D = st["case"]["rot"], x.shape[-1]
    angle = pos.double()[..., None] * st["freq"]
    cos, sin = angle.cos().float()[..., None, :], (sign * angle.sin()).float()[..., None, :]
    xr = x[..., :rot]
    if st["case"]["style"] == "half":
        a, b = xr[..., :rot // 2], xr[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = xr[..., 0::2], xr[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return y if rot == D else torch.cat([y, x[..., rot:]], dim=-1)


def _norm_positions(st):
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


def _normed(x, w, st):
    """The normalised heads (fp32, without the weights), their factor, and the weights."""
    xf = x.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    return xf * r, r, w.float() + st["case"]["plus"]


def _plain_norm(st):
    pos = _norm_positions(st)
    outs, grads = [], []
    for n in "qk":
        x, r, w = _normed(st[n], st["w" + n], st)
        if st["case"]["direction"] == "fwd":
            outs.append(_rotate(x * w, pos, st, 1.0).to(st[n].dtype))
            continue
        dz = _rotate(st["d" + n + "_out"].float(), pos, st, -1.0)
        g = dz * w
        outs.append((r * (g - x * (g * x).mean(-1, keepdim=True))).to(st[n].dtype))
        grads.append((dz * x).flatten(0, -2).sum(0, dtype=torch.float64).float())
    return (*outs, *grads)


def _token_places(st):
    """(sequence, place in it) of each new token, the padding rows left out."""
    cu, lens = st["cu"].long(), st["kv_lens"].long()
    row = torch.arange(st["T"] - st["case"]["pad"], device="cuda")
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq, lens[seq] - (cu[seq + 1] - cu[seq]) + row - cu[seq]


def _plain_append(st):
    seq, place = _token_places(st)
    n, page = seq.numel(), st["case"]["page"]
    where = st["table"][seq, place // page].long(), place % page
    pos = st["positions"][:n] if st["case"]["tree"] else place
    for x, w, dst, at in (("q", "wq", "q_out", slice(n)), ("k", "wk", "k_pages", where)):
        y, _, weight = _normed(st[x][:n], st[w], st)
        st[dst][at] = _rotate(y * weight, pos, st, 1.0).to(st[x].dtype)
    st["v_pages"][where] = st["v"][:n]
    return st["q_out"], st["k_pages"], st["v_pages"]


def _plain_tree(st):
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
    node = key[None] - (lens - new)[:, None]        # which new token a key is, or negative
    word = st["masks"][rows].gather(2, (node.clamp(min=0) // 32).clamp(max=c["words"] - 1)
                                    [:, None].expand(n, mq, mk))
    bit = (word >> (node % 32)[:, None].int()) & 1
    seen = held[:, None] & ((node < 0)[:, None] | ((bit > 0) & (node < 32 * c["words"])[:, None]))
    s = torch.where(seen[:, None, :, None, :], s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -torch.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, H_kv, mq * G, mk) @ v).view(n, H_kv, mq, G, D) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0]
    st["out"][rows[real]] = o.permute(0, 2, 1, 3, 4).reshape(n, mq, H, D)[real].to(st["out"].dtype)
    st["lse"][rows[real]] = lse.permute(0, 2, 1, 3).reshape(n, mq, H)[real]
    return st["out"], st["lse"]


def _plain_keep(st):
    page, kept = st["case"]["page"], st["kept"]
    n, K = kept.shape
    first = (st["kv_lens"] - (st["cu"][1:] - st["cu"][:-1])).long()
    real = kept >= 0
    seq = torch.arange(n, device="cuda")[:, None].expand(n, K)
    src = first[:, None] + kept.clamp(min=0)
    dst = torch.where(real, first[:, None] + torch.arange(K, device="cuda"), src)

    def slot(at):
        return st["table"][seq, at // page].long(), at % page

    for pages in (st["k_pages"], st["v_pages"]):
        (sp, so), (dp, do) = slot(src), slot(dst)
        pages[:, dp, do] = pages[:, sp, so]
    st["lens"].copy_(first + real.sum(1))
    return st["k_pages"], st["v_pages"], st["lens"]


def _own_norm(st, cea):
    c = st["case"]
    more = dict(rope=st["rope"], eps=EPS, weight_offset=c["plus"], positions=st.get("positions"),
                layout="contiguous" if c["layout"] == "given" else c["layout"], P=c["P"],
                cu_seqlens=st.get("cu"))
    if c["direction"] == "fwd":
        return cea.qk_norm_rope_fwd(st["q"], st["k"], st["wq"], st["wk"], q_out=st["q_res"],
                                    k_out=st["k_res"], **more)
    return cea.qk_norm_rope_bwd(st["q"], st["k"], st["wq"], st["wk"], st["dq_out"], st["dk_out"],
                                dq=st["q_res"], dk=st["k_res"], workspace=st["workspace"], **more)


def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "reserve":
            step = _plain_reserve(st)
            _plain_release(st)
            return (*step, st["table"], st["held"], st["count"], st["free"])
        return {"norm": _plain_norm, "append": _plain_append, "tree": _plain_tree,
                "keep": _plain_keep}[c["op"]](st)
    import context_exact_attention_gb300 as cea
    if c["op"] == "reserve":
        # the step's pages, and back again to the lengths before it
        pool = st["pool"]
        s = cea.paged_reserve(pool, st["new"], st["lens"], st["table"], c["page"], st["step"],
                              parents=st.get("parents"))
        cea.paged_release(pool, st["lens"], st["table"], c["page"])
        masks = (s.masks,) if c["words"] else ()
        return (s.cu_new, s.kv_lens, s.positions, s.slots, *masks, st["table"], pool.held,
                pool.count, pool.free)
    if c["op"] == "norm":
        return _own_norm(st, cea)
    if c["op"] == "append":
        cea.paged_kv_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["cu"],
                            st["kv_lens"], rope=st["rope"], q=st["q"], q_out=st["q_out"],
                            positions=st.get("positions"), q_weight=st["wq"], k_weight=st["wk"],
                            eps=EPS, weight_offset=c["plus"])
        return st["q_out"], st["k_pages"], st["v_pages"]
    if c["op"] == "tree":
        return cea.paged_attn_fwd(st["q"], st["k_pages"], st["v_pages"], st["table"], st["cu"],
                                  st["kv_lens"], masks=st["masks"], out=st["out"], lse=st["lse"],
                                  workspace=st["workspace"])
    cea.paged_kv_keep(st["kept"], st["k_pages"], st["v_pages"], st["table"], st["cu"],
                      st["kv_lens"], lens=st["lens"])
    return st["k_pages"], st["v_pages"], st["lens"]


# ------------------------------------------------------------------ floor and 64 bits --

def work(case):
    if case["op"] == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["B"] * case["L"]
        n, back = rows * (case["H"] + case["H_kv"]), case["direction"] == "bwd"
        weights = 2 * case["D"] * (2 if case["weight"] == "bf16" else 4)
        return {"bytes": (3 if back else 2) * n * case["D"] * e + weights * (1 + back)
                + (4 * rows if case["layout"] == "given" else 0),
                "flops": n * ((9 if back else 4) * case["D"] + 3 * case["rot"])}
    new, kv = _lengths(case)
    n, T, page = len(new), sum(new), case["page"]
    if case["op"] == "reserve":
        T += case["pad"]
        more = sum(-(-x // page) - -(-(x - t) // page) for t, x in zip(new, kv))
        # rows' outputs (and parents), the sequences' arrays, and pages there and back
        return {"bytes": T * (12 + (4 + 4 * case["words"] if case["words"] else 0)) + 28 * n + 16 * more,
                "flops": 2 * T + 4 * n}
    e = 2 if case["dtype"] == "bf16" else 4
    H_kv, D = case["H_kv"], case["D"]
    tables = 8 * n + 4 * sum(-(-x // page) for x in kv)
    if case["op"] == "keep":
        paths = _paths(case)
        moved = sum(a != b for p in paths for b, a in enumerate(p))
        return {"bytes": 4 * moved * H_kv * D * e * case["layers"] + 12 * n + 4 * n * case["path"],
                "flops": n}
    H = case["H"]
    if case["op"] == "append":
        return {"bytes": 2 * T * (H + 2 * H_kv) * D * e + 12 * n + 4 * T * (1 + case["tree"]),
                "flops": T * (H + H_kv) * (4 * D + 3 * case["rot"])}
    masks = _masks_of(_parents(new, _tree_seed(case)), new, case["words"])[0]
    pairs = sum(t * (x - t) for t, x in zip(new, kv)) + sum(bin(w & 0xffffffff).count("1")
                                                             for m in masks for w in m)
    return {"bytes": 2 * T * H * D * e + 4 * T * (H + case["words"]) + 2 * sum(kv) * H_kv * D * e
            + tables, "flops": 4 * D * H * pairs}


def _exact_heads(x, w, case, positions):
    """x [rows, H, D] normalised over D, weighted, its pairs turned as complex numbers."""
    x = x.double()
    y = (w.double() + case["plus"]) * x / (x.pow(2).sum(-1, keepdim=True) / case["D"] + EPS).sqrt()
    half = case["rot"] // 2
    freq = torch.tensor([case["base"] ** (-2 * j / case["rot"]) for j in range(half)],
                        dtype=torch.float64, device="cuda")
    angle = torch.outer(positions.double(), freq)[:, None]
    turn = torch.complex(angle.cos(), angle.sin())
    if case["style"] == "half":
        z = torch.complex(y[..., :half], y[..., half:2 * half]) * turn
        return torch.cat([z.real, z.imag, y[..., 2 * half:]], -1)
    z = torch.complex(y[..., 0:2 * half:2], y[..., 1:2 * half:2]) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), y[..., 2 * half:]], -1)


def exact(case, seed):
    if case["op"] == "reserve":
        return None                          # whole numbers, held against the plain form's
    st = prepare(case, seed)
    if case["op"] == "norm":
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
        outs, grads = [], []
        for n in "qk":
            x = st[n].reshape(-1, st[n].shape[-2], case["D"]).double()
            w = st["w" + n].double()
            if case["direction"] == "fwd":
                outs.append(_exact_heads(x, w, case, pos).view(st[n].shape))
                continue
            x.requires_grad_(True)
            w.requires_grad_(True)
            _exact_heads(x, w, case, pos).backward(st["d" + n + "_out"].double().view(x.shape))
            outs.append(x.grad.view(st[n].shape))
            grads.append(w.grad)
        return (*outs, *grads)
    new, kv = _lengths(case)
    page, D, H_kv = case["page"], case["D"], case["H_kv"]

    def slots(g, a, b):
        at = torch.arange(a, b, device="cuda")
        return st["table"][g].long()[at // page] * page + at % page

    if case["op"] == "keep":
        k, v = (st[x].double().view(case["layers"], -1, H_kv, D) for x in ("k_pages", "v_pages"))
        for g, path in enumerate(_paths(case)):
            at = slots(g, kv[g] - new[g], kv[g])
            for to, node in enumerate(path):
                k[:, at[to]], v[:, at[to]] = k[:, at[node]].clone(), v[:, at[node]].clone()
        lens = [x - t + len(p) for t, x, p in zip(new, kv, _paths(case))]
        shape = st["k_pages"].shape
        return k.view(shape), v.view(shape), _ints(lens)
    if case["op"] == "append":
        q, kp, vp = (st[x].double() for x in ("q_out", "k_pages", "v_pages"))
        at = 0
        for g, (t, x) in enumerate(zip(new, kv)):
            rows, flat = slice(at, at + t), slots(g, x - t, x)
            pos = st["positions"][rows] if case["tree"] else torch.arange(x - t, x, device="cuda")
            q[rows] = _exact_heads(st["q"][rows], st["wq"], case, pos)
            kp.view(-1, H_kv, D)[flat] = _exact_heads(st["k"][rows], st["wk"], case, pos)
            vp.view(-1, H_kv, D)[flat] = st["v"][rows].double()
            at += t
        return q, kp, vp
    out, lse = st["out"].double(), st["lse"].double()
    parents = _parents(new, _tree_seed(case))
    at, H = 0, case["H"]
    for g, (t, x) in enumerate(zip(new, kv)):
        hidden = torch.zeros((t, x), dtype=torch.float64)
        for i in range(t):
            hidden[i, x - t:] = -math.inf
            node = i
            while node >= 0:
                hidden[i, x - t + node] = 0.0
                node = parents[at + node]
        hidden, flat = hidden.cuda(), slots(g, 0, x)
        for h in range(H_kv):
            k = st["k_pages"].view(-1, H_kv, D)[flat, h].double()
            v = st["v_pages"].view(-1, H_kv, D)[flat, h].double()
            for f in range(h * (H // H_kv), (h + 1) * (H // H_kv)):
                s = st["q"][at:at + t, f].double() @ k.T / D ** 0.5 + hidden
                lse[at:at + t, f] = torch.logsumexp(s, -1)
                out[at:at + t, f] = torch.softmax(s, -1) @ v
        at += t
    return out, lse
