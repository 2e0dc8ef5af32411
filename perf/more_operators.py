"""Measured cases of the paged cache's 4-bit formats and of its page management: rows written to
4-bit pages and read back, attention of new tokens over 4-bit pages, pages copied, sequences
forked, grown and freed, and pools compacted.

``run`` computes an operator in its plain form, in elementary torch operations, or (``own``)
through the library's public calls.  Sizes follow the repository's workloads: 12 and 32 heads
of 128 channels, chunks of 3 x 30 x 52 = 4680 tokens, 32760 cached tokens; and generic ones for
grouped heads, single-token decoding and sampling several continuations of a prompt.

A 4-bit row: groups of 16 channels, a the row's largest magnitude, a_g a group's, TOP the largest
code (6 for E2M1, 7 for INT4); scale s = a / (64 TOP) in fp32, group scale t = E4M3(64 a_g / a),
code = round(x 64 TOP / (a t)) to 4 bits, value = s t code.  Two codes a byte, the first one in
the low four bits.
"""
import math
import random

import torch

own = False

D = 128
GROUP = 16
CHUNK_GRID = (30, 52)  # rows and columns of a frame of the 1.3B-class shape
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "int8": torch.int8,
         "e2m1": torch.float4_e2m1fn_x2, "int4": torch.uint8}
NBYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
TOP = {"e2m1": 6.0, "int4": 7.0}  # largest code
# bytes of one row of a page: codes, group scales, scale
ROW = {"bf16": 256, "fp16": 256, "e4m3": 132, "int8": 132, "e2m1": 76, "int4": 76}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ALL = 2 ** 31 - 1


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the last few tokens of a chunk, turned and rounded to E2M1 and read back: latency
        dict(name="store_few_e2m1", kind="store", tokens=61, heads=8, dtype="fp16", fmt="e2m1",
             page=16, layout="half", rot=128, axes=1, far=100000, out="bf16"),
        # seven chunks of video tokens, turned on three axes, into INT4 pages and read back for compression
        dict(name="store_window_int4", kind="store", tokens=32760, heads=12, dtype="bf16", fmt="int4",
             page=64, layout="interleaved", rot=128, axes=3, far=60, out="bf16"),
        # one new token of eight short sequences over E2M1 pages: latency
        dict(name="decode_small_e2m1", kind="attend", seqs=8, q_lo=1, q_hi=1, len_lo=100, len_hi=2000,
             lens_seed=1, q_heads=32, heads=8, dtype="bf16", fmt="e2m1", page=16, causal=True,
             window=0, lse=False),
        # one new token of 32 long sequences over INT4 pages, to be joined with another part by its log-sum-exp
        dict(name="decode_long_int4", kind="attend", seqs=32, q_lo=1, q_hi=1, len_lo=9000,
             len_hi=20000, lens_seed=2, q_heads=32, heads=8, dtype="bf16", fmt="int4", page=64,
             causal=True, window=0, lse=True),
        # ragged prompts with what is cached before them, grouped heads, a sliding window
        dict(name="prefill_ragged_int4", kind="attend", seqs=6, q_lo=17, q_hi=2000, len_lo=500,
             len_hi=9000, lens_seed=3, q_heads=32, heads=8, dtype="fp16", fmt="int4", page=32,
             causal=True, window=4096, lse=True),
        # a video chunk over the seven chunks of its history: every query sees every key
        dict(name="chunk_over_e2m1", kind="attend", seqs=1, q_lo=4680, q_hi=4680, len_lo=32760,
             len_hi=32760, lens_seed=0, q_heads=12, heads=12, dtype="bf16", fmt="e2m1", page=64,
             causal=False, window=0, lse=False),
        # the part-filled pages of a few sequences
        dict(name="copy_few_bf16", kind="copy", count=9, pages=64, heads=8, page=16, fmt="bf16", part=True),
        # a 32760-token window of a 12-head layer, moved within a pool of 8-bit pages
        dict(name="copy_window_e4m3", kind="copy", count=512, pages=1500, heads=12, page=64, fmt="e4m3",
             part=False),
        # four continuations of one prompt started again, a token each: latency
        dict(name="branch_few", kind="branch", prompts=1, each=4, len_lo=900, len_hi=900, lens_seed=4,
             heads=8, page=16, fmt="e4m3", new=1),
        # seven continuations of each of 64 prompts started again, five tokens each
        dict(name="branch_many", kind="branch", prompts=64, each=7, len_lo=200, len_hi=3000, lens_seed=5,
             heads=8, page=16, fmt="int4", new=5),
        # a small pool of 16-bit pages, a third of them live
        dict(name="compact_small", kind="compact", seqs=5, len_lo=0, len_hi=900, lens_seed=6, share=0,
             pages=400, heads=4, page=16, fmt="fp16"),
        # a serving pool after most of its sequences ended, prompts shared by pairs of those left
        dict(name="compact_large_int4", kind="compact", seqs=64, len_lo=2000, len_hi=12000, lens_seed=7,
             share=1500, pages=30000, heads=8, page=32, fmt="int4"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["store", "store", "attend", "attend", "attend", "attend", "copy", "branch", "compact"])
    page = rng.choice([16, 32, 64, 128])
    any_fmt = rng.choice(["bf16", "fp16", "e4m3", "int8", "e2m1", "int4"])
    if kind == "store":
        heads = _log_int(rng, 1, 32)
        layout = rng.choice(["none", "half", "interleaved"])
        return dict(kind=kind, tokens=_log_int(rng, 1, 32760 * 12 // heads), heads=heads,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), fmt=rng.choice(["e2m1", "int4"]), page=page,
                    layout=layout, rot=0 if layout == "none" else rng.choice([32, 64, 128]),
                    axes=rng.choice([1, 3]), far=_log_int(rng, 10, 1000000),
                    out=rng.choice(["bf16", "fp16", "fp32"]))
    if kind == "copy":
        heads = _log_int(rng, 1, 32)
        count = _log_int(rng, 1, max(2, 400000 // (heads * page)))
        return dict(kind=kind, count=count, pages=2 * count + _log_int(rng, 1, 50), heads=heads, page=page,
                    fmt=any_fmt, part=rng.random() < 0.5)
    if kind == "branch":
        heads, prompts = _log_int(rng, 1, 16), _log_int(rng, 1, 64)
        top = _log_int(rng, 1, max(2, 1500000 // (heads * prompts)))
        return dict(kind=kind, prompts=prompts, each=_log_int(rng, 1, 8), len_lo=rng.choice([0, top // 2, top]),
                    len_hi=top, lens_seed=rng.randrange(1 << 30), heads=heads, page=page, fmt=any_fmt,
                    new=rng.choice([0, 1, 1, 5, 16, 100]))
    if kind == "compact":
        heads, seqs = _log_int(rng, 1, 16), _log_int(rng, 1, 64)
        top = _log_int(rng, 1, max(2, 3000000 // (heads * seqs)))
        share = rng.choice([0, 0, top // 4])
        need = seqs * (-(-top // page))
        return dict(kind=kind, seqs=seqs, len_lo=rng.choice([0, top // 2, top]), len_hi=top,
                    lens_seed=rng.randrange(1 << 30), share=share, pages=need + _log_int(rng, 1, 2 * need + 2),
                    heads=heads, page=page, fmt=any_fmt)
    dtype = rng.choice(["bf16", "fp16"])
    heads = rng.choice([1, 2, 4, 8, 12])
    q_heads = heads * rng.choice([1, 1, 2, 4, 7, 8])
    decode = rng.random() < 0.4
    if decode:
        seqs, q_hi = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 5])
        len_hi = _log_int(rng, 8, max(16, 5000000 // (seqs * heads)))
    else:
        seqs, q_hi = _log_int(rng, 1, 12), _log_int(rng, 2, 4096)
        len_hi = _log_int(rng, q_hi, max(q_hi + 1, 1800000000 // (seqs * q_heads * q_hi)))
    len_hi = min(len_hi, 130000)
    q_hi = min(q_hi, len_hi)
    return dict(kind=kind, seqs=seqs, q_lo=q_hi if decode else rng.choice([0, 1, q_hi]), q_hi=q_hi,
                len_lo=rng.choice([0, len_hi // 2, len_hi]), len_hi=len_hi,
                lens_seed=rng.randrange(1 << 30), q_heads=q_heads, heads=heads, dtype=dtype,
                fmt=rng.choice(["e2m1", "int4"]), page=page, causal=rng.random() < 0.6,
                window=rng.choice([0, 0, 1 + len_hi // 3]), lse=rng.random() < 0.5)


def _lengths(case):
    """(query tokens, cached tokens) of each sequence, the same for every seed of the inputs."""
    r = random.Random(case["lens_seed"])
    n_seqs = case["seqs"] if "seqs" in case else case["prompts"]
    kv = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n_seqs)]
    q = [min(r.randint(case["q_lo"], case["q_hi"]), n) if "q_lo" in case else 0 for n in kv]
    if "q_lo" in case and sum(q) == 0:
        q[0], kv[0] = max(1, case["q_lo"]), max(kv[0], 1, case["q_lo"])
    return q, kv


# ---------------------------------------------------------------- 4-bit rows in 32 bits

def _amax(x):
    return x.abs().amax(-1)


def _codes(x, fmt):
    """(bytes of two codes, group scales, scale) of fp32 rows x."""
    top = TOP[fmt]
    g = x.unflatten(-1, (D // GROUP, GROUP))
    ag = _amax(g)
    a = ag.amax(-1)
    live = a > 0
    t = torch.where(live[..., None], ag * 64.0 / a[..., None], 0.0).to(torch.float8_e4m3fn)
    t32 = t.float()
    y = torch.where((t32 > 0)[..., None], (g * (64.0 * top)) / (a[..., None] * t32)[..., None], 0.0)
    m = y.abs()
    if fmt == "int4":
        q = y.round().clamp(-top, top).to(torch.int32) & 15
    else:
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
        m = (torch.round(m / step) * step).clamp(max=top)
        q = torch.where(m <= 2, 2 * m, torch.where(m <= 4, m + 2, 7.0)).to(torch.int32)
        q = q + torch.where(y < 0, 8, 0)
    q = q.flatten(-2).unflatten(-1, (D // 2, 2))
    return (q[..., 0] | (q[..., 1] << 4)).to(torch.uint8), t, a / (64.0 * top)


def _values(pages, t, scale, fmt):
    """fp32 rows of 4-bit pages."""
    b = pages.view(torch.uint8).to(torch.int32)
    q = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    if fmt == "int4":
        c = (q - ((q & 8) << 1)).float()
    else:
        c = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=b.device)[q]
    c = c.unflatten(-1, (D // GROUP, GROUP)) * t.float()[..., None]
    return c.flatten(-2) * scale[..., None]


def _new_pool(case, pages):
    """Empty pages of a format: codes of K and V, their scales, their group scales."""
    fmt, shape = case["fmt"], (pages, case["heads"], case["page"])
    out = {}
    for name in ("k", "v"):
        if fmt in TOP:
            out[name] = torch.zeros((*shape, D // 2), dtype=torch.uint8, device="cuda").view(TORCH[fmt])
            out[name + "_group"] = torch.zeros((*shape, D // GROUP), dtype=torch.uint8,
                                               device="cuda").view(torch.float8_e4m3fn)
        else:
            out[name] = torch.zeros((*shape, D), dtype=TORCH[fmt], device="cuda")
            out[name + "_group"] = None
        out[name + "_scale"] = None if fmt in ("bf16", "fp16") else torch.zeros(shape, device="cuda")
    return out


POOLS = ("k", "v", "k_scale", "v_scale", "k_group", "v_group")


def _raw(st):
    """The pools as whole numbers: copies are of bits, whatever they stand for."""
    return [st[x].view(torch.int32 if x.endswith("scale") else torch.uint8) for x in POOLS if st[x] is not None]


# ---------------------------------------------------------------- inputs

def _frequencies(case):
    """(angle per position of each pair in radians, axis of each pair, pairs of each axis)."""
    half, axes = case["rot"] // 2, case["axes"]
    counts = [half] if axes == 1 else [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    freq, axis = [], []
    for a, n in enumerate(counts):
        freq += [1e4 ** (-i / n) for i in range(n)]
        axis += [a] * n
    return torch.tensor(freq, dtype=torch.float64), axis, counts


def _positions(case, n, gen):
    """int64 [axes][n]: grid positions of a video chunk, or a sequence's from a far one on."""
    start = int(torch.randint(0, max(1, case["far"]), (1,), generator=torch.Generator().manual_seed(gen.initial_seed())))
    i = torch.arange(n, device="cuda")
    if case["axes"] == 3:
        h, w = CHUNK_GRID
        return torch.stack([start + i // (h * w), i // w % h, i % w])
    return (start + i).view(1, n)


def _order(case, pages, gen):
    return torch.randperm(pages, generator=torch.Generator().manual_seed(gen.initial_seed())).tolist()


def _attend_state(case, gen):
    """4-bit pages with their tables and lengths; what no sequence reaches holds NaN scales and
    any codes, as memory that nobody wrote may."""
    q, kv = _lengths(case)
    page, heads, fmt = case["page"], case["heads"], case["fmt"]
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 3
    order = _order(case, pages, gen)
    table = torch.full((len(kv), max(1, max(need))), -1, dtype=torch.int32)
    token = torch.full((pages, page), False)  # written rows
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[sum(need[:b]):sum(need[:b]) + n], dtype=torch.int32)
        rows = token.new_zeros(n * page)
        rows[:kv[b]] = True
        token[table[b, :n].long()] = rows.view(n, page)
    token = token.to("cuda")[:, None, :]
    st = {}
    for name in ("k", "v"):
        x = torch.randn((pages, heads, page, D), device="cuda", generator=gen)
        x[..., 5::41] *= 6.0  # a few outlier channels, as keys have
        codes, t, scale = _codes(x, fmt)
        st[name], st[name + "_group"] = codes.view(TORCH[fmt]), t
        st[name + "_scale"] = torch.where(token, scale, float("nan"))
    st["table"] = table.to("cuda")
    st["lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    st["cu_q"] = torch.tensor([sum(q[:b]) for b in range(len(q) + 1)], dtype=torch.int32, device="cuda")
    st["max_q"], st["max_kv"] = max(q), max(kv)
    st["Q"] = torch.randn((sum(q), case["q_heads"], D), device="cuda", generator=gen).to(TORCH[case["dtype"]])
    return st


def _fill(st, gen):
    """Any codes and positive scales."""
    for name in POOLS:
        if st[name] is None:
            continue
        if name.endswith("scale"):
            st[name].copy_(torch.rand(st[name].shape, device="cuda", generator=gen))
        else:
            b = st[name].view(torch.uint8)
            b.copy_(torch.randint(0, 120, b.shape, dtype=torch.uint8, device="cuda", generator=gen))


def _branch_layout(case):
    """Rows: the prompts, then `each` continuations of every prompt.  (lengths, parents)."""
    _, lens = _lengths(case)
    n, each = case["prompts"], case["each"]
    parents = [-1] * n + [i // each for i in range(n * each)]
    return lens, parents


def _branch_state(case, gen):
    lens, parents = _branch_layout(case)
    page, n, kids = case["page"], case["prompts"], case["prompts"] * case["each"]
    top = -(-(max(lens) + case["new"]) // page) + 1
    own_pages = [-(-x // page) for x in lens]
    # what the continuations hold from before: a page or two of their own
    left = [random.Random(case["lens_seed"] + i).randint(0, 2 * page) for i in range(kids)]
    left = [min(x, top * page) for x in left]
    grow = -(-case["new"] // page) + 2
    pages = sum(own_pages) + sum(-(-x // page) for x in left) + kids * grow + 5
    order = _order(case, pages, gen)
    table = torch.full((n + kids, top), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    for b, x in enumerate(lens + left):
        m = -(-x // page)
        mine, order = order[:m], order[m:]
        table[b, :m] = torch.tensor(mine, dtype=torch.int32)
        refs[torch.tensor(mine, dtype=torch.int64)] += 1
    st = _new_pool(case, pages)
    _fill(st, gen)
    st["table"], st["refs"] = table.to("cuda"), refs.to("cuda")
    st["lens"] = torch.tensor(lens + left, dtype=torch.int32, device="cuda")
    st["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
    st["drop"] = torch.tensor([0] * n + [ALL] * kids, dtype=torch.int32, device="cuda")
    st["counts"] = torch.tensor([0] * n + [case["new"]] * kids, dtype=torch.int32, device="cuda")
    st["total"] = kids * case["new"]
    return st


def _compact_layout(case):
    """(lengths, pages that pairs of sequences share at their start)."""
    _, lens = _lengths(case)
    page = case["page"]
    shared = [min(case["share"] // page, lens[b] // page, lens[b + 1] // page) if b % 2 == 0 and b + 1 < len(lens)
              else 0 for b in range(len(lens))]
    return lens, shared


def _compact_state(case, gen):
    lens, shared = _compact_layout(case)
    page, pages = case["page"], case["pages"]
    order = _order(case, pages, gen)
    table = torch.full((len(lens), max(1, max(-(-x // page) for x in lens))), -1, dtype=torch.int32)
    for b, x in enumerate(lens):
        m = -(-x // page)
        same = shared[b - 1] if b % 2 else 0
        mine, order = order[:m - same], order[m - same:]
        table[b, :m] = torch.cat([table[b - 1, :same], torch.tensor(mine, dtype=torch.int32)])
    refs = torch.zeros(pages, dtype=torch.int32)
    refs.scatter_add_(0, table[table >= 0].long(), torch.ones(int((table >= 0).sum()), dtype=torch.int32))
    st = _new_pool(case, pages)
    _fill(st, gen)
    st["table"], st["refs"] = table.to("cuda"), refs.to("cuda")
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    live = int((refs > 0).sum())
    st["out"] = _new_pool(case, max(1, live))
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    if kind == "attend":
        st = _attend_state(case, gen)
    elif kind == "branch":
        st = _branch_state(case, gen)
    elif kind == "compact":
        st = _compact_state(case, gen)
    elif kind == "copy":
        st = _new_pool(case, case["pages"])
        _fill(st, gen)
        order = _order(case, case["pages"], gen)
        n = case["count"]
        st["src"] = torch.tensor(order[:n], dtype=torch.int32, device="cuda")
        st["dst"] = torch.tensor(order[n:2 * n], dtype=torch.int32, device="cuda")
        st["rows"] = None
        if case["part"]:
            st["rows"] = torch.randint(0, case["page"] + 1, (n,), device="cuda", generator=gen, dtype=torch.int32)
    else:
        n, h, page = case["tokens"], case["heads"], case["page"]
        rows = torch.randn((n, 2 * h, D), device="cuda", generator=gen)
        rows[..., 5::41] += 20.0
        rows = rows.to(TORCH[case["dtype"]])
        need = -(-n // page)
        order = torch.tensor(_order(case, need + 2, gen)[:need], device="cuda")
        i = torch.arange(n, device="cuda")
        st = _new_pool(case, need + 2)
        st["K"], st["V"] = rows[:, :h], rows[:, h:]
        st["slots"] = order[i // page] * page + i % page
        st["table"] = order.to(torch.int32).view(1, need)
        st["lens"] = torch.tensor([n], dtype=torch.int32, device="cuda")
        if case["rot"]:
            st["freq"], st["axis"], st["counts"] = _frequencies(case)
            st["freq_gpu"] = st["freq"].to("cuda")
            st["axis_gpu"] = torch.tensor(st["axis"], device="cuda")
            st["pos"] = _positions(case, n, gen)
    st["case"] = case
    return st


# ---------------------------------------------------------------- the plain forms

def _rotate(x, st):
    """x [n][heads][128] in 32 bits, turned; angles in 64 bits (positions reach the millions)."""
    case = st["case"]
    rot = case["rot"]
    angle = st["pos"][st["axis_gpu"]].T.to(torch.float64) * st["freq_gpu"]
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _get(st, name):
    """[seq][heads][tokens][128] in 32 bits of pool `name` by the page tables."""
    table = st["table"].long().clamp(min=0)
    x = _values(st[name].view(torch.uint8)[table], st[name + "_group"].view(torch.uint8)[table].view(torch.float8_e4m3fn),
                st[name + "_scale"][table], st["case"]["fmt"])
    return x.transpose(1, 2).flatten(2, 3)


def _plain_store(st):
    case, n = st["case"], st["case"]["tokens"]
    page = case["page"]
    at, row = st["slots"] // page, st["slots"] % page
    for name, x in (("k", st["K"].float()), ("v", st["V"].float())):
        if name == "k" and case["rot"]:
            x = _rotate(x, st)
        codes, t, scale = _codes(x, case["fmt"])
        st[name].view(torch.uint8)[at, :, row] = codes
        st[name + "_group"].view(torch.uint8)[at, :, row] = t.view(torch.uint8)
        st[name + "_scale"][at, :, row] = scale
    both = torch.stack([_get(st, "k"), _get(st, "v")], 2)[:, :, :, :n]
    seen = torch.arange(n, device="cuda") < st["lens"][:, None]
    return torch.where(seen[:, None, None, :, None], both, 0.0).to(TORCH[case["out"]]).flatten(1, 2)


def _plain_attend(st):
    case = st["case"]
    Q, lens, cu = st["Q"], st["lens"].long(), st["cu_q"].long()
    heads, group, n_seq = case["heads"], case["q_heads"] // case["heads"], case["seqs"]
    mq = st["max_q"]
    k, v = _get(st, "k"), _get(st, "v")
    n = k.shape[2]
    key = torch.arange(n, device="cuda")
    i = torch.arange(mq, device="cuda")
    rows = (cu[:-1, None] + i).clamp(max=Q.shape[0] - 1)
    qp = Q[rows].float().view(n_seq, mq, heads, group, D).permute(0, 2, 3, 1, 4)
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + i  # position of each query in its sequence
    seen = (key < lens[:, None])[:, None, :].expand(n_seq, mq, n)
    if case["causal"]:
        seen = seen & (key <= pos[..., None])
    if case["window"]:
        seen = seen & (key > pos[..., None] - case["window"])
    v = torch.where((key < lens[:, None])[:, None, :, None], v, 0.0)
    s = (qp.flatten(2, 3) @ k.transpose(2, 3)).view(n_seq, heads, group, mq, n).mul_(D ** -0.5)
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(n_seq, heads, group, mq, D) / torch.where(total > 0, total, 1.0)
    r = torch.arange(Q.shape[0], device="cuda")
    b = torch.searchsorted(cu, r, right=True) - 1
    at = r - cu[b]
    out = {"out": o.permute(0, 3, 1, 2, 4)[b, at].flatten(1, 2).to(Q.dtype)}
    if case["lse"]:
        out["lse"] = (top + total.log())[..., 0].permute(0, 3, 1, 2)[b, at].flatten(1, 2)
    return out


def _copy_rows(pools, src, dst, rows, page, to=None):
    """Rows below rows[i] (all of them without) of pages src[i] to pages dst[i]."""
    live = None if rows is None else torch.arange(page, device="cuda") < rows[:, None]
    for x, y in zip(pools, pools if to is None else to):
        if live is None:
            y[dst] = x[src]
        else:
            mask = live[:, None, :] if x.dim() == 3 else live[:, None, :, None]
            y[dst] = torch.where(mask, x[src], y[dst])


def _plain_copy(st):
    _copy_rows(_raw(st), st["src"].long(), st["dst"].long(), st["rows"], st["case"]["page"])
    return _raw(st)


def _plain_branch(st):
    page = st["case"]["page"]
    table, refs, lens = st["table"], st["refs"], st["lens"]
    rows, top = table.shape
    entry = torch.arange(top, device="cuda")

    def held():
        return entry < ((lens + page - 1) // page)[:, None]

    def count(mask, by):
        refs.scatter_add_(0, table.clamp(min=0).long().flatten(), (by * mask.int()).flatten())
    # the continuations' pages are given back
    gone = (st["drop"] > 0)[:, None] & held()
    count(gone, -1)
    table.masked_fill_(gone, -1)
    lens.masked_fill_(st["drop"] > 0, 0)
    # they begin again with their prompts' pages; the part-filled one is copied
    free = torch.sort((refs > 0).int(), stable=True).indices
    kid = st["parents"] >= 0
    p = st["parents"].clamp(min=0).long()
    full, rest = lens[p] // page, lens[p] % page
    lens.copy_(torch.where(kid, lens[p], lens))
    table.copy_(torch.where(kid[:, None] & (entry < full[:, None]), table[p], table))
    need = (kid & (rest > 0)).int()
    fresh = free[(need.cumsum(0) - need).long()]
    own_page = kid[:, None] & (rest > 0)[:, None] & (entry == full[:, None])
    last = table[p, full.clamp(max=top - 1).long()]
    table.copy_(torch.where(own_page, fresh[:, None].int(), table))
    count(kid[:, None] & held(), 1)
    _copy_rows(_raw(st), last.clamp(min=0).long()[need.bool()], fresh[need.bool()], rest[need.bool()], page)
    # and get pages for their new tokens
    free = torch.sort((refs > 0).int(), stable=True).indices
    counts = st["counts"]
    have = (lens + page - 1) // page
    more = (lens + counts + page - 1) // page - have
    first = more.cumsum(0) - more
    new = (entry >= have[:, None]) & (entry < (have + more)[:, None])
    rank = (first[:, None] + entry - have[:, None]).clamp(min=0, max=refs.shape[0] - 1)
    table.copy_(torch.where(new, free[rank.long()].int(), table))
    count(new, 1)
    row = torch.repeat_interleave(torch.arange(rows, device="cuda"), counts, output_size=st["total"])
    start = (counts.cumsum(0) - counts)[row]
    pos = lens[row].long() + torch.arange(st["total"], device="cuda") - start
    slots = table[row, pos // page].long() * page + pos % page
    lens.add_(counts)
    return {"pools": _raw(st), "table": table, "refs": refs, "lens": lens, "slots": slots, "positions": pos}


def _plain_compact(st):
    case, refs, table = st["case"], st["refs"], st["table"]
    live = refs > 0
    place = (live.cumsum(0) - 1).int()
    page = case["page"]
    held = torch.arange(table.shape[1], device="cuda") < ((st["lens"] + page - 1) // page)[:, None]
    new_table = torch.where(held, place[table.clamp(min=0).long()], -1)
    old = live.nonzero()[:, 0]
    out_refs = torch.zeros(st["out"]["k"].shape[0], dtype=torch.int32, device="cuda")
    out_refs[:old.shape[0]] = refs[old]
    _copy_rows(_raw(st), old, torch.arange(old.shape[0], device="cuda"), None, page, _raw(st["out"]))
    return {"pools": _raw(st["out"]), "table": new_table, "refs": out_refs, "live": live.sum().int().view(1)}


def _plain(st):
    return {"store": _plain_store, "attend": _plain_attend, "copy": _plain_copy, "branch": _plain_branch,
            "compact": _plain_compact}[st["case"]["kind"]](st)


# ---------------------------------------------------------------- the library's calls

def _handles(st):
    """What a program makes once and keeps: the caches' descriptions and the rotary table."""
    from video_kv_cache_gb300 import api
    if "handles" not in st:
        rope = to = None
        if st["case"].get("rot", 0):
            rope = api.rope_table(st["case"]["rot"], freqs=st["freq"], sections=st["counts"],
                                  interleaved=st["case"]["layout"] == "interleaved", device="cuda")
        kv = api.PagedKV(*(st[x] for x in POOLS))
        if "out" in st:
            to = api.PagedKV(*(st["out"][x] for x in POOLS))
        st["handles"] = (api, kv, rope, to)
    return st["handles"]


def _own(st):
    api, kv, rope, to = _handles(st)
    case, kind = st["case"], st["case"]["kind"]
    if kind == "store":
        api.page_write(kv, st["K"], st["V"], st["slots"], rope=rope, positions=st.get("pos"))
        return api.page_read(kv, st["table"], st["lens"], case["tokens"], out_dtype=TORCH[case["out"]])
    if kind == "attend":
        got = api.page_attention(st["Q"], kv, st["table"], st["lens"], cu_q=st["cu_q"], max_q=st["max_q"],
                                 max_kv=st["max_kv"], causal=case["causal"], window=case["window"],
                                 return_lse=case["lse"])
        return {"out": got[0], "lse": got[1]} if case["lse"] else {"out": got}
    if kind == "copy":
        api.page_copy(kv, st["src"], st["dst"], rows=st["rows"])
        return _raw(st)
    table, refs, lens = st["table"], st["refs"], st["lens"]
    if kind == "branch":
        api.page_free(kv, refs, table, lens, last=st["drop"])
        api.page_fork(kv, refs, table, lens, st["parents"])
        slots, positions = api.page_append(kv, refs, table, lens, st["counts"], st["total"])
        return {"pools": _raw(st), "table": table, "refs": refs, "lens": lens, "slots": slots, "positions": positions}
    new_table, new_refs, live = api.page_compact(kv, refs, table, lens, to)
    return {"pools": _raw(st["out"]), "table": new_table, "refs": new_refs, "live": live}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def _visible(case):
    """(visible query-key pairs, keys that some query sees) over the sequences, one head."""
    pairs = keys = 0
    for nq, n in zip(*_lengths(case)):
        if not nq:
            continue
        last = [n - nq + i if case["causal"] else n - 1 for i in range(nq)]
        first = [max(0, n - nq + i - case["window"] + 1) if case["window"] else 0 for i in range(nq)]
        pairs += sum(b - a + 1 for a, b in zip(first, last))
        keys += last[-1] + 1 - first[0]
    return pairs, keys


def work(case):
    kind, row = case["kind"], 2 * case["heads"] * ROW[case["fmt"]]  # bytes of a token's keys and values
    page = case["page"]
    if kind == "store":
        n, wide = case["tokens"], 2 * case["heads"] * D
        return {"bytes": n * (wide * NBYTES[case["dtype"]] + row + 8 + (8 * case["axes"] if case["rot"] else 0)
                              + wide * NBYTES[case["out"]]),
                "flops": 4 * n * wide}
    if kind == "copy":  # half a page on average where only a part is copied
        tokens = case["count"] * page // (2 if case["part"] else 1)
        return {"bytes": 2 * tokens * row + 8 * case["count"], "flops": 0}
    if kind == "branch":
        lens, parents = _branch_layout(case)
        moved = entries = 0
        for b, p in enumerate(parents):
            if p >= 0:
                moved += lens[p] % page * row
                entries += -(-(lens[p] + case["new"]) // page)
        kids = len(parents) - case["prompts"]
        # a table entry read, written and counted
        return {"bytes": 2 * moved + 16 * entries + 16 * kids * case["new"] + 20 * len(parents), "flops": 0}
    if kind == "compact":
        lens, shared = _compact_layout(case)
        entries = sum(-(-x // page) for x in lens)
        live = entries - sum(shared)
        return {"bytes": 2 * live * page * row + 8 * entries + 4 * case["pages"] + 4 * live, "flops": 0}
    q, kv = _lengths(case)
    pairs, keys = _visible(case)
    return {"bytes": 2 * sum(q) * case["q_heads"] * D * NBYTES[case["dtype"]] + keys * row
            + (4 * sum(q) * case["q_heads"] if case["lse"] else 0),
            "flops": 4 * D * pairs * case["q_heads"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_turn(x, st):
    """Each pair as a complex number times exp(i angle), in 64 bits."""
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    x = x.double().clone()
    turn = torch.stack([st["pos"][a].double() * float(f) for a, f in zip(st["axis"], st["freq"])], -1)
    w = torch.polar(torch.ones_like(turn), turn)
    for p in range(half):
        i, j = (p, p + half) if case["layout"] == "half" else (2 * p, 2 * p + 1)
        z = torch.complex(x[:, :, i], x[:, :, j]) * w[:, p, None]
        x[:, :, i], x[:, :, j] = z.real, z.imag
    return x


def _nearest(y, bits, lowest):
    """y to `bits` bits after the leading one, steps of `lowest` at least, ties to even."""
    step = torch.exp2(torch.frexp(y).exponent.double() - 1 - bits).clamp(min=lowest)
    return torch.round(y / step) * step


def _exact_store(st):
    case, n = st["case"], st["case"]["tokens"]
    out = torch.zeros((1, 2 * case["heads"], n, D), dtype=torch.float64, device="cuda")
    top = TOP[case["fmt"]]
    for which, x in enumerate((st["K"], st["V"])):
        x = _exact_turn(x, st) if which == 0 and case["rot"] else x.double()
        a = x.abs().amax(-1, keepdim=True)
        for c in range(0, D, GROUP):
            g = x[..., c:c + GROUP]
            t = _nearest(64 * g.abs().amax(-1, keepdim=True) / a, 3, 2.0 ** -9)  # E4M3
            y = torch.where(t > 0, g * (64 * top) / (a * t), 0.0)
            y = torch.round(y) if case["fmt"] == "int4" else _nearest(y, 1, 0.5)
            value = (a / (64 * top)) * t * y.clamp(-top, top)
            out[0, which::2, :, c:c + GROUP] = value.transpose(0, 1)
    return out


def _exact_rows(st, name, b):
    """[heads][tokens][128] of sequence b in 64 bits."""
    case, n = st["case"], int(st["lens"][b])
    ids = st["table"][b, : -(-n // case["page"])].long()
    raw = st[name].view(torch.uint8)[ids]
    x = torch.zeros((*raw.shape[:3], D), dtype=torch.float64, device="cuda")
    numbers = [float(v) for v in list(E2M1) + [-v for v in E2M1]] if case["fmt"] == "e2m1" else \
        [float(v - 16 * (v > 7)) for v in range(16)]
    lookup = torch.tensor(numbers, dtype=torch.float64, device="cuda")
    x[..., 0::2], x[..., 1::2] = lookup[(raw % 16).long()], lookup[(raw // 16).long()]
    t = st[name + "_group"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
    x = x * t.repeat_interleave(GROUP, -1) * st[name + "_scale"][ids].double()[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_attend(st):
    case = st["case"]
    group = case["q_heads"] // case["heads"]
    out = torch.zeros(st["Q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["Q"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    for b, (nq, n) in enumerate(zip(*_lengths(case))):
        if not nq:
            continue
        first = int(st["cu_q"][b])
        k, v = _exact_rows(st, "k", b), _exact_rows(st, "v", b)
        key = torch.arange(n, device="cuda")
        for r0 in range(0, nq, 2048):
            r1 = min(nq, r0 + 2048)
            pos = torch.arange(n - nq + r0, n - nq + r1, device="cuda")[:, None]
            hidden = torch.zeros((r1 - r0, n), dtype=torch.bool, device="cuda")
            if case["causal"]:
                hidden |= key > pos
            if case["window"]:
                hidden |= key <= pos - case["window"]
            for h in range(case["q_heads"]):
                s = st["Q"][first + r0:first + r1, h].double() @ k[h // group].T / math.sqrt(D)
                s = s.masked_fill_(hidden, float("-inf"))
                z = torch.logsumexp(s, -1)
                out[first + r0:first + r1, h] = (s - z[:, None]).exp_().nan_to_num_(0.0) @ v[h // group]
                lse[first + r0:first + r1, h] = z
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_branch(st):
    """Sequence by sequence, with lists."""
    case, page = st["case"], st["case"]["page"]
    lens, parents = _branch_layout(case)
    rows, top = st["table"].shape
    held = [st["table"][b, : -(-lens[b] // page)].tolist() if p < 0 else [] for b, p in enumerate(parents)]
    size = [lens[b] if p < 0 else 0 for b, p in enumerate(parents)]
    users = [0] * st["refs"].shape[0]
    for row in held:
        for x in row:
            users[x] += 1
    pools = [x.clone() for x in _raw(st)]

    def take():
        x = users.index(0)
        users[x] = 1
        return x
    for b, p in enumerate(parents):
        if p < 0:
            continue
        full, rest = size[p] // page, size[p] % page
        held[b], size[b] = held[p][:full], size[p]
        for x in held[b]:
            users[x] += 1
        if rest:
            held[b].append(take())
            for pool in pools:
                pool[held[b][-1], :, :rest] = pool[held[p][full], :, :rest]
    slots, positions = [], []
    for b, p in enumerate(parents):
        for _ in range(case["new"] if p >= 0 else 0):
            if size[b] % page == 0:
                held[b].append(take())
            slots.append(held[b][-1] * page + size[b] % page)
            positions.append(size[b])
            size[b] += 1

    def on_gpu(x, dtype):
        return torch.tensor(x, dtype=dtype, device="cuda")
    return {"pools": pools, "table": on_gpu([row + [-1] * (top - len(row)) for row in held], torch.int32),
            "refs": on_gpu(users, torch.int32), "lens": on_gpu(size, torch.int32),
            "slots": on_gpu(slots, torch.int64), "positions": on_gpu(positions, torch.int64)}


def _exact_compact(st):
    page = st["case"]["page"]
    lens, _ = _compact_layout(st["case"])
    table = st["table"].tolist()
    names = sorted({x for row, n in zip(table, lens) for x in row[: -(-n // page)]})
    new = {x: i for i, x in enumerate(names)}
    rows = [[new[x] for x in row[: -(-n // page)]] + [-1] * (len(row) - -(-n // page)) for row, n in zip(table, lens)]
    users = [0] * st["out"]["k"].shape[0]
    for row in rows:
        for x in row:
            if x >= 0:
                users[x] += 1
    pools = []
    for x, y in zip(_raw(st), _raw(st["out"])):
        y = y.clone()
        y[:len(names)] = x[torch.tensor(names, dtype=torch.int64, device="cuda")]
        pools.append(y)
    return {"pools": pools, "table": torch.tensor(rows, dtype=torch.int32, device="cuda"),
            "refs": torch.tensor(users, dtype=torch.int32, device="cuda"),
            "live": torch.tensor([len(names)], dtype=torch.int32, device="cuda")}


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "store":
        return _exact_store(st)
    if kind == "attend":
        return _exact_attend(st)
    if kind == "branch":
        return _exact_branch(st)
    if kind == "compact":
        return _exact_compact(st)
    pools = [x.clone() for x in _raw(st)]
    rows = st["rows"].tolist() if case["part"] else [case["page"]] * case["count"]
    for i, (a, b) in enumerate(zip(st["src"].tolist(), st["dst"].tolist())):
        for pool, old in zip(pools, _raw(st)):
            pool[b, :, :rows[i]] = old[a, :, :rows[i]]
    return pools
