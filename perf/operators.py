"""Measured cases of the paged-cache operators: rotary positions, writing and reading a paged
K/V cache (16-bit or 8-bit with a scale per token and head), and the attention of new tokens
over it.

``run`` computes an operator in its plain form, in elementary torch operations, or (``own``)
through the library's public calls.  Sizes follow the repository's workloads: 12 and 32 heads
of 128 channels, chunks of 3 x 30 x 52 = 4680 tokens, 32760 and 280800 cached tokens, frames of
64 x 64 tokens; and generic ones for grouped heads and single-token decoding.
"""
import math
import random

import torch

own = False

D = 128
CHUNK_GRID = (30, 52)  # rows and columns of a frame of the 1.3B-class shape
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
NBYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "int8": 1}
TOP = {"e4m3": 448.0, "int8": 127.0}  # largest code of the 8-bit formats


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of eight sequences, far positions of a stretched context, part of the head
        dict(name="rope_decode", kind="rope", tokens=8, heads=32, dtype="fp16", layout="half",
             rot=64, axes=1, base=1e6, scaling="by_parts", factor=16.0, far=1000000, backward=False),
        # the queries of one 4680-token chunk, (frame, row, column) positions, fused QKV rows
        dict(name="rope_chunk_video", kind="rope", tokens=4680, heads=12, dtype="bf16",
             layout="interleaved", rot=128, axes=3, base=1e4, scaling="none", factor=1.0, far=60,
             backward=False),
        # the gradient of a long training sequence's queries
        dict(name="rope_long_backward", kind="rope", tokens=65536, heads=32, dtype="bf16",
             layout="half", rot=128, axes=1, base=1e4, scaling="linear", factor=4.0, far=65536,
             backward=True),
        # one new token of 61 sequences, rotated and written in 8 bits
        dict(name="write_decode_e4m3", kind="write", tokens=61, heads=8, dtype="bf16", fmt="e4m3",
             page=16, layout="half", rot=128, axes=1, far=100000),
        # a chunk of video tokens, rotated on three axes and written in 8 bits
        dict(name="write_chunk_e4m3", kind="write", tokens=4680, heads=12, dtype="bf16", fmt="e4m3",
             page=64, layout="interleaved", rot=128, axes=3, far=60),
        # seven chunks written in 8-bit integers (keys before rotation) and read back for compression
        dict(name="store_window_int8", kind="store", tokens=32760, heads=12, dtype="bf16", fmt="int8",
             page=64, layout="none", rot=0, axes=1, far=0, out="bf16"),
        # a layer's whole stream read back
        dict(name="read_stream_e4m3", kind="read", seqs=1, len_lo=280800, len_hi=280800, lens_seed=0,
             heads=12, fmt="e4m3", page=128, out="bf16"),
        # one new token of eight short sequences: latency
        dict(name="decode_small", kind="attend", seqs=8, q_lo=1, q_hi=1, len_lo=100, len_hi=2000,
             lens_seed=1, q_heads=32, heads=8, dtype="bf16", fmt="bf16", page=16, causal=True,
             window=0, lse=False),
        # one new token of 32 long sequences over an 8-bit cache
        dict(name="decode_long_int8", kind="attend", seqs=32, q_lo=1, q_hi=1, len_lo=9000,
             len_hi=20000, lens_seed=2, q_heads=32, heads=8, dtype="bf16", fmt="int8", page=64,
             causal=True, window=0, lse=True),
        # ragged prompts with what is cached before them, grouped heads, a sliding window
        dict(name="prefill_ragged_window", kind="attend", seqs=6, q_lo=17, q_hi=2000, len_lo=500,
             len_hi=9000, lens_seed=3, q_heads=32, heads=8, dtype="fp16", fmt="fp16", page=32,
             causal=True, window=4096, lse=True),
        # a video chunk over the seven chunks of its history: every query sees every key
        dict(name="chunk_over_history", kind="attend", seqs=1, q_lo=4680, q_hi=4680, len_lo=32760,
             len_hi=32760, lens_seed=0, q_heads=12, heads=12, dtype="bf16", fmt="bf16", page=64,
             causal=False, window=0, lse=False),
        # a 64 x 64 frame over eight of them in 8 bits, causal
        dict(name="frame_over_e4m3", kind="attend", seqs=1, q_lo=4096, q_hi=4096, len_lo=32768,
             len_hi=32768, lens_seed=0, q_heads=32, heads=32, dtype="bf16", fmt="e4m3", page=128,
             causal=True, window=0, lse=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "write", "store", "read", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "rope":
        axes = rng.choice([1, 1, 3])
        heads = _log_int(rng, 1, 48)
        return dict(kind=kind, tokens=_log_int(rng, 1, max(2, 65536 * 32 // (heads * 2))), heads=heads,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    layout=rng.choice(["half", "interleaved"]), rot=rng.choice([32, 64, 96, 128]),
                    axes=axes, base=rng.choice([1e4, 5e5, 1e6]),
                    scaling=rng.choice(["none", "linear", "stretched", "by_parts"]),
                    factor=rng.choice([2.0, 8.0, 32.0]), far=_log_int(rng, 10, 2000000),
                    backward=rng.random() < 0.5)
    if kind in ("write", "store"):
        heads = _log_int(rng, 1, 32)
        layout = rng.choice(["none", "half", "interleaved"])
        case = dict(kind=kind, tokens=_log_int(rng, 1, 32760 * 12 // heads), heads=heads,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    fmt=rng.choice(["e4m3", "bf16", "fp16"] if kind == "write" else ["e4m3", "int8", "fp16"]),
                    page=rng.choice([16, 32, 64, 128]), layout=layout,
                    rot=0 if layout == "none" else rng.choice([32, 64, 128]),
                    axes=rng.choice([1, 3]), far=_log_int(rng, 10, 1000000))
        return dict(case, out=rng.choice(["bf16", "fp16"])) if kind == "store" else case
    if kind == "read":
        heads, seqs = _log_int(rng, 1, 32), _log_int(rng, 1, 16)
        top = _log_int(rng, 1, max(2, 240000 * 10 // (heads * seqs)))
        return dict(kind=kind, seqs=seqs, len_lo=rng.choice([0, top // 2]), len_hi=top,
                    lens_seed=rng.randrange(1 << 30), heads=heads,
                    fmt=rng.choice(["bf16", "fp16", "e4m3", "int8"]), page=rng.choice([16, 32, 64, 128]),
                    out=rng.choice(["bf16", "fp16", "fp32"]))
    heads = rng.choice([1, 2, 4, 8, 12])
    q_heads = heads * rng.choice([1, 1, 2, 4, 7, 8])
    decode = rng.random() < 0.4
    if decode:
        seqs, q_hi = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 5])
        len_hi = _log_int(rng, 8, max(16, 5000000 // (seqs * heads)))
    else:
        seqs, q_hi = _log_int(rng, 1, 12), _log_int(rng, 2, 4096)
        len_hi = _log_int(rng, q_hi, max(q_hi + 1, 2000000000 // (seqs * q_heads * q_hi)))
    len_hi = min(len_hi, 130000)
    q_hi = min(q_hi, len_hi)
    return dict(kind=kind, seqs=seqs, q_lo=q_hi if decode else rng.choice([0, 1, q_hi]), q_hi=q_hi,
                len_lo=rng.choice([0, len_hi // 2, len_hi]), len_hi=len_hi,
                lens_seed=rng.randrange(1 << 30), q_heads=q_heads, heads=heads, dtype=dtype,
                fmt=rng.choice([dtype, "e4m3", "int8"]), page=rng.choice([16, 32, 64, 128]),
                causal=rng.random() < 0.6, window=rng.choice([0, 0, 1 + len_hi // 3]),
                lse=rng.random() < 0.5)


def _lengths(case):
    """(query tokens, cached tokens) of each sequence, the same for every seed of the inputs."""
    r = random.Random(case["lens_seed"])
    kv = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    q = [min(r.randint(case["q_lo"], case["q_hi"]), n) if "q_lo" in case else 0 for n in kv]
    if "q_lo" in case and sum(q) == 0:
        q[0], kv[0] = max(1, case["q_lo"]), max(kv[0], 1, case["q_lo"])
    return q, kv


# ---------------------------------------------------------------- inputs

def _frequencies(case):
    """(angle per position of each pair in radians, axis of each pair, factor on the rotated part)."""
    half, axes, base = case["rot"] // 2, case["axes"], case.get("base", 1e4)
    scaling, factor = case.get("scaling", "none"), case.get("factor", 1.0)
    counts = [half] if axes == 1 else [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    if scaling == "stretched":  # a larger base, so that the slowest pair turns `factor` times slower
        base = base * factor ** (half / (half - 1.0))
    freq, axis = [], []
    for a, n in enumerate(counts):
        freq += [base ** (-i / n) for i in range(n)]
        axis += [a] * n
    if scaling == "linear":
        freq = [f / factor for f in freq]
    mscale = 1.0
    if scaling == "by_parts":
        # fast pairs (over 32 turns in 4096 positions) as they are, slow ones (under 1) divided
        # by the factor, a linear ramp over the number of turns between (YaRN, arXiv 2309.00071)
        keep = [min(1.0, max(0.0, (4096 * f / (2 * math.pi) - 1.0) / 31.0)) for f in freq]
        freq = [f * k + f / factor * (1 - k) for f, k in zip(freq, keep)]
        mscale = 0.1 * math.log(factor) + 1.0
    return torch.tensor(freq, dtype=torch.float64), axis, counts, mscale


def _positions(case, n, gen):
    """int64 [axes][n]: grid positions of a video chunk, or far positions of separate tokens."""
    start = int(torch.randint(0, max(1, case["far"]), (1,), generator=torch.Generator().manual_seed(gen.initial_seed())))
    i = torch.arange(n, device="cuda")
    if case["axes"] == 3:
        h, w = CHUNK_GRID
        return torch.stack([start + i // (h * w), i // w % h, i % w])
    if n <= 256:
        return torch.randint(0, max(1, case["far"]), (1, n), device="cuda", generator=gen)
    return (start + i).view(1, n)


def _kv_rows(n, heads, width, dtype, gen):
    """Rows of a fused projection [n][width][128] with a few outlier channels, as keys have."""
    x = torch.randn((n, width, D), device="cuda", generator=gen, dtype=torch.float32)
    x[..., 5::41] += 20.0
    return x.to(dtype)


def _pool(case, gen):
    """Pages [pages][heads][page][128] of K and of V with their scales, page tables and lengths;
    what no sequence reaches holds NaN, as memory that nobody wrote may."""
    q, kv = _lengths(case)
    page, heads, fmt = case["page"], case["heads"], TORCH[case["fmt"]]
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 3
    cpu = torch.Generator().manual_seed(gen.initial_seed())
    order = torch.randperm(pages, generator=cpu).tolist()
    table = torch.full((len(kv), max(1, max(need))), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[sum(need[:b]):sum(need[:b]) + n], dtype=torch.int32)
    token = torch.full((pages, page), False)  # written rows
    for b, n in enumerate(kv):
        rows = token.new_zeros(need[b] * page)
        rows[:n] = True
        token[table[b, :need[b]].long()] = rows.view(need[b], page)
    token = token.to("cuda")[:, None, :]
    out = {}
    for name in ("k", "v"):
        x = torch.randn((pages, heads, page, D), device="cuda", generator=gen)
        if case["fmt"] in TOP:
            amax = x.abs().amax(-1)
            codes = x * (TOP[case["fmt"]] / amax)[..., None]
            codes = codes.round().to(fmt) if case["fmt"] == "int8" else codes.to(fmt)
            out[name] = codes
            out[name + "_scale"] = torch.where(token, amax / TOP[case["fmt"]], float("nan"))
        else:
            out[name] = torch.where(token[..., None], x, float("nan")).to(fmt)
            out[name + "_scale"] = None
    out["table"] = table.to("cuda")
    out["lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    kind = case["kind"]
    if case.get("rot", 0):
        st["freq"], st["axis"], st["counts"], st["mscale"] = _frequencies(case)
        st["freq_gpu"] = st["freq"].to("cuda")
        st["axis_gpu"] = torch.tensor(st["axis"], device="cuda")
    if kind == "rope":
        n, h = case["tokens"], case["heads"]
        width = 3 * h if case["axes"] == 3 else h  # a fused projection's rows, or its own tensor
        st["x"] = torch.randn((n, width, D), device="cuda", generator=gen).to(TORCH[case["dtype"]])[:, :h]
        st["pos"] = _positions(case, n, gen)
    elif kind in ("write", "store"):
        n, h, page = case["tokens"], case["heads"], case["page"]
        rows = _kv_rows(n, h, 2 * h, TORCH[case["dtype"]], gen)
        st["K"], st["V"] = rows[:, :h], rows[:, h:]
        pages = -(-n // page) + 2
        need = -(-n // page)
        order = torch.randperm(pages, device="cuda", generator=gen)[:need]
        i = torch.arange(n, device="cuda")
        st["slots"] = order[i // page] * page + i % page
        if n <= 256 and kind == "write":  # separate sequences: anywhere in the pool
            pages = n + 2
            st["slots"] = (torch.randperm(pages, device="cuda", generator=gen)[:n] * page +
                           torch.randint(0, page, (n,), device="cuda", generator=gen))
        for name in ("k", "v"):
            st[name] = torch.zeros((pages, h, page, D), device="cuda", dtype=TORCH[case["fmt"]])
            st[name + "_scale"] = (torch.zeros((pages, h, page), device="cuda")
                                   if case["fmt"] in TOP else None)
        st["table"] = order.to(torch.int32).view(1, need)
        st["lens"] = torch.tensor([n], dtype=torch.int32, device="cuda")
        if case["rot"]:
            st["pos"] = _positions(case, n, gen)
    else:
        st.update(_pool(case, gen))
        if kind == "attend":
            q, kv = _lengths(case)
            st["cu_q"] = torch.tensor([sum(q[:b]) for b in range(len(q) + 1)], dtype=torch.int32, device="cuda")
            st["max_q"], st["max_kv"], st["total_q"] = max(q), max(kv), sum(q)
            st["Q"] = (1.5 * torch.randn((sum(q), case["q_heads"], D), device="cuda", generator=gen)).to(TORCH[case["dtype"]])
        else:
            st["count"] = max(1, case["len_hi"])
    return st


# ---------------------------------------------------------------- the plain forms

def _rotate(x, st, backward=False):
    """x [n][heads][128] in 32 bits, rotated; angles in 64 bits (positions reach the millions)."""
    case = st["case"]
    rot = case["rot"]
    angle = st["pos"][st["axis_gpu"]].T.to(torch.float64) * st["freq_gpu"]
    c = (angle.cos() * st["mscale"]).float()[:, None, :]
    s = (angle.sin() * (-st["mscale"] if backward else st["mscale"])).float()[:, None, :]
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _put(st, name, x):
    """Rows x [n][heads][128] in 32 bits into the pool `name` at the slots."""
    case, pool = st["case"], st[name]
    page = case["page"]
    at, row = st["slots"] // page, st["slots"] % page
    if case["fmt"] not in TOP:
        pool[at, :, row] = x.to(pool.dtype)
        return
    top = TOP[case["fmt"]]
    amax = x.abs().amax(-1)
    y = x * torch.where(amax > 0, top / amax, 0.0)[..., None]
    codes = y.round().to(torch.int8) if case["fmt"] == "int8" else y.to(torch.float8_e4m3fn)
    pool.view(torch.uint8)[at, :, row] = codes.view(torch.uint8)
    st[name + "_scale"][at, :, row] = amax / top


def _get(st, name, pages):
    """[seq][heads][tokens][128] in 32 bits of pool `name` by the page tables."""
    table = st["table"][:, :pages].long().clamp(min=0)
    x = st[name][table].float()
    if st[name + "_scale"] is not None:
        x = x * st[name + "_scale"][table][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_read(st, count, out):
    page = st["case"]["page"]
    pages = min(st["table"].shape[1], -(-count // page))
    both = torch.stack([_get(st, "k", pages), _get(st, "v", pages)], 2)[:, :, :, :count]
    seen = torch.arange(both.shape[3], device="cuda") < st["lens"][:, None]
    both = torch.where(seen[:, None, None, :, None], both, 0.0).to(out)
    return torch.nn.functional.pad(both, (0, 0, 0, count - both.shape[3])).flatten(1, 2)


def _plain_attend(st):
    case = st["case"]
    Q, lens, cu = st["Q"], st["lens"].long(), st["cu_q"].long()
    heads, group, n_seq = case["heads"], case["q_heads"] // case["heads"], case["seqs"]
    mq = st["max_q"]
    k, v = _get(st, "k", st["table"].shape[1]), _get(st, "v", st["table"].shape[1])
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


def _pools(st):
    return [st[x] for x in ("k", "v", "k_scale", "v_scale") if st[x] is not None]


def _plain(st):
    case, kind = st["case"], st["case"]["kind"]
    if kind == "rope":
        return _rotate(st["x"].float(), st, case["backward"]).to(st["x"].dtype)
    if kind in ("write", "store"):
        K = st["K"].float()
        _put(st, "k", _rotate(K, st) if case["rot"] else K)
        _put(st, "v", st["V"].float())
        return _pools(st) if kind == "write" else _plain_read(st, case["tokens"], TORCH[case["out"]])
    if kind == "read":
        return _plain_read(st, st["count"], TORCH[case["out"]])
    return _plain_attend(st)


# ---------------------------------------------------------------- the library's calls

def _handles(st):
    """What a program makes once and keeps: the cache's description and the rotary table."""
    from video_kv_cache_gb300 import api
    if "handles" not in st:
        table = kv = None
        if st["case"].get("rot", 0):
            table = api.rope_table(st["case"]["rot"], freqs=st["freq"], sections=st["counts"],
                                   interleaved=st["case"]["layout"] == "interleaved",
                                   mscale=st["mscale"], device="cuda")
        if "k" in st:
            kv = api.PagedKV(st["k"], st["v"], st["k_scale"], st["v_scale"])
        st["handles"] = (api, table, kv)
    return st["handles"]


def _own(st):
    api, rope, kv = _handles(st)
    case, kind = st["case"], st["case"]["kind"]
    if kind == "rope":
        return api.rope(st["x"], st["pos"], rope, backward=case["backward"])
    if kind in ("write", "store"):
        api.page_write(kv, st["K"], st["V"], st["slots"], rope=rope, positions=st.get("pos"))
        if kind == "write":
            return _pools(st)
        return api.page_read(kv, st["table"], st["lens"], case["tokens"], out_dtype=TORCH[case["out"]])
    if kind == "read":
        return api.page_read(kv, st["table"], st["lens"], st["count"], out_dtype=TORCH[case["out"]])
    got = api.page_attention(st["Q"], kv, st["table"], st["lens"], cu_q=st["cu_q"], max_q=st["max_q"],
                             max_kv=st["max_kv"], causal=case["causal"], window=case["window"],
                             return_lse=case["lse"])
    return {"out": got[0], "lse": got[1]} if case["lse"] else {"out": got}


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
    kind = case["kind"]
    if kind == "rope":
        rows = case["tokens"] * case["heads"]
        return {"bytes": 2 * rows * D * NBYTES[case["dtype"]] + 8 * case["tokens"] * case["axes"],
                "flops": 3 * rows * case["rot"]}
    row = D * NBYTES[case["fmt"]] + (4 if case["fmt"] in TOP else 0)
    if kind in ("write", "store"):
        rows = 2 * case["tokens"] * case["heads"]
        moved = rows * (D * NBYTES[case["dtype"]] + row) + 8 * case["tokens"]
        if case["rot"]:
            moved += 8 * case["tokens"] * case["axes"]
        if kind == "store":
            moved += rows * D * NBYTES[case["out"]]
        return {"bytes": moved, "flops": 3 * rows * D}
    q, kv = _lengths(case)
    if kind == "read":
        wide = 2 * case["heads"] * D * NBYTES[case["out"]]
        return {"bytes": 2 * case["heads"] * sum(kv) * row + case["seqs"] * max(1, case["len_hi"]) * wide,
                "flops": 2 * case["heads"] * sum(kv) * D}
    pairs, keys = _visible(case)
    return {"bytes": 2 * sum(q) * case["q_heads"] * D * NBYTES[case["dtype"]] + 2 * keys * case["heads"] * row
            + (4 * sum(q) * case["q_heads"] if case["lse"] else 0),
            "flops": 4 * D * pairs * case["q_heads"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rotate(x, st, backward):
    """Each pair as a complex number times exp(i angle), in 64 bits."""
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    x = x.double().clone()
    turn = torch.stack([st["pos"][a].double() * float(f) for a, f in zip(st["axis"], st["freq"])], -1)
    w = torch.polar(torch.full_like(turn, st["mscale"]), -turn if backward else turn)
    for p in range(half):
        i, j = (p, p + half) if case["layout"] == "half" else (2 * p, 2 * p + 1)
        z = torch.complex(x[:, :, i], x[:, :, j]) * w[:, p, None]
        x[:, :, i], x[:, :, j] = z.real, z.imag
    return x


def _exact_codes(x, fmt):
    """(codes as 64-bit values, scale) of rows of one 8-bit format."""
    top = TOP[fmt]
    scale = x.abs().amax(-1) / top
    y = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    step = torch.ones_like(y)
    if fmt == "e4m3":  # three bits after the leading one, down to steps of 2^-9
        step = torch.exp2(torch.frexp(y).exponent.double() - 1 - 3).clamp(min=2.0 ** -9)
    return (torch.round(y / step) * step).clamp(-top, top), scale


def _exact_store(st):
    """Values and scales of the pools after the write, in 64 bits."""
    case, pools = st["case"], {}
    for name, x in (("k", st["K"]), ("v", st["V"])):
        x = _exact_rotate(x, st, False) if name == "k" and case["rot"] else x.double()
        pool = st[name].double()
        at, row = st["slots"] // case["page"], st["slots"] % case["page"]
        if case["fmt"] in TOP:
            codes, scale = _exact_codes(x, case["fmt"])
            scales = st[name + "_scale"].double()
            pool[at, :, row], scales[at, :, row] = codes, scale
            pools[name + "_scale"] = scales
        else:
            pool[at, :, row] = x
        pools[name] = pool
    return pools


def _exact_rows(st, pools, name, b):
    """[heads][tokens][128] of sequence b in 64 bits."""
    n = int(st["lens"][b])
    page = st["case"]["page"]
    ids = st["table"][b, : -(-n // page)].long()
    x = pools[name][ids].double()
    if pools.get(name + "_scale") is not None:
        x = x * pools[name + "_scale"][ids].double()[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_read(st, pools, count):
    case = st["case"]
    out = torch.zeros((len(st["lens"]), 2 * case["heads"], count, D), dtype=torch.float64, device="cuda")
    for b in range(len(st["lens"])):
        for which, name in enumerate(("k", "v")):
            x = _exact_rows(st, pools, name, b)[:, :count]
            out[b, which::2, : x.shape[1]] = x
    return out


def _exact_attend(st):
    case = st["case"]
    group = case["q_heads"] // case["heads"]
    out = torch.zeros(st["Q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["Q"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    for b, (nq, n) in enumerate(zip(*_lengths(case))):
        if not nq:
            continue
        first = int(st["cu_q"][b])
        k, v = _exact_rows(st, st, "k", b), _exact_rows(st, st, "v", b)
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


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return _exact_rotate(st["x"], st, case["backward"])
    if kind in ("write", "store"):
        pools = _exact_store(st)
        if kind == "store":
            return _exact_read(st, pools, case["tokens"])
        return [pools[x] for x in ("k", "v", "k_scale", "v_scale") if x in pools]
    if kind == "read":
        return _exact_read(st, st, st["count"])
    return _exact_attend(st)
