"""A stream of video chunks through the paged cache and into the compressed one.

Each chunk's queries and keys are turned by their (frame, row, column) positions; keys and
values go into pages, rounded to the pages' format as they are written; the chunk's queries
attend to the pages: every token of the chunk to all of it and to the chunks kept before it.
Once more than ``window`` chunks are cached, the oldest is read back, compressed by k-means
(qvg_quantize, warm-started from the chunk before), and its pages serve the next chunk.

    python examples/paged_stream.py                 # 12 heads, chunks of 3 x 32 x 48 tokens
    python examples/paged_stream.py --format bf16 --window 2

Inputs are seeded random numbers in the place of a model's projections.
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass, field

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from video_kv_cache_gb300 import api

FORMATS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@dataclass
class Stream:
    """One layer's caches: the pages of the recent chunks, in order, and what was compressed."""
    heads: int
    grid: tuple                 # (frames of a chunk, rows, columns)
    window: int                 # chunks kept in pages beside the newest
    chunks: int                 # most chunks of the stream
    pages: api.PagedKV = None
    rope: api.RopeTable = None
    compressed: api.CompressedKV = None
    table: list = field(default_factory=list)   # pages of the cached tokens, oldest first
    free: list = field(default_factory=list)
    done: int = 0               # chunks seen
    packed: int = 0             # chunks compressed

    @property
    def chunk(self):
        return self.grid[0] * self.grid[1] * self.grid[2]


def make_stream(heads=12, grid=(3, 32, 48), window=3, chunks=8, fmt="e4m3", page=64, C=256,
                device="cuda") -> Stream:
    s = Stream(heads, grid, window, chunks)
    if s.chunk % page:
        raise ValueError("a chunk's %d tokens must fill whole pages of %d" % (s.chunk, page))
    n = (window + 1) * s.chunk // page
    s.pages = api.allocate_pages(n, heads, page, FORMATS[fmt], device)
    s.free = list(range(n))
    s.rope = api.rope_table(128, sections=(22, 21, 21), interleaved=True, device=device)
    s.compressed = api.allocate(2 * heads, chunks * s.chunk, min(C, s.chunk), 2, 2, 32, chunks, device)
    return s


def positions(s: Stream, device) -> torch.Tensor:
    """(frame, row, column) of every token of the next chunk."""
    f, h, w = s.grid
    i = torch.arange(s.chunk, device=device)
    return torch.stack([s.done * f + i // (h * w), i // w % h, i % w])


def step(s: Stream, Q, K, V) -> torch.Tensor:
    """Attention output of the next chunk, Q, K, V [chunk][heads][128]."""
    dev, page, n = Q.device, s.pages.page_tokens, s.chunk // s.pages.page_tokens
    if len(s.table) == (s.window + 1) * n:
        pack_oldest(s)
    new = [s.free.pop() for _ in range(n)]
    s.table += new
    slots = (torch.tensor(new, device=dev)[:, None] * page + torch.arange(page, device=dev)).flatten()
    pos = positions(s, dev)
    Q = api.rope(Q, pos, s.rope)
    api.page_write(s.pages, K, V, slots, rope=s.rope, positions=pos)
    s.done += 1
    table = torch.tensor([s.table], dtype=torch.int32, device=dev)
    lens = torch.tensor([len(s.table) * page], dtype=torch.int32, device=dev)
    return api.page_attention(Q, s.pages, table, lens, causal=False)


def pack_oldest(s: Stream) -> None:
    """Compress the oldest cached chunk and give its pages back."""
    dev, n = s.pages.k.device, s.chunk // s.pages.page_tokens
    table = torch.tensor([s.table[:n]], dtype=torch.int32, device=dev)
    lens = torch.tensor([s.chunk], dtype=torch.int32, device=dev)
    X = api.page_read(s.pages, table, lens, s.chunk)[0]  # [2 * heads][chunk][128]
    c = s.compressed
    warm = dict(warm=c.centroids[:, s.packed - 1], warm_stride=c.centroids.stride(0)) if s.packed else {}
    api.quantize(X, c.C, c.T, c.bits, c.group, iters=2 if s.packed else 10, seed=1, out=c,
                 token_offset=s.packed * s.chunk, table_index=s.packed, **warm)
    s.free += s.table[:n]
    s.table = s.table[n:]
    s.packed += 1


def inputs(s: Stream, seed: int, device):
    g = torch.Generator(device=device).manual_seed(seed)
    rows = torch.randn((s.chunk, 3 * s.heads, 128), generator=g, device=device).to(torch.bfloat16)
    return rows[:, :s.heads], rows[:, s.heads:2 * s.heads], rows[:, 2 * s.heads:]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--heads", type=int, default=12)
    ap.add_argument("--grid", type=int, nargs=3, default=(3, 32, 48), metavar=("FRAMES", "ROWS", "COLS"))
    ap.add_argument("--window", type=int, default=3)
    ap.add_argument("--chunks", type=int, default=8)
    ap.add_argument("--format", default="e4m3", choices=sorted(FORMATS))
    a = ap.parse_args()
    s = make_stream(a.heads, tuple(a.grid), a.window, a.chunks, a.format)
    for k in range(a.chunks):
        x = inputs(s, k, "cuda")
        torch.cuda.synchronize()
        t = time.perf_counter()
        out = step(s, *x)
        torch.cuda.synchronize()
        print("chunk %d: %d tokens attend to %d, %d chunks compressed, %.2f ms, |out| %.4f"
              % (k, s.chunk, len(s.table) * s.pages.page_tokens, s.packed,
                 (time.perf_counter() - t) * 1e3, float(out.float().abs().mean())))
    print("pages hold %.1f MB, the compressed cache %.1f MB"
          % (s.pages.nbytes() / 1e6, s.compressed.nbytes() / 1e6))


if __name__ == "__main__":
    main()
