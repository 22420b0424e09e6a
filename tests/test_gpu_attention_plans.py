"""qmm_paged_attention in each way that the host lays a call out: whole items,
pieces of few items, and equal runs over many; one and several chunks of
columns; up to 64 sequences and more. Each case says which one it takes, and the
workspace that the library asks for confirms it."""
import numpy as np
import pytest
import torch

from tests import _gpu
from tests.test_gpu_paged_attention import Problem

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def layout(B, Hkv, G, D, max_rows, max_context, window=0, sinks=0):
    """("whole" | "pieces" | "runs", chunks, column tiles), from the workspace's bytes:
    [items] pairs of numbers, rounded to 16, and for each run two partial results
    of 16 * tiles columns with D + 2 floats."""
    tiles = -(-max_rows * G // 16)
    most = {64: 6, 96: 4, 128: 6, 192: 3, 256: 3}[D]
    chunks = -(-tiles // most)
    per = -(-tiles // chunks)
    per += per == 5
    chunks = -(-tiles // per)
    items = B * Hkv * chunks
    size = _gpu.lib().qmm_paged_attention_workspace_bytes(max(B * max_rows, 1), B, Hkv * G, Hkv, D, max_rows, max_context,
                                                          window, sinks)
    if size == 0:
        return "whole", chunks, per
    runs, rest = divmod(size - (items * 8 + 15) // 16 * 16, 2 * 16 * per * (D + 2) * 4)
    assert rest == 0 and runs > 0
    return "pieces" if items * 4 <= runs else "runs", chunks, per


def ragged(B, most, seed, none=(), empty=()):
    """Lengths of B sequences up to `most`; those in `empty` have none."""
    lens = np.random.default_rng(seed).integers(1, most + 1, B)
    lens[0] = most
    lens[list(empty)] = 0
    return lens.tolist()


# (sequences, kv heads, group, head, rows, longest, page, window, sinks), layout
CASES = [
    # up to 64 sequences and one chunk: mostly runs, which walk from head to head and sequence to sequence
    ((40, 4, 6, 256, 1, 300, 16, 0, 0), ("runs", 1, 1)),
    ((64, 4, 6, 128, 1, 300, 16, 0, 0), ("runs", 1, 1)),
    ((64, 8, 2, 64, 1, 400, 24, 0, 0), ("runs", 1, 1)),
    ((50, 4, 3, 96, 2, 330, 16, 0, 0), ("runs", 1, 1)),
    ((40, 3, 2, 192, 3, 420, 17, 0, 0), ("runs", 1, 1)),
    ((30, 4, 8, 128, 8, 300, 16, 0, 0), ("pieces", 1, 4)),
    ((40, 4, 8, 128, 8, 300, 16, 0, 0), ("runs", 1, 4)),
    ((30, 6, 8, 64, 8, 300, 32, 0, 0), ("pieces", 1, 4)),
    ((40, 6, 8, 64, 8, 300, 32, 0, 0), ("runs", 1, 4)),
    ((30, 6, 8, 96, 8, 300, 16, 0, 0), ("runs", 1, 4)),
    ((35, 2, 6, 256, 8, 700, 64, 0, 0), ("runs", 1, 3)),
    ((35, 2, 10, 128, 8, 500, 16, 0, 0), ("runs", 1, 6)),
    ((40, 4, 6, 256, 3, 700, 16, 300, 4), ("runs", 1, 2)),
    ((60, 8, 4, 64, 2, 900, 48, 390, 5), ("runs", 1, 1)),
    # more than 64 sequences: the plan reads the lengths again
    ((70, 4, 6, 128, 1, 300, 16, 0, 0), ("runs", 1, 1)),
    ((130, 2, 6, 128, 1, 300, 16, 0, 0), ("runs", 1, 1)),
    ((65, 2, 4, 256, 3, 300, 32, 0, 0), ("runs", 1, 1)),
    ((200, 2, 3, 192, 1, 280, 16, 0, 0), ("runs", 1, 1)),
    ((130, 2, 2, 256, 2, 700, 16, 260, 3), ("runs", 1, 1)),
    # several chunks of columns
    ((20, 2, 12, 128, 16, 300, 16, 0, 0), ("runs", 2, 6)),
    ((10, 2, 12, 256, 16, 300, 16, 0, 0), ("runs", 4, 3)),
    ((66, 1, 12, 128, 16, 300, 16, 0, 0), ("runs", 2, 6)),
    ((10, 2, 12, 256, 16, 800, 16, 300, 4), ("runs", 4, 3)),
    ((12, 2, 12, 192, 16, 300, 33, 0, 0), ("runs", 4, 3)),
    ((16, 4, 12, 96, 16, 300, 16, 0, 0), ("runs", 3, 4)),
    # pieces of few items
    ((2, 1, 12, 128, 16, 2000, 16, 0, 0), ("pieces", 2, 6)),
    ((2, 2, 12, 256, 16, 2000, 64, 0, 0), ("pieces", 4, 3)),
    ((3, 2, 6, 96, 2, 1500, 16, 0, 0), ("pieces", 1, 1)),
    ((3, 2, 6, 192, 5, 1500, 17, 0, 0), ("pieces", 1, 2)),
    ((2, 2, 8, 128, 8, 1500, 16, 0, 0), ("pieces", 1, 4)),
    ((2, 2, 8, 64, 8, 1500, 16, 0, 0), ("pieces", 1, 4)),
    ((3, 1, 4, 256, 2, 3000, 64, 1000, 4), ("pieces", 1, 1)),
    ((65, 1, 4, 128, 1, 700, 16, 0, 0), ("pieces", 1, 1)),
    ((130, 1, 4, 64, 1, 700, 16, 0, 0), ("pieces", 1, 1)),
    ((65, 1, 12, 64, 16, 700, 16, 0, 0), ("pieces", 2, 6)),
    # whole items, with several chunks and more sequences too
    ((3, 2, 6, 256, 40, 250, 16, 0, 0), ("whole", 5, 3)),
    ((70, 2, 3, 128, 40, 200, 16, 0, 0), ("whole", 2, 4)),
    ((130, 8, 2, 128, 1, 600, 16, 0, 0), ("whole", 1, 1)),
]


@pytest.mark.parametrize("shape,want", CASES, ids=str)
def test_layouts(shape, want):
    B, Hkv, G, D, rows, longest, page, window, sinks = shape
    assert layout(B, Hkv, G, D, rows, longest, window, sinks) == want
    rng = np.random.default_rng(B + D)
    empty = [B // 2, B - 1] if B > 4 else []
    lens = ragged(B, longest, B, empty=empty)
    n = rng.integers(0 if B > 4 else 1, rows + 1, B)  # sequences without rows among them
    n[0] = rows
    n = np.where(n > np.maximum(lens, 1), 1, n).tolist()
    p = Problem(lens, n, Hkv, G, D, page, BF16 if (B + D // 32) % 2 else F16, seed=B, q_scale=1.5)
    out, lse = p.check(window, sinks, max_context=longest, max_rows=rows)
    # again, and with the estimate of the longest context wrong either way
    again, again_lse = p.run(window, sinks, max_context=longest, max_rows=rows)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    if window == 0:
        p.check(max_context=257, max_rows=rows)
        p.check(max_context=4 * longest, max_rows=rows)


@pytest.mark.parametrize("D", [128, 192, 256])
@pytest.mark.parametrize("max_context", [1, 400])
def test_lengths_around_tiles_of_128(D, max_context):
    lens = [126, 127, 128, 129, 130, 255, 256, 257, 383, 384, 385]
    for rows, G in ((1, 2), (2, 3), (8, 12) if D == 128 else (8, 6)):
        Problem(lens, [min(rows, 1 + i % rows) for i in range(11)], 1, G, D, 16, BF16, seed=D + rows).check(
            max_context=max_context, max_rows=rows)


@pytest.mark.parametrize("D", [192, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (127, 0), (128, 1), (129, 130), (200, 3)])
@pytest.mark.parametrize("max_context", [1, 900])
def test_windows_of_wide_heads(D, window, sinks, max_context):
    Problem([5, 128, 300, 640, 900], [2, 1, 3, 2, 3], 2, 2, D, 24, F16, seed=window).check(window, sinks,
                                                                                         max_context=max_context)
