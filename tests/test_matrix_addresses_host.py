"""Every address that the pipelined weight gradients' loads form, replayed on
the host from the kernels' formulas (k_ckpt8_wgrad.hip): no load passes its
matrix, and no offset is negative or as large as a descriptor's reach.  Buffer
addressing takes a negative 32-bit offset for one of 2^31 to 2^32, which a
descriptor without an end lets through."""
import random

import numpy as np
import pytest

import matrix_plan as plan
from matrix_ref import up

ST = 32
REACH = 0x7FFFFFFF
LANE = np.arange(64)


def check_load(first, off, size, total, esize, what):
    """Loads of `size` elements at offset `off` from element `first` of a matrix of `total`."""
    assert (off >= 0).all(), ("negative", what)
    assert ((off + size) * esize <= REACH).all(), ("past the descriptor", what)
    assert first >= 0 and (first + off + size <= total).all(), ("past the matrix", what)


def check_x(t0, rows, t, d0, piece, pitch, epitch, what):
    codes, exps = np.minimum(d0 + piece * 16, pitch - 16), np.minimum((d0 + piece * 16) // 128 * 4, epitch - 4)
    check_load(t0 * pitch, t * pitch + codes, 16, rows * pitch, 1, what)
    check_load(t0 * epitch, t * epitch + exps, 4, rows * epitch, 1, what)


def bf16_loads(rows, n, dim, ldy, tile, per, from_tile=False):
    """k_ckpt8_wgrad_pipe.  from_tile: offsets count from the tile's first column (they do not)."""
    waves = 4 if tile == 128 else 8
    pitch, epitch, row_bytes = up(dim, 32), up(dim, 128) // 32, tile * 2
    loads, tokens_wave = ST * row_bytes // 1024 // waves, 1024 // tile
    for t_first in range(0, rows, per):
        tokens = min(rows - t_first, per)
        stages, whole = -(-tokens // (2 * ST)) * 2, tokens // ST
        last_piece = (n - 1) // 8 * 8
        patch = t_first + tokens == rows and n % 8 != 0
        fast = {s + u + 3 for s in range(0, max(whole - 7, 0), 4) for u in range(4)}  # batches loaded by the main loop
        for batch in range(stages):
            t0 = batch * ST if batch in fast else min(batch * ST, tokens - 1)
            for n0 in range(0, n, tile):
                for i in range(waves * loads):
                    tok = i * (1024 // row_bytes) + LANE // (row_bytes // 16)
                    col = np.minimum(n0 + ((LANE % (row_bytes // 16)) ^ (2 * (tok & 7))) * 8, last_piece)
                    if batch not in fast:
                        last = min(tokens - 1 - t0, ST)
                        tok = np.minimum(tok, last)
                        col = np.where(patch & (tok == last) & (col == last_piece), n - 8, col)
                    base = n0 if from_tile else 0
                    check_load((t_first + t0) * ldy + base, tok * ldy + col - base, 8,
                               (rows - 1) * ldy + n, 2, ("dY", t_first, batch, n0))
        for stage in range(stages + 1):
            quick = stage - 1 in fast
            t0 = stage * ST if quick else min(stage * ST, tokens - 1)
            for w in range(waves):
                t = w * tokens_wave + LANE // (tile // 16)
                if not quick:
                    t = np.minimum(t, min(tokens - 1 - t0, ST))
                for d0 in range(0, dim, tile):
                    what = ("X", t_first, stage, d0)
                    check_x(t_first + t0, rows, t, d0, LANE % (tile // 16), pitch, epitch, what)


def f32_loads(rows, n, dim, ldy, tile, per):
    """k_ckpt8_wgrad_pipe_f32."""
    pitch, epitch = up(dim, 32), up(dim, 128) // 32
    tokens_wave, waves = 1024 // tile, 8
    for t_first in range(0, rows, per):
        tokens = min(rows - t_first, per)
        stages = -(-tokens // ST)
        fast = {s + u + 4 for s in range(0, max(stages - 6, 0), 2) for u in range(2)}
        last_piece = (n - 1) // 4 * 4
        for stage in range(stages):
            t0, have = stage * ST, min(tokens - stage * ST, ST)
            assert have == ST or stage not in fast
            for n0 in range(0, n, 128):
                col = np.minimum(n0 + (LANE & 31) * 4, last_piece)
                over = np.maximum(col + 4 - n, 0)
                for i in range(waves * 2):
                    t = i * 2 + (LANE >> 5)
                    if stage in fast:
                        off = t * ldy + col
                    else:
                        t = np.minimum(t, have - 1)
                        off = t * ldy + col - np.where(t_first + t0 + t == rows - 1, over, 0)
                    check_load((t_first + t0) * ldy, off, 4, (rows - 1) * ldy + n, 4, ("dY", t_first, stage, n0))
            for w in range(waves):
                t = np.minimum(w % (ST // tokens_wave) * tokens_wave + LANE // (tile // 16), have - 1)
                for d0 in range(0, dim, tile):
                    what = ("X", t_first, stage, d0)
                    check_x(t_first + t0, rows, t, d0, LANE % (tile // 16), pitch, epitch, what)


def sizes():
    r = random.Random(1)
    out = [(1, 8, 1), (1, 9, 33), (31, 15, 31), (33, 8, 160), (64, 130, 127), (65, 513, 70), (97, 255, 300)]
    for _ in range(25):
        rows = r.choice([1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 97, r.randint(1, 900)])
        out.append((rows, r.randint(8, 600), r.randint(1, 400)))
    return out


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_loads_stay_inside(bf16):
    for rows, n, dim in sizes() + ([] if bf16 else [(70, 4, 40), (1, 5, 40), (33, 6, 40), (300, 7, 40)]):
        for ldy in (n, n + 1, n + 5, up(n, 8)):
            for per in {64, up(rows, 64), up(-(-rows // 2), 64), plan.wgrad(rows, n, dim, bf16)[3]}:
                for tile in (128, 256):
                    (bf16_loads if bf16 else f32_loads)(rows, n, dim, ldy, tile, per)


def test_loads_of_long_splits():
    """The main loops' loads, in splits of more than one turn."""
    for rows, n, dim in ((704, 13, 40), (1000, 141, 300), (640, 16, 129), (999, 9, 33)):
        for per in (384, up(rows, 64)):
            for tile in (128, 256):
                bf16_loads(rows, n, dim, n + 1, tile, per)
                f32_loads(rows, n, dim, n + 1, tile, per)


def test_largest_strides_stay_in_reach():
    """Rows at their limit of 2^23 elements apart."""
    bf16_loads(100, 20, 40, 1 << 23, 128, 128)
    f32_loads(100, 20, 40, 1 << 23, 256, 128)


def test_offsets_counted_from_the_tile_are_caught():
    """Planted: offsets that count from the tile's first column and not from
    column 0 are negative where a tile's first piece is the last row's short one."""
    with pytest.raises(AssertionError, match="negative"):
        bf16_loads(65, 129, 40, 129, 128, 128, True)
