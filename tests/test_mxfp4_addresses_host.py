"""Every address that the MXFP4 products' loads into LDS form, replayed on the
host with the offsets read from the kernels' source (k_matmul_mxfp4.hip): no
offset is negative, which buffer addressing would take for one past the
descriptor, none reaches past its descriptor, no descriptor past its matrix,
and what is used comes from its place."""
import random
import re

import numpy as np
import pytest

import mx_plan as plan
from matrix_ref import up

LANE = np.arange(64)
REACH = 0x7FFFFFFF
STAGE, CHUNK, SLAB = 128, 4, 256


def struct(name):
    return re.search(rf"struct {name} \{{.*?\n\}};", plan.TEXT, re.S).group(0)


def offsets(name, call):
    """The arguments of each such call in a struct, compiled."""
    text, out = struct(name), []
    for start in re.finditer(rf"{call}\(", text):
        parts, depth, at = [""], 0, start.end()
        while depth >= 0:
            ch = text[at]
            depth += (ch == "(") - (ch == ")")
            if ch == "," and depth == 0:
                parts.append("")
            else:
                parts[-1] += ch
            at += 1
        parts[-1] = parts[-1][:-1]  # the call's own parenthesis
        out.append([compile(" ".join(p.split()), call, "eval") for p in parts])
    return out


CODES = offsets("Loader", "load_lds16")
WHOLE, ANY = (c[2:4] for c in CODES)
(SLAB_CODES,), (SLAB_SCALES,) = ([c[2:4] for c in offsets("SlabLoader", f)] for f in ("load_lds16", "load_lds4"))
(QUICK_SCALES,), (ANY_SCALES,) = ([c[3:4] for c in offsets("ScaleLoader", f)] for f in ("load_lds16_if", "load_lds4_if"))


def value(code, **names):
    return eval(code, {"min": np.minimum, "max": np.maximum, "lane_id": lambda: LANE, "__builtins__": {}}, names)


def check(voff, soff, size, reach, what):
    assert (voff >= 0).all(), ("negative", what)
    assert 0 <= soff <= REACH and reach <= REACH and (voff + soff + size <= reach).all(), ("past the descriptor", what)


def check_place(at, row, pitch, byte, there, what):
    assert (at[there] == (row * pitch + byte)[there]).all(), ("another place", what)


def piece_slot(row, piece):
    return piece ^ ((row >> 1) & 7)


def codes_of_tile(rows, row0, tile, pitch, length, stages, nb, base, total, any_=None):
    """Loader<tile>, `length` bytes of a row from byte `base` of the matrix on."""
    last = min(rows - 1 - row0, tile - 1)
    reach = last * pitch + length
    assert base + reach <= total, "descriptor past the matrix"
    for i in range(tile // 8):
        row = i * 8 + LANE // 8
        piece = piece_slot(row, LANE % 8)
        off = np.minimum(row, last) * pitch + piece * 16
        for s in range(stages + nb):
            names = dict(off=[off], i=0, s=s, kStage=STAGE, len=length, wave=0, piece=lambda *_: piece)
            quick = (s + 1) * STAGE <= length
            for v, w in ([WHOLE] if quick else []) + [any_ or ANY]:
                what = ("codes", rows, row0, tile, pitch, length, s)
                voff, soff = value(v, **names), value(w, **names)
                check(voff, soff, 16, reach, what)
                byte = s * STAGE + piece * 16
                check_place(voff + soff, row, pitch, byte, (row <= last) & (byte < length), what)


def scales_of_tile(rows, row0, tile, pitch, length, stages, nb, quick_stages, base, total):
    """ScaleLoader, `length` bytes of a row."""
    last = min(rows - 1 - row0, tile - 1)
    reach = last * pitch + length
    assert base + reach <= total, "descriptor past the matrix"
    any_ = set(range((CHUNK + nb - 1) // CHUNK + 1)) | {(s + nb) // CHUNK + 1 for s in range(stages)}
    quick = {(s + nb) // CHUNK + 1 for s in range(quick_stages)}
    for first in range(0, tile, 32):
        for c in any_ | quick:
            names = dict(c=c, first=first, last=last, pitch=pitch, len=length)
            what = ("scales", rows, row0, tile, pitch, length, first, c)
            if c in quick:
                r = LANE >> 1
                byte = c * 32 + ((LANE & 1) ^ ((r >> 3) & 1)) * 16
                voff = value(QUICK_SCALES[0], **names, r=r, at=np.minimum(byte, length - 16))
                check(voff, 0, 16, reach, what)
                check_place(voff, first + r, pitch, byte, (first + r <= last) & (byte < length), what)
            for e in range(4):
                slot = e * 16 + (LANE >> 2)
                r = slot >> 1
                at = c * 32 + ((slot & 1) ^ ((r >> 3) & 1)) * 16 + (LANE & 3) * 4
                voff = value(ANY_SCALES[0], **names, r=r, at=at)
                check(voff, 0, 4, reach, what)
                check_place(voff, first + r, pitch, at, (first + r <= last) & (at < length), what)


def pipe_loads(rows, k, tile, shape, splits, any_=None):
    """A side of `rows` rows in tiles of `tile`, k in `splits` parts."""
    pitch, spitch = up(k, 32) // 2, up(k, 128) // 32
    nb, all_stages = plan.BUFFERS[shape], -(-pitch // STAGE)
    each = -(-all_stages // splits)
    for first in range(0, all_stages, each):
        length, slength = min(pitch - first * STAGE, each * STAGE), spitch - first * 8
        stages = -(-length // STAGE)
        whole = length // STAGE
        end = min(whole, whole if slength % 16 == 0 else slength // 32 * CHUNK - CHUNK)
        quick = max(-(-(end - 2 * nb + 1) // nb), 0) * nb
        for row0 in {0, (rows - 1) // tile * tile}:
            codes_of_tile(rows, row0, tile, pitch, length, stages, nb, row0 * pitch + first * STAGE, rows * pitch, any_)
            scales_of_tile(rows, row0, tile, spitch, slength, stages, nb, quick, row0 * spitch + first * 8, rows * spitch)


def slab_loads(rows, k, tile):
    """SlabLoader<tile>"""
    pitch, spitch = up(k, 32) // 2, up(k, 128) // 32
    for row0 in {0, (rows - 1) // tile * tile}:
        last = min(rows - 1 - row0, tile - 1)
        for slab in range(-(-pitch // SLAB)):
            what = ("slab", rows, row0, tile, k, slab)
            for i in range(tile // 4):
                row = i * 4 + LANE // 16
                piece = (LANE % 16) ^ (row & 15)
                off = np.minimum(row, last) * pitch + piece * 16
                names = dict(off=[off], i=0, slab=slab, kSlab=SLAB, pitch=pitch, piece=lambda *_: piece)
                voff, soff = (value(c, **names) for c in SLAB_CODES)
                check(voff, soff, 16, (last + 1) * pitch, what)
                byte = slab * SLAB + piece * 16
                check_place(voff + soff, row, pitch, byte, (row <= last) & (byte < pitch), what)
            for i in range(tile // 16):
                row = i * 16 + LANE // 4
                soffs = np.minimum(row, last) * spitch + LANE % 4 * 4
                names = dict(soff=[soffs], i=0, slab=slab, spitch=spitch)
                voff, soff = (value(c, **names) for c in SLAB_SCALES)
                check(voff, soff, 4, (last + 1) * spitch, what)
                byte = slab * 16 + LANE % 4 * 4
                check_place(voff + soff, row, spitch, byte, (row <= last) & (byte < spitch), what)


def sizes():
    r = random.Random(2)
    out = [(1, 1), (1, 33), (3, 256), (64, 257), (65, 512), (255, 1000), (257, 2043), (300, 96)]
    return out + [(r.randint(1, 600), r.randint(1, 6000)) for _ in range(12)]


@pytest.mark.parametrize("shape", range(plan.FIRST_PIPE, len(plan.SHAPES)))
def test_loads_of_pipelined_tiles_stay_inside(shape):
    for tile in {int(v) for v in plan.SHAPES[shape][:2]}:
        for rows, k in sizes():
            for splits in (1, 2, 8):
                pipe_loads(rows, k, tile, shape, splits)


@pytest.mark.parametrize("tile", [16, 32, 64])
def test_loads_of_few_tokens_stay_inside(tile):
    for rows, k in sizes():
        slab_loads(rows, k, tile)


def test_longest_rows_stay_in_reach():
    """2^23 values: the last stages of the first and the last rows."""
    pitch = 1 << 22
    for tile in (64, 256):
        last = tile - 1
        for i in (0, tile // 8 - 1):
            row = i * 8 + LANE // 8
            piece = piece_slot(row, LANE % 8)
            for s in (pitch // STAGE - 1, pitch // STAGE, pitch // STAGE + 3):
                names = dict(off=[row * pitch + piece * 16], i=0, s=s, kStage=STAGE, len=pitch, wave=0,
                             piece=lambda *_: piece)
                for v, w in [ANY] + ([WHOLE] if s * STAGE < pitch else []):
                    check(value(v, **names), value(w, **names), 16, last * pitch + pitch, ("longest", tile, i, s))


def test_a_stage_beside_the_lane_s_offset_is_caught():
    """Planted: the stage as the wave's offset, what is over taken off the lane's."""
    over = [compile(c, "planted", "eval") for c in
            ("off[i] - max(s * kStage + piece(wave, i, lane_id()) * 16 - (len - 16), 0)", "s * kStage")]
    with pytest.raises(AssertionError, match="negative"):
        pipe_loads(65, 300, 64, plan.FIRST_PIPE, 1, over)
