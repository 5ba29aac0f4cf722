"""Which kernel, tile and splits the matrix operators take for given sizes:
the choices of k_ckpt8_wgrad.hip (plan_of, launch_ckpt8_wgrad) and
k_matmul_int8.hip (shape_of) with the constants read from their tables, so
that tests can say which sizes reach which path."""
import os
import re

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "embedding_communication_codecs_amd",
                    "csrc")


def _table(file, name):
    with open(os.path.join(CSRC, file)) as f:
        body = re.search(r"constexpr Shape %s\[\] = \{(.*?)\};" % name, f.read(), re.S).group(1)
    # the kernels hold them as fp32
    return [[float(np.float32(v)) for v in re.findall(r"[0-9.]+", row)] for row in re.findall(r"\{([^{}]*)\}", body)]


WGRAD = {True: _table("k_ckpt8_wgrad.hip", "kBf16Shapes"), False: _table("k_ckpt8_wgrad.hip", "kF32Shapes")}
PRODUCT = _table("k_matmul_int8.hip", "kShapes")


def wgrad(rows, n, dim, bf16):
    """(kernel, input channels of a tile, splits, tokens of a split)."""
    units = max(-(-rows // 64), 1)
    best, least = None, 0.0
    for bn, bd, slots, stage_us, store_us, alone_us in WGRAD[bf16]:
        tiles = -(-n // int(bn)) * -(-dim // int(bd))
        for want in (1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64):
            if want > units:
                break
            per = -(-units // want)
            splits = -(-units // per)
            blocks = tiles * splits
            us = -(-blocks // int(slots)) * (2.0 * per * (alone_us if blocks <= 256 else stage_us) + store_us)
            if splits > 1:
                us += 2.8 + 0.1 * splits + (splits + 1) * n * dim * (4.0 / 8e6)
            if best is None or us < least:
                least, best = us, (int(bd), splits, per * 64)
    kernel = "simple" if n < (8 if bf16 else 4) else "pipelined"
    return (kernel, 128 if kernel == "simple" else best[0], *best[1:])


def main_loop_turns(rows, n, dim, bf16):
    """How often each split runs the pipelined kernel's loop over whole stages."""
    kernel, _, splits, per = wgrad(rows, n, dim, bf16)
    if kernel == "simple":
        return [0] * splits
    out = []
    for first in range(0, rows, per):
        tokens = min(rows - first, per)
        if bf16:  # four stages a turn while the stages up to s + 7 are whole
            out.append(max(-(-(tokens // 32 - 7) // 4), 0))
        else:  # two while s + 6 is one
            out.append(max(-(-(-(-tokens // 32) - 6) // 2), 0))
    return out


def product(m, n):
    """Number of the tile shape."""
    best, least = len(PRODUCT) - 1, 1e300
    for i, (bn, bm, round_us) in enumerate(PRODUCT):
        blocks = -(-n // int(bn)) * -(-m // int(bm))
        us = -(-blocks // 256) * round_us
        if us < least and blocks < 1 << 23:
            best, least = i, us
    return best
