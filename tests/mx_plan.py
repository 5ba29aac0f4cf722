"""Which tile and how many parts of k the MXFP4 product takes for given sizes:
the choice of k_matmul_mxfp4.hip (choose) with the constants read from its
table, so that tests can say which sizes reach which path."""
import os
import re

import numpy as np

FILE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "embedding_communication_codecs_amd",
                    "csrc", "k_matmul_mxfp4.hip")
with open(FILE) as f:
    TEXT = f.read()
# the kernel holds them as fp32
SHAPES = [[float(np.float32(v)) for v in re.findall(r"[0-9.]+(?=f?\b)", row)] for row in re.findall(
    r"\{([^{}]*)\}", re.search(r"constexpr Shape kShapes\[\] = \{(.*?)\};", TEXT, re.S).group(1))]
FIRST_PIPE = int(re.search(r"kFirstPipe = (\d+)", TEXT).group(1))
MAX_SPLITS, LEAST_STAGES = (int(re.search(rf"{n} = (\d+)", TEXT).group(1)) for n in ("kMaxSplits", "kLeastStages"))
FEW = int(re.search(r"kFew = (\d+)", TEXT).group(1))
# stages of codes in LDS, of the pipelined tiles by their number
BUFFERS = {int(i): int(nb) for i, nb in re.findall(r"case (\d): return launch_pipe<T, ADD, [\d, ]*, (\d)>", TEXT)}
BUFFERS[len(SHAPES) - 1] = int(re.search(r"default: return launch_pipe<T, ADD, [\d, ]*, (\d)>", TEXT).group(1))


def product(m, n, k):
    """(number of the tile shape, parts of k, stages of a part)."""
    stages = -(-(-(-k // 32) * 16) // 128)
    best, least = (len(SHAPES) - 1, 1, stages), 1e300
    for i, (bn, bm, first, first_k, more, more_k) in enumerate(SHAPES):
        blocks = -(-n // int(bn)) * -(-m // int(bm))
        if blocks >= 1 << 23:
            continue
        splits = 1
        while splits <= (MAX_SPLITS if i >= FIRST_PIPE else 1):
            each = -(-stages // splits)
            if splits > 1 and (each < LEAST_STAGES or blocks * splits > 512):
                break
            parts = -(-stages // each)
            kk = float(k) if splits == 1 else each * 256.0
            us = first + first_k * kk / 1024.0 + (blocks * parts - 1) // 256 * (more + more_k * kk / 1024.0)
            if parts > 1:
                us += 2.5 + m * n * 4.0 * 2 * parts / 4e6
            if us < least:
                best, least = (i, parts, each), us
            splits *= 2
    return best


def fast_turns(k, shape, stages=None):
    """How often the pipelined kernel's loop over whole stages runs, in its first part."""
    nb = BUFFERS[shape]
    pitch, spitch = -(-k // 32) * 16, -(-k // 128) * 4
    length = min(pitch, (stages or 1 << 40) * 128)
    whole = length // 128
    end = min(whole, whole if spitch % 16 == 0 else spitch // 32 * 4 - 4)
    return max(-(-(end - 2 * nb + 1) // nb), 0)
