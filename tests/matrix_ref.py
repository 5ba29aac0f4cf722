"""Plain 64-bit forms of the matrix operators (INT8 rows and their product,
8-bit checkpoints, the weight gradient taken from them, the gated
activation), on the host, and input matrices where they can go wrong."""
import numpy as np
import torch

GROUP = 32
EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step


def up(v, unit):
    return -(-v // unit) * unit


def int8_rows(x):
    """(codes int8, scale fp32) of a [rows][dim] host tensor."""
    x = x.double().numpy()
    bad = ~np.isfinite(x).all(1)
    amax = np.abs(np.where(np.isfinite(x), x, 0.0)).max(1)
    # the double quotient of an fp32 number by 127, rounded once more to fp32,
    # is the correctly rounded one (53 >= 2 * 24 + 2 bits)
    scale = (amax / 127.0).astype(np.float32)
    s = scale.astype(np.float64)[:, None]
    q = np.clip(np.rint(np.where(s > 0, x / np.where(s > 0, s, 1.0), 0.0)), -127, 127)
    q[bad] = 0
    scale[bad] = np.nan
    return q.astype(np.int8), scale


def matmul(a, sa, b, sb):
    s = a.astype(np.int64) @ b.astype(np.int64).T
    return s.astype(np.float64) * sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None, :]


def ckpt8(x):
    """(codes int8 [rows][pitch], exps uint8 [rows][epitch]) of a host tensor."""
    x = x.double().numpy()
    rows, dim = x.shape
    codes = np.zeros((rows, up(dim, GROUP)), np.int8)
    exps = np.zeros((rows, up(dim, 4 * GROUP) // GROUP), np.uint8)
    for g in range(-(-dim // GROUP)):
        part = x[:, g * GROUP: min(dim, (g + 1) * GROUP)]
        bad = ~np.isfinite(part).all(1)
        amax = np.abs(np.where(np.isfinite(part), part, 0.0)).max(1)
        e = np.full(rows, -126)
        for cand in range(-126, 122):  # the smallest that holds amax (121 at most)
            e = np.where((amax > 127.0 * 2.0 ** (cand - 1)) & (cand > -126), cand, e)
        q = np.clip(np.rint(part * (2.0 ** -e.astype(np.float64))[:, None]), -127, 127)
        q[bad] = 0
        codes[:, g * GROUP: g * GROUP + part.shape[1]] = q
        exps[:, g] = np.where(bad, 255, e + 127)
    return codes, exps


def held(codes, exps, dim):
    """What a checkpoint stands for, in 64 bits."""
    rows = codes.shape[0]
    step = np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - 127))
    step = np.repeat(step, GROUP, 1)[:, : codes.shape[1]]
    return (codes.astype(np.float64) * step)[:, :dim].reshape(rows, dim)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def matrix(rows, dim, seed, dtype, spread=1.0):
    """Seeded activations: channels and tokens of different size."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, dim), generator=g)
    x = x * torch.exp(spread * torch.randn((1, dim), generator=g)) * torch.exp(0.5 * torch.randn((rows, 1), generator=g))
    return x.to(dtype)


def hard_rows(dim, dtype):
    """Rows where a row's or group's statistic or rounding can go wrong."""
    fmax = torch.finfo(dtype).max
    tiny = 2.0 ** -133 if dtype is torch.bfloat16 else 2.0 ** -149
    k = torch.arange(dim, dtype=torch.float64)
    rows = [
        torch.zeros(dim, dtype=torch.float64),
        -torch.zeros(dim, dtype=torch.float64),
        (k % 255) - 127,                                    # whole steps
        ((k % 254) - 127) + 0.5,                            # half steps of the checkpoint: ties
        ((k % 509) - 254) / 2 * 2.0 ** -100,
        torch.where(k == dim - 1, fmax, 0.0),               # one huge value, last
        torch.full((dim,), fmax),
        torch.full((dim,), -fmax),
        torch.full((dim,), tiny),                           # the smallest subnormal
        torch.where(k % 3 == 0, 190 * tiny, -tiny),
        ((k % 37) - 18) * 2.0 ** -126,                      # around the smallest normal
        torch.where(k % 32 == 0, 1.984375, 0.25),           # 127 steps of 2^-6 exactly
        torch.where(k % 32 == 0, 1.9921875, 0.25),          # just above
        torch.where(k % 64 == 0, 1e30, 1e-30),
        torch.where(k == 0, torch.inf, 1.0),
        torch.where(k == dim - 1, -torch.inf, 1.0),
        torch.where(k == dim // 2, torch.nan, 3.0),
        torch.full((dim,), torch.nan),
    ]
    return torch.stack(rows).to(torch.float32).to(dtype)
