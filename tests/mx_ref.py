"""Plain 64-bit forms, on the host, of the 4-bit matrix operators (MXFP4 and
its product) and of the AdamW step with its 8-bit states, and inputs where
they can go wrong."""
import numpy as np
import torch

GROUP = 32
BLOCK = 256
U32 = 2.0 ** -24  # half a step of fp32, relative
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MID_ELEM, MID_STEP = 0x91E10DA5, 0xC13FA9A9


def up(v, unit):
    return -(-v // unit) * unit


# ------------------------------------------------------------------ MXFP4


def encode(x):
    """(codes uint8 [rows][pitch], scales uint8 [rows][spitch]) of a host tensor."""
    x = x.double().numpy()
    rows, dim = x.shape
    wide = np.zeros((rows, up(dim, GROUP)), np.uint8)
    scales = np.zeros((rows, up(dim, 4 * GROUP) // GROUP), np.uint8)
    for g in range(-(-dim // GROUP)):
        part = x[:, g * GROUP: min(dim, (g + 1) * GROUP)]
        bad = ~np.isfinite(part).all(1)
        amax = np.abs(np.where(np.isfinite(part), part, 0.0)).max(1)
        # 2^E with the smallest E in [-126, 126] that has amax < 7 * 2^E
        frac, e = np.frexp(amax)
        e = np.clip(np.where(amax == 0, -126, np.where(frac < 0.875, e - 3, e - 2)), -126, 126)
        assert (bad | (amax < 7 * 2.0 ** e)).all() and (bad | (e == -126) | (amax >= 3.5 * 2.0 ** e)).all()
        y = np.abs(np.where(bad[:, None], 0.0, part)) * (2.0 ** -e.astype(np.float64))[:, None]
        low = np.clip(np.searchsorted(VALUES, y, side="right") - 1, 0, 6)  # y in [VALUES[low], VALUES[low + 1])
        below, above = y - VALUES[low], VALUES[low + 1] - y
        code = np.where((above < below) | ((above == below) & (low % 2 == 1)), low + 1, low)
        code = np.where(bad[:, None], 0, code + 8 * np.signbit(part))
        wide[:, g * GROUP: g * GROUP + part.shape[1]] = code
        scales[:, g] = np.where(bad, 255, e + 127)
    return wide[:, 0::2] | (wide[:, 1::2] << 4), scales


def held(codes, scales, dim):
    """What codes and scales stand for, in 64 bits."""
    rows = codes.shape[0]
    wide = np.stack([codes & 15, codes >> 4], 2).reshape(rows, -1)
    v = VALUES[wide & 7] * np.where(wide & 8, -1.0, 1.0)
    step = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * np.repeat(step, GROUP, 1)[:, : v.shape[1]])[:, :dim]


def hard_rows(dim, dtype):
    """Rows where a group's scale or a code's rounding can go wrong."""
    fmax, tiny = torch.finfo(dtype).max, 2.0 ** -133 if dtype is torch.bfloat16 else 2.0 ** -149
    k = torch.arange(dim, dtype=torch.float64)
    ties = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    near = ties * torch.where(k[: 8] == 0, 1.0, 1 + 2.0 ** -7)
    below = ties * torch.where(k[: 8] == 0, 1.0, 1 - 2.0 ** -8) if dim >= 8 else ties
    pick = lambda t: t[(torch.arange(dim) % t.numel())]  # noqa: E731
    rows = [
        torch.zeros(dim, dtype=torch.float64),
        -torch.zeros(dim, dtype=torch.float64),
        pick(ties), -pick(ties), pick(near) if dim >= 8 else pick(ties), pick(below),
        pick(ties) * 2.0 ** -100, pick(ties) * 2.0 ** 100,
        torch.where(k % 32 == 0, 6.96875, 1.0),              # just below 7 steps (bf16 has 6.96875)
        torch.where(k % 32 == 0, 7.0, 1.0),                  # 7 steps: the next power of two
        torch.where(k % 32 == 31, -7.0 * 2.0 ** -40, 2.0 ** -40),
        torch.where(k == dim - 1, fmax, 0.0),
        torch.full((dim,), fmax), torch.full((dim,), -fmax),
        torch.full((dim,), tiny), torch.where(k % 3 == 0, 190 * tiny, -tiny),
        ((k % 37) - 18) * 2.0 ** -126,                       # around the smallest normal
        (k % 13) * 2.0 ** -128,                              # the smallest scale: codes of half steps
        torch.where(k % 64 == 0, 1e30, 1e-30),
        torch.where(k == 0, torch.inf, 1.0),
        torch.where(k == dim - 1, -torch.inf, 1.0),
        torch.where(k == dim // 2, torch.nan, 3.0),
        torch.full((dim,), torch.nan),
    ]
    return torch.stack([r.to(torch.float64) for r in rows]).to(torch.float32).to(dtype)


def random_mx(rows, dim, seed, low=100, high=140):
    """Random codes (zeros past dim) and scale bytes."""
    g = np.random.default_rng(seed)
    wide = g.integers(0, 16, (rows, up(dim, GROUP)), dtype=np.uint8)
    wide[:, dim:] = 0
    scales = g.integers(low, high, (rows, up(dim, 4 * GROUP) // GROUP), dtype=np.uint8)
    scales[:, up(dim, GROUP) // GROUP:] = 0
    return wide[:, 0::2] | (wide[:, 1::2] << 4), scales


# ------------------------------------------------------------ 8-bit states


class Kind:
    """low: fraction bits of fp32 that a code drops."""

    def __init__(self, signed):
        self.signed, self.low = signed, 20 if signed else 19
        self.first, self.top = (896, 127) if signed else (1792, 255)
        self.shift = 0 if signed else 1 << 31
        self.largest, self.least = self.f(self.top), self.f(1)

    def f(self, c):
        """F(c), from the definition of its bits."""
        bits = ((self.first + np.asarray(c, np.uint32)) << self.low).astype(np.uint32)
        return bits.view(np.float32).astype(np.float64)


M, R = Kind(True), Kind(False)


def blocks(x):
    pad = -x.size % BLOCK
    return np.concatenate([x, np.zeros(pad, x.dtype)]).reshape(-1, BLOCK)


def state_values(kind, codes, scale):
    c = codes.astype(np.uint32)
    mag = c & 127 if kind.signed else c
    f = np.where(mag > 0, kind.f(mag), 0.0)
    if kind.signed:
        f = np.where(c & 128, -f, f)
    return (blocks(f) * scale.astype(np.float64)[:, None]).reshape(-1)[: codes.size]


def state_scale(kind, x):
    """Scales of 64-bit values x, not rounded to fp32."""
    with np.errstate(invalid="ignore"):
        amax = np.abs(blocks(x)).max(1)
        s = np.where(amax > 0, np.maximum(amax / kind.largest, 2.0 ** -100), 0.0)
    return np.where(np.isfinite(blocks(x)).all(1), s, np.nan)


def dither(kind, i, t):
    """u in [0, 1)"""
    return ((MID_ELEM * i + MID_STEP * t + kind.shift) % (1 << 32)) / 2.0 ** 32


def check_codes(kind, codes, scale, x, u, err):
    """Codes of values x (64 bits, known to a relative error of err) with these
    fp32 scales and thresholds u: a code is the rounded one, or its neighbour
    where y lies so near the border of the two that its error decides.  y
    = |x| / scale is formed with two roundings (the reciprocal and the product)
    on top of err."""
    s = np.repeat(scale.astype(np.float64), BLOCK)[: x.size]
    c = codes.astype(np.int64)
    mag = c & 127 if kind.signed else c
    nan = ~np.isfinite(s)
    assert (c[nan | (s == 0)] == 0).all()
    ok = ~nan & (s > 0)
    c, mag, x, u, s = c[ok], mag[ok], x[ok], u[ok], s[ok]
    if kind.signed:
        assert (((c & 128) != 0) == ((x < 0) & (mag > 0))).all()
    bound = []
    for sign in (-1, 1):
        y = np.abs(x) / s * (1 + sign * (err + 2 * U32))
        # the place among codes: code k covers [F(k), F(k + 1))
        e = np.floor(np.log2(np.maximum(y, kind.least)))
        gap = 2.0 ** (e + kind.low - 23)
        up_to = np.floor(y / gap + u) * gap  # F of the rounded code, below the top
        code = (np.minimum(up_to, kind.largest).astype(np.float32).view(np.uint32) >> kind.low).astype(np.int64) - kind.first
        if kind.signed:
            small = (y > u * kind.least * (1 - sign * 2.0 ** -23)).astype(np.int64)
        else:
            small = (y > 0).astype(np.int64)
        bound.append(np.where(y < kind.least, small, np.minimum(code, kind.top)))
    assert (mag >= bound[0]).all() and (mag <= bound[1]).all(), "codes off their rounding"
    # the allowance is for borders only
    assert (bound[0] != bound[1]).mean() < 1e-3 or x.size < 5000


# -------------------------------------------------------------------- AdamW


def adamw(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step, scale=1.0):
    """(p, m, v, size of the update) in 64 bits."""
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    with np.errstate(invalid="ignore", divide="ignore"):
        upd = lr / (1 - beta1 ** step) * m / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - upd, m, v, np.abs(upd)
