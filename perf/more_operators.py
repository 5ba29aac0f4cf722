"""Training and serving in few bits: workloads of the microscaled 4-bit
(MXFP4) linear layer and of the AdamW step over a list of tensors.

Each case is one pass of one operator on synthetic activations, weights,
gradients and optimizer states.  ``own`` chooses between the operators of the
library and their plain form in elementary torch operations; ``exact``
computes the same results in 64 bits from the definitions.

Definitions:

* MXFP4: per group of 32 consecutive values of a row, E is the smallest
  integer in [-126, 126] with max|x| < 7 * 2^E; the code is the nearest of
  0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code) to |x| * 2^-E, with x's
  sign.  Two codes a byte, the first in its low half; a row of codes is
  16 * ceil(dim / 32) bytes, a row of scale bytes E + 127 is
  4 * ceil(dim / 128), zeros where there are no values.
* linear: y = Q(x) Q(w)^T; training adds dx = Q(dy) Q(w) with groups along
  the output channels, and dw = Q(dy)^T Q(x) with groups along the tokens.
* AdamW, decoupled weight decay: with g the gradient (times the clipping
  coefficient min(1, max_norm / norm)),
  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
  p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps).
* states in 8 bits: m and r = sqrt(v), per block of 256 consecutive elements
  of the concatenated list, as F(c) * s with s = max|x| / F(top), at least
  2^-100.  m: a sign and c of 7 bits, F(c) = the fp32 number with the bits
  (896 + c) << 20; r: c of 8 bits, (1792 + c) << 19; F(0) = 0.  x / s lies
  between two codes and is rounded up where its place between them is above
  1 - u, u = ((0x91E10DA5 i + 0xC13FA9A9 t) mod 2^32) / 2^32 for element i at
  step t (r: u + 1/2 mod 1); an r above zero never becomes zero.
"""
import math
import random

import torch

own = False

GROUP = 32
BLOCK = 256
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ADAM = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1}
MAX_NORM = 1.0
STEP = 100  # steps behind the first one
MID_M, MID_R = 0x91E10DA5, 0xC13FA9A9


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one new token through a square projection: latency, then the weights' bytes
        {"name": "linear_one_token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16"},
        # a batch of decoding requests, an odd number of them, through a wide projection
        {"name": "linear_37_tokens", "op": "linear", "m": 37, "n": 8192, "k": 2048, "dtype": "bf16"},
        # one sequence of prefill, sizes that fill no tile, an fp32 model
        {"name": "linear_ragged_f32", "op": "linear", "m": 1003, "n": 1530, "k": 2043, "dtype": "f32"},
        # a large micro-batch through the widest layer
        {"name": "linear_16384_tokens", "op": "linear", "m": 16384, "n": 8192, "k": 8192, "dtype": "bf16"},
        # a training step of a small fp32 layer, no size a multiple of a tile
        {"name": "train_ragged_f32", "op": "train", "m": 1027, "n": 510, "k": 770, "dtype": "f32"},
        # a training step of a square projection over one sequence: weights and activations in both orientations
        {"name": "train_4096_tokens", "op": "train", "m": 4096, "n": 4096, "k": 4096, "dtype": "bf16"},
        # a few rows saved in 4 bits and restored: latency
        {"name": "quantise_5_rows_f32", "op": "quantise", "rows": 5, "dim": 515, "dtype": "f32"},
        # the weights of a wide layer, in both orientations
        {"name": "quantise_8192_rows", "op": "quantise", "rows": 8192, "dim": 8192, "dtype": "bf16"},
        # gains and biases of a small model: latency
        {"name": "adamw_small_list", "op": "adamw", "tensors": 24, "n": 40000, "ptype": "f32", "gtype": "f32",
         "master": False, "bits": 32, "clip": True},
        # a small bf16 model's list of odd sizes, states in 8 bits
        {"name": "adamw8_ragged_list", "op": "adamw", "tensors": 77, "n": 3000001, "ptype": "bf16", "gtype": "bf16",
         "master": False, "bits": 8, "clip": True},
        # one GPU's share of a model in fp32
        {"name": "adamw_268m", "op": "adamw", "tensors": 150, "n": 268435456, "ptype": "f32", "gtype": "f32",
         "master": False, "bits": 32, "clip": True},
        # the same in bf16 with fp32 master weights and states in 8 bits
        {"name": "adamw8_268m", "op": "adamw", "tensors": 150, "n": 268435456, "ptype": "bf16", "gtype": "bf16",
         "master": True, "bits": 8, "clip": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Log-uniform; half the time rounded to a multiple of 64, as layers are."""
    v = _log(rng, lo, hi)
    if v >= 64 and rng.random() < 0.5:
        v = min(hi, (v + 32) // 64 * 64)
    return v


def draw(rng):
    op = rng.choice(["linear", "linear", "train", "quantise", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "linear":
        return {"op": op, "m": _size(rng, 1, 16384), "n": _size(rng, 64, 8192), "k": _size(rng, 32, 8192), "dtype": dtype}
    if op == "train":
        return {"op": op, "m": _size(rng, 1, 8192), "n": _size(rng, 64, 4096), "k": _size(rng, 32, 4096), "dtype": dtype}
    if op == "quantise":
        return {"op": op, "rows": _size(rng, 1, 8192), "dim": _size(rng, 8, 8192), "dtype": dtype}
    n = _size(rng, 1000, 1 << 28)
    return {"op": op, "tensors": _log(rng, 1, 200), "n": n, "ptype": dtype, "gtype": rng.choice([dtype, "f32"]),
            "master": dtype == "bf16" and rng.random() < 0.5, "bits": rng.choice([8, 8, 32]), "clip": rng.random() < 0.5}


def _held_bytes(rows, dim):
    return rows * (_up(dim, GROUP) // 2 + _up(dim, GROUP) // GROUP)


def work(case):
    if case["op"] == "adamw":
        p, g = (2 if case[k] == "bf16" else 4 for k in ("ptype", "gtype"))
        state = 2 * 8 if case["bits"] == 32 else 2 * (2 + 8 / BLOCK) + 4  # the 8-bit states' values in bf16 are outputs
        return {"bytes": case["n"] * (g + state + (p + 8 if case["master"] else 2 * p)), "flops": 20 * case["n"]}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quantise":
        r, d = case["rows"], case["dim"]
        return {"bytes": 3 * r * d * e + 2 * (_held_bytes(r, d) + _held_bytes(d, r)), "flops": 8 * r * d}
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "linear":
        return {"bytes": m * k * e + _held_bytes(n, k) + m * n * e, "flops": 2 * m * n * k}
    return {"bytes": 2 * e * (m * k + m * n) + n * k * (e + 8), "flops": 6 * m * n * k}


# ----------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g)


def _activations(rows, dim, g):
    """Normal values with a spread of channel gains, one channel in 256 an
    outlier, and tokens of different size, as hidden states have."""
    gain = torch.exp(0.5 * _normal((dim,), g))
    pick = torch.rand((dim,), generator=g, device="cuda") < 1.0 / 256
    gain = torch.where(pick, gain * 20.0, gain)
    return _normal((rows, dim), g) * gain * torch.exp(0.3 * _normal((rows, 1), g))


def _gradients(rows, dim, g):
    return _normal((rows, dim), g) * (1e-3 * torch.exp(0.5 * _normal((rows, 1), g)))


def _weights(n, k, g):
    return _normal((n, k), g) * (k ** -0.5) * torch.exp(0.2 * _normal((n, 1), g))


def _up(v, unit):
    return -(-v // unit) * unit


def _mx_buffers(rows, dim):
    """Buffers of a matrix in MXFP4: codes and scale bytes."""
    return (torch.zeros((rows, _up(dim, GROUP) // 2), dtype=torch.uint8, device="cuda"),
            torch.zeros((rows, _up(dim, 4 * GROUP) // GROUP), dtype=torch.uint8, device="cuda"))


def _sizes(case):
    """Sizes of the tensors of a list, n elements in all: a few of them hold most."""
    rng = random.Random(case["tensors"] * 1000003 + case["n"])
    count = min(case["tensors"], case["n"])
    share = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(count)]
    spare, total = case["n"] - count, sum(share)
    sizes = [1 + int(spare * s / total) for s in share]
    sizes = [s // 64 * 64 if s >= 64 and rng.random() < 0.5 else s for s in sizes]
    sizes[-1] += case["n"] - sum(sizes)
    return sizes


def _list_of(sizes, dtype):
    """A zero buffer that holds tensors of these sizes, each from a multiple of
    64 elements on, as an allocator lays them out; and the tensors."""
    at = [0]
    for s in sizes:
        at.append(at[-1] + _up(s, 64))
    flat = torch.zeros(at[-1], dtype=dtype, device="cuda")
    return flat, [flat[a: a + s] for a, s in zip(at, sizes)]


def _pointers(tensors):
    return torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64, device="cuda")


def _prepare_adamw(s, g):
    n, sizes = s["n"], _sizes(s)
    s["sizes"] = sizes
    s["params"], s["param_list"] = _list_of(sizes, DTYPES[s["ptype"]])
    s["grads"], s["grad_list"] = _list_of(sizes, DTYPES[s["gtype"]])
    # parameters and gradients of a tensor are of one size, which differs from tensor to tensor
    size_of = torch.repeat_interleave(torch.exp(_normal((len(sizes),), g)), torch.tensor(sizes, device="cuda"),
                                      output_size=n)
    p = _normal((n,), g) * size_of * 0.02
    torch._foreach_copy_(s["param_list"], list(p.split(sizes)))
    s["master_p"] = p if s["master"] else None
    grad = _normal((n,), g) * size_of * 1e-3
    # rows of embeddings that no token of the batch used have no gradient
    grad *= (torch.rand((n,), generator=g, device="cuda") > 0.05)
    torch._foreach_copy_(s["grad_list"], list(grad.split(sizes)))
    # what earlier steps left
    m = (grad + _normal((n,), g) * size_of * 1e-3) * 0.3
    r = size_of * 1e-3 * torch.exp(0.3 * _normal((n,), g))
    if s["bits"] == 32:
        s["m"], s["v"] = m, r.square()
    else:
        nb = -(-n // BLOCK)
        s["m_codes"], s["r_codes"] = (torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        s["m_scale"], s["r_scale"] = (torch.empty(nb, dtype=torch.float32, device="cuda") for _ in range(2))
        dither = torch.full((n,), 1 << 31, dtype=torch.int64, device="cuda")
        _save_state(m, dither, 20, s["m_codes"], s["m_scale"])
        _save_state(r, dither, 19, s["r_codes"], s["r_scale"])
        s["m_values"], s["r_values"] = (torch.empty(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    # the list's tables: pointers, prefix sums of the sizes, and the tensor that holds each 4096th element
    s["xs"], s["gs"] = _pointers(s["param_list"]), _pointers(s["grad_list"])
    offsets = torch.zeros(len(sizes) + 1, dtype=torch.int64)
    offsets[1:] = torch.tensor(sizes).cumsum(0)
    marks = torch.clamp(torch.arange(-(-n // 4096) + 1) * 4096, max=n - 1)
    s["seg_first"] = (torch.searchsorted(offsets, marks, right=True) - 1).to(torch.int32).cuda()
    s["offsets"] = offsets.cuda()
    s["norm"] = torch.ones(2, dtype=torch.float32, device="cuda")
    s["step"] = STEP
    s["workspace"] = None


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "adamw":
        _prepare_adamw(s, g)
        return s
    t = DTYPES[case["dtype"]]
    if case["op"] == "quantise":
        rows, dim = case["rows"], case["dim"]
        s["x"] = _weights(rows, dim, g).to(t)
        s["kept"], s["kept_t"] = _mx_buffers(rows, dim), _mx_buffers(dim, rows)
        s["y"], s["yt"] = torch.empty_like(s["x"]), torch.empty((dim, rows), dtype=t, device="cuda")
        return s
    m, n, k = case["m"], case["n"], case["k"]
    s["x"] = _activations(m, k, g).to(t)
    s["y"] = torch.empty((m, n), dtype=t, device="cuda")
    s["workspace"] = None
    w = _weights(n, k, g)
    if case["op"] == "linear":
        s["w"] = _mx_buffers(n, k)  # laid out once when the model is loaded
        _pack(w.to(t).float(), *s["w"])
        return s
    s["w"], s["dy"] = w.to(t), _gradients(m, n, g).to(t)
    for name, (r, d) in (("x", (m, k)), ("w", (n, k)), ("dy", (m, n))):
        s[name + "_kept"], s[name + "_kept_t"] = _mx_buffers(r, d), _mx_buffers(d, r)
    s["dx"] = torch.empty((m, k), dtype=t, device="cuda")
    # what the first micro-batch of the step left in the gradient
    s["dw"] = _normal((n, k), g) * (1e-3 * m ** 0.5)
    return s


# ------------------------------------------------- plain form: the 4-bit layer


def _save(x):
    """Codes [rows, groups, 32] (0..15) and scale bytes [rows, groups] of an fp32 matrix."""
    rows, dim = x.shape
    x = torch.nn.functional.pad(x, (0, _up(dim, GROUP) - dim)).view(rows, -1, GROUP)
    bits = x.abs().amax(2).view(torch.int32)
    # 7 = 1.75 * 2^2: a fraction from there on needs the next power of two
    byte = ((bits >> 23) - 2 + ((bits & 0x7FFFFF) >= 0x600000)).clamp(1, 253)
    y = x.abs() * ((254 - byte) << 23).view(torch.float32)[:, :, None]
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    return code + 8 * torch.signbit(x), byte


def _pack(x, codes, scales):
    c, byte = _save(x)
    scales[:, : byte.shape[1]] = byte.to(torch.uint8)
    c = c.view(c.shape[0], -1, 2)
    codes.copy_(c[:, :, 0] | (c[:, :, 1] << 4))


def _restore(code, byte, dim):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    v = torch.cat([table, -table])[code.int()] * (byte.to(torch.int32) << 23).view(torch.float32)[:, :, None]
    return v.reshape(v.shape[0], -1)[:, :dim]


def _held(x):
    return _restore(*_save(x.float()), x.shape[1])


def _unpacked(codes, scales, dim):
    c = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1, GROUP)
    return _restore(c, scales[:, : c.shape[1]], dim)


# ---------------------------------------------------- plain form: the optimizer


def _save_state(x, u, low, codes, scale):
    """x in blocks: magnitudes rounded at bit `low` with thresholds u (32 bits), r where low is 19, m where it is 20."""
    n, nb = x.numel(), scale.numel()
    signed = low == 20
    first, top = (896, 127) if signed else (1792, 255)
    pad = nb * BLOCK - n
    xb = torch.nn.functional.pad(x, (0, pad)).view(nb, BLOCK)
    amax = xb.abs().amax(1)
    largest = torch.tensor((first + top) << low, dtype=torch.int32, device="cuda").view(torch.float32)
    least = torch.tensor((first + 1) << low, dtype=torch.int32, device="cuda").view(torch.float32)
    s = torch.where(amax > 0, torch.clamp(amax * (1.0 / largest), min=2.0 ** -100), torch.zeros_like(amax))
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    y = (xb.abs() * inv[:, None]).view(-1)[:n]
    c = ((y.view(torch.int32) + (u >> (32 - low)).to(torch.int32)) >> low) - first
    # below the first code there is only zero
    under = y > (u >> 8).to(torch.float32) * (least * 2.0 ** -24) if signed else y > 0
    c = torch.where(y < least, under.to(torch.int32), c.clamp(max=top))
    codes.copy_(c | ((x < 0).to(torch.int32) << 7) * (c > 0) if signed else c)
    scale.copy_(s)


def _state(codes, scale, low):
    signed = low == 20
    c = codes.to(torch.int32)
    mag = c & 127 if signed else c
    f = torch.where(mag > 0, (((896 if signed else 1792) + mag) << low).view(torch.float32), torch.zeros((), device="cuda"))
    f = torch.where(c >= 128, -f, f) if signed else f
    nb = scale.numel()
    f = torch.nn.functional.pad(f, (0, nb * BLOCK - f.numel())).view(nb, BLOCK)
    return (f * scale[:, None]).view(-1)[: codes.numel()]


def _plain_adamw(s):
    s["step"] += 1
    n, t = s["n"], s["step"]
    g = torch.cat(s["grad_list"]).float()
    if s["clip"]:
        norm = g.double().square().sum().sqrt()
        s["norm"].copy_(torch.stack([norm, torch.clamp(MAX_NORM / norm, max=1.0)]))
        g = g * s["norm"][1]
    p = s["master_p"] if s["master"] else torch.cat(s["param_list"]).float()
    b1, b2 = ADAM["beta1"], ADAM["beta2"]
    m = s["m"] if s["bits"] == 32 else _state(s["m_codes"], s["m_scale"], 20)
    v = s["v"] if s["bits"] == 32 else _state(s["r_codes"], s["r_scale"], 19).square()
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + g * g * (1.0 - b2)
    r = v.sqrt()
    p = p * (1.0 - ADAM["lr"] * ADAM["weight_decay"])
    p = p - m * (ADAM["lr"] / (1.0 - b1 ** t)) / (r * (1.0 / math.sqrt(1.0 - b2 ** t)) + ADAM["eps"])
    if s["master"]:
        s["master_p"].copy_(p)
    torch._foreach_copy_(s["param_list"], list(p.split(s["sizes"])))
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        u = torch.arange(n, device="cuda") * MID_M + t * MID_R
        _save_state(m, u & 0xFFFFFFFF, 20, s["m_codes"], s["m_scale"])
        _save_state(r, (u + (1 << 31)) & 0xFFFFFFFF, 19, s["r_codes"], s["r_scale"])
        s["m_values"].copy_(_state(s["m_codes"], s["m_scale"], 20))
        s["r_values"].copy_(_state(s["r_codes"], s["r_scale"], 19))
    return _adamw_outputs(s)


def _adamw_outputs(s):
    out = {"params": s["params"], "norm": s["norm"]}
    if s["master"]:
        out["master"] = s["master_p"]
    if s["bits"] == 32:
        return out | {"m": s["m"], "v": s["v"]}
    # states in 8 bits: the values they stand for, and the blocks' scales
    return out | {"m": s["m_values"], "r": s["r_values"], "m_scale": s["m_scale"], "r_scale": s["r_scale"]}


def _plain(s):
    if s["op"] == "adamw":
        return _plain_adamw(s)
    t = s["x"].dtype
    if s["op"] == "quantise":
        x = s["x"].float()
        return {"rows": _held(x).to(t), "columns": _held(x.t().contiguous()).to(t)}
    if s["op"] == "linear":
        return (_held(s["x"]) @ _unpacked(*s["w"], s["k"]).t()).to(t)
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    y = _held(x) @ _held(w).t()
    dx = _held(dy) @ _held(w.t().contiguous()).t()
    s["dw"] += _held(dy.t().contiguous()) @ _held(x.t().contiguous()).t()
    return {"y": y.to(t), "dx": dx.to(t), "dw": s["dw"]}


# ------------------------------------------------- the library's operators


def _space(s, need):
    """Workspace, kept by the program as the weights are."""
    if s["workspace"] is None:
        s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _library_adamw(qc, s):
    s["step"] += 1
    pt, gt = (qc.QC_BF16 if s[k] == "bf16" else qc.QC_F32 for k in ("ptype", "gtype"))
    tables = (s["offsets"], s["seg_first"], len(s["sizes"]), s["n"])
    coefficient = None
    if s["clip"]:
        space = _space(s, qc.qc_grad_norm_workspace(s["n"]))
        qc.qc_grad_norm_multi(s["gs"], gt, *tables, MAX_NORM, space, s["norm"])
        coefficient = s["norm"][1:]
    if s["bits"] == 32:
        qc.qc_adamw_multi(s["xs"], pt, s["gs"], gt, *tables, s["master_p"], s["m"], s["v"], step=s["step"],
                          grad_scale=coefficient, **ADAM)
    else:
        qc.qc_adamw8_multi(s["xs"], pt, s["gs"], gt, *tables, s["master_p"], s["m_codes"], s["m_scale"], s["r_codes"],
                           s["r_scale"], step=s["step"], grad_scale=coefficient, **ADAM)
        qc.qc_decode_state8(qc.QC_STATE_M, s["m_codes"], s["m_scale"], s["n"], s["m_values"], qc.QC_BF16)
        qc.qc_decode_state8(qc.QC_STATE_R, s["r_codes"], s["r_scale"], s["n"], s["r_values"], qc.QC_BF16)
    return _adamw_outputs(s)


def _library(s):
    import embedding_communication_codecs_amd as qc

    if s["op"] == "adamw":
        return _library_adamw(qc, s)
    t = qc.QC_BF16 if s["dtype"] == "bf16" else qc.QC_F32
    if s["op"] == "quantise":
        rows, dim = s["rows"], s["dim"]
        qc.qc_encode_mxfp4(s["x"], t, rows, dim, dim, *s["kept"], *s["kept_t"])
        qc.qc_decode_mxfp4(*s["kept"], rows, dim, s["y"], t, dim)
        qc.qc_decode_mxfp4(*s["kept_t"], dim, rows, s["yt"], t, rows)
        return {"rows": s["y"], "columns": s["yt"]}
    m, n, k = s["m"], s["n"], s["k"]
    if s["op"] == "linear":
        space = _space(s, qc.qc_linear_mxfp4_workspace(m, n, k, t))
        qc.qc_linear_mxfp4(s["x"], t, k, *s["w"], m, n, k, s["y"], t, n, space)
        return s["y"]
    # forward, then the gradients of the input and of the weights
    need = max(qc.qc_matmul_mxfp4_workspace(m, n, k), qc.qc_matmul_mxfp4_workspace(m, k, n),
               qc.qc_matmul_mxfp4_workspace(n, k, m))
    space = _space(s, need)
    qc.qc_encode_mxfp4(s["x"], t, m, k, k, *s["x_kept"], *s["x_kept_t"])
    qc.qc_encode_mxfp4(s["w"], t, n, k, k, *s["w_kept"], *s["w_kept_t"])
    qc.qc_matmul_mxfp4(*s["x_kept"], *s["w_kept"], m, n, k, s["y"], t, n, False, space)
    qc.qc_encode_mxfp4(s["dy"], t, m, n, n, *s["dy_kept"], *s["dy_kept_t"])
    qc.qc_matmul_mxfp4(*s["dy_kept"], *s["w_kept_t"], m, k, n, s["dx"], t, k, False, space)
    qc.qc_matmul_mxfp4(*s["dy_kept_t"], *s["x_kept_t"], n, k, m, s["dw"], qc.QC_F32, k, True, space)
    return {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------- 64-bit definitions


def _two_to(e):
    """2^e in 64 bits from its bit pattern (a power function may round it)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest4(x):
    """x as MXFP4 holds it, groups along the rows, in 64 bits."""
    x = x.double()
    out = torch.empty_like(x)
    for at in range(0, x.shape[1], GROUP):
        part = x[:, at: at + GROUP]
        mant, e = torch.frexp(part.abs().max(1).values)  # mant in [0.5, 1), times 2^e
        step = _two_to(torch.where(mant * 8 < 7, e - 3, e - 2).clamp(-126, 126))[:, None]
        y = part.abs() / step
        # neighbours are 1/2 apart below 2, 1 below 4, 2 above
        gap = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0).double())
        out[:, at: at + GROUP] = torch.copysign(torch.round(y / gap) * gap * step, part)
    return out


def _kept_values(codes, scales, dim):
    out = torch.empty((codes.shape[0], _up(dim, GROUP)), dtype=torch.float64, device="cuda")
    half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], dtype=torch.float64, device="cuda")
    out[:, 0::2] = half[(codes % 16).long()]
    out[:, 1::2] = half[(codes // 16).long()]
    step = _two_to(scales.int() - 128)  # a half step, as `half` counts halves
    return (out * step.repeat_interleave(GROUP, 1)[:, : out.shape[1]])[:, :dim]


def _product(a, b):
    """a b^T"""
    return a.contiguous() @ b.t().contiguous()


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _of_state(codes, scale, bits):
    """64-bit values of a state with `bits` bits of magnitude: exponent and
    fraction read off the code."""
    keep = bits - 4
    c = codes.long()
    mag = c % (1 << bits)
    f = (1 + (mag % (1 << keep)).double() / (1 << keep)) * _two_to(mag // (1 << keep) - 15)
    f = torch.where(mag == 0, 0.0, f) * torch.where(c >= (1 << bits), -1.0, 1.0).double()
    return (_blocks(f) * scale.double()[:, None]).view(-1)[: codes.numel()]


def _rounded_state(x, u, bits):
    """The values that the state of x stands for, and the blocks' scales."""
    keep = bits - 4
    top = 2.0 - 2.0 ** -keep
    first = (1 + 2.0 ** -keep) * 2.0 ** -15
    b = _blocks(x)
    amax = b.abs().max(1).values
    s = torch.where(amax > 0, torch.clamp(amax / top, min=2.0 ** -100), 0.0).float().double()
    y = (b.abs() / torch.where(s > 0, s, 1.0)[:, None]).view(-1)[: x.numel()]
    gap = _two_to(torch.frexp(y.clamp(min=2.0 ** -15)).exponent - 1 - keep)
    q = torch.clamp(torch.floor(y / gap + u) * gap, max=top)
    low = y > u * first if bits == 7 else y > 0
    q = torch.where(y < first, torch.where(low, first, 0.0), q) * torch.where(x < 0, -1.0, 1.0)
    return (_blocks(q) * s[:, None]).view(-1)[: x.numel()], s


def _exact_adamw(s):
    n, sizes, t = s["n"], s["sizes"], STEP + 1
    g = torch.cat(s["grad_list"]).double()
    norm = s["norm"].double()
    if s["clip"]:
        norm = torch.linalg.vector_norm(g)
        norm = torch.stack([norm, torch.clamp(MAX_NORM / norm, max=1.0)])
        g *= norm[1]
    p = s["master_p"].double() if s["master"] else torch.cat(s["param_list"]).double()
    m = s["m"].double() if s["bits"] == 32 else _of_state(s["m_codes"], s["m_scale"], 7)
    v = s["v"].double() if s["bits"] == 32 else _of_state(s["r_codes"], s["r_scale"], 8) ** 2
    m = torch.lerp(m, g, 1 - ADAM["beta1"])
    v = v + (1 - ADAM["beta2"]) * (g * g - v)
    m_hat, v_hat = m / (1 - ADAM["beta1"] ** t), v / (1 - ADAM["beta2"] ** t)
    p = p - ADAM["lr"] * (ADAM["weight_decay"] * p + m_hat / (torch.sqrt(v_hat) + ADAM["eps"]))
    del g, m_hat, v_hat
    flat, parts = _list_of(sizes, torch.float64)
    torch._foreach_copy_(parts, list(p.split(sizes)))
    out = {"params": flat, "norm": norm}
    if s["master"]:
        out["master"] = p
    if s["bits"] == 32:
        return out | {"m": m, "v": v}
    u = torch.remainder(torch.arange(n, device="cuda") * MID_M + t * MID_R, 1 << 32).double() / 2.0 ** 32
    out["m"], out["m_scale"] = _rounded_state(m, u, 7)
    out["r"], out["r_scale"] = _rounded_state(v.sqrt(), torch.remainder(u + 0.5, 1.0), 8)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    if case["op"] == "quantise":
        return {"rows": _nearest4(s["x"]), "columns": _nearest4(s["x"].t())}
    if case["op"] == "linear":
        return _product(_nearest4(s["x"]), _kept_values(*s["w"], case["k"]))
    x, w, dy = s["x"], s["w"], s["dy"]
    return {"y": _product(_nearest4(x), _nearest4(w)), "dx": _product(_nearest4(dy), _nearest4(w.t())),
            "dw": s["dw"].double() + _product(_nearest4(dy.t()), _nearest4(x.t()))}
