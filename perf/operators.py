"""What is measured of the 8-bit layer and the attention input that follows it.

Four operators, each in its plain form (elementary torch operations, below) and as the call a
user of the library makes:

- ``gemm``    the product of int8 activations and int8 weights, a scale for each token and each
              output channel, the centering's rank-1 term and a bias (gemm_w8a8);
- ``linear``  the whole layer on it: center, rotate, quantize, multiply (linear_w8a8);
- ``heads``   the norm of every query and key head and the rotation of its position, one pass
              (qk_norm_rope);
- ``qkv``     the projection to queries, keys and values with that pass behind it (linear_qkv).

Widths are those of the library's layers (1920, 4096, 12288) or generic; the activations are
the diffusion transformer's (unit normal entries, one in a hundred of heavy tail, a mean for
each token), the weights normal with variance 1/d.
"""
import math

import numpy as np
import torch

own = False

HEAVY = 0.01        # share of activation entries drawn from a heavy tail
MEAN_STD = 3 ** 0.5  # deviation of the tokens' means
EPS = 1e-10         # floor of a token's largest magnitude


# ---- cases ----------------------------------------------------------------------------------

def _gemm(name, T, K, N, out="bf16", mean=True, bias=True):
    return {"name": name, "op": "gemm", "T": T, "K": K, "N": N, "out": out, "mean": mean,
            "bias": bias}


def _linear(name, T, d, N, center=True, bias=True):
    return {"name": name, "op": "linear", "T": T, "d": d, "N": N, "center": center, "bias": bias}


def _heads(name, B, S, Hq, Hk, D, norm, rope, rot, packed, heads_first):
    return {"name": name, "op": "heads", "B": B, "S": S, "Hq": Hq, "Hk": Hk, "D": D,
            "norm": norm, "rope": rope, "rot": rot, "packed": packed, "heads_first": heads_first}


def _qkv(name, B, S, d, Hq, Hk, D, bits, norm, rope, rot, center):
    return {"name": name, "op": "qkv", "B": B, "S": S, "d": d, "Hq": Hq, "Hk": Hk, "D": D,
            "bits": bits, "norm": norm, "rope": rope, "rot": rot, "center": center}


def listed():
    return [
        # one token through a square projection: the latency of a decoding step
        _gemm("gemm_1x4096x4096", 1, 4096, 4096),
        # a small serving batch through a fused projection of a narrow model
        _gemm("gemm_24x1920x5760", 24, 1920, 5760, mean=False),
        # raw sums for a user who applies scales of their own; odd token count, K no multiple of 128
        _gemm("gemm_333x2080x1200_sums", 333, 2080, 1200, out="acc", mean=False, bias=False),
        # the wide half of a transformer's MLP over an image's tokens: the largest product
        _gemm("gemm_4096x4096x12288", 4096, 4096, 12288),
        # the whole layer for a handful of tokens (two rounds of the rotation)
        _linear("linear_7x1920x1920", 7, 1920, 1920),
        # the whole layer over an image's tokens
        _linear("linear_4096x4096x4096", 4096, 4096, 4096),
        # a decoding step of four sequences, each at its own position, grouped keys
        _heads("heads_decode_4x1", 4, 1, 32, 8, 128, "rms", "halves", 128, True, False),
        # an odd length, a head size that is no power of two, part of it rotated, layer norm,
        # and an output laid out head by head for the attention
        _heads("heads_3x777_part", 3, 777, 12, 12, 96, "layer", "pairs", 64, False, True),
        # a batch of long sequences out of the packed projection
        _heads("heads_2x8192", 2, 8192, 32, 8, 128, "rms", "halves", 128, True, True),
        # one token's queries, keys and values
        _qkv("qkv_1x4096", 1, 1, 4096, 32, 8, 128, 8, "rms", "halves", 128, True),
        # a narrow model's text tokens through 4-bit weights, heads of 64 under a layer norm
        _qkv("qkv_226x1920_w4", 1, 226, 1920, 30, 30, 64, 4, "layer", "pairs", 64, True),
        # an image's tokens, heads of 128
        _qkv("qkv_4096x4096", 1, 4096, 4096, 32, 8, 128, 8, "rms", "pairs", 128, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, m):
    return max(lo, min(hi, m * max(1, round(_log(rng, lo, hi) / m))))


WIDTHS = (256, 640, 1152, 1920, 2560, 4096)


def draw(rng):
    op = rng.choice(["gemm", "linear", "heads", "qkv"])
    if op == "gemm":
        K, N = _multiple(rng, 256, 12288, 32), _multiple(rng, 256, 12288, 16)
        T = _log(rng, 1, min(8192, 4096 * 4096 * 12288 // (K * N)))
        out = rng.choice(["bf16", "bf16", "bf16", "acc"])
        return {"op": op, "T": T, "K": K, "N": N, "out": out,
                "mean": out == "bf16" and rng.random() < 0.5,
                "bias": out == "bf16" and rng.random() < 0.5}
    if op == "linear":
        return {"op": op, "T": _log(rng, 1, 4096), "d": rng.choice(WIDTHS),
                "N": _multiple(rng, 256, 4096, 16), "center": rng.random() < 0.7,
                "bias": rng.random() < 0.5}
    if op == "heads":
        D = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 8, 12])
        Hq, B = Hk * rng.choice([1, 2, 4]), rng.choice([1, 2, 3, 8])
        S = _log(rng, 1, min(2048, 2 * 8192 * 40 * 128 // (B * (Hq + Hk) * D)))
        return {"op": op, "B": B, "S": S, "Hq": Hq, "Hk": Hk, "D": D,
                "norm": rng.choice(["rms", "rms", "layer"]),
                "rope": rng.choice(["pairs", "halves"]), "rot": rng.choice([D, D, D // 32 * 16 or D]),
                "packed": rng.random() < 0.5, "heads_first": rng.random() < 0.5}
    d, D = rng.choice(WIDTHS), rng.choice([64, 96, 128, 128])
    Hk = rng.choice([1, 2, 4, 8])
    return {"op": op, "B": rng.choice([1, 2, 4]), "S": _log(rng, 1, 1024), "d": d,
            "Hq": Hk * rng.choice([1, 2, 4]), "Hk": Hk, "D": D, "bits": rng.choice([8, 8, 8, 4]),
            "norm": rng.choice(["rms", "rms", "layer"]), "rope": rng.choice(["pairs", "halves"]),
            "rot": rng.choice([D, D, D // 2]), "center": rng.random() < 0.7}


# ---- inputs ---------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, T, d):
    x = _normal(g, T, d)
    tail = 3 ** 0.5 * _normal(g, T, d) / (_normal(g, 3, T, d).square().sum(0).sqrt() + 1e-3)
    x = torch.where(torch.rand(T, d, generator=g, device="cuda") < HEAVY, tail, x)
    return (x + MEAN_STD * _normal(g, T, 1)).bfloat16()


def _weights(g, N, d, top, center):
    """Codes and scales of weights with variance 1/d, and their row sums."""
    w = _normal(g, N, d) / d ** 0.5
    s = w.abs().amax(1) / top
    codes = torch.round(w / s[:, None]).clamp_(-top, top).to(torch.int8)
    return codes, s, (_normal(g, N) if center else None)


def _pack4(codes):
    """The 4-bit layout: byte j of a 16-byte group holds elements j (low) and 16 + j (high)."""
    n, k = codes.shape
    c = (codes.view(n, k // 32, 2, 16) & 15).to(torch.uint8)
    return (c[:, :, 0] | (c[:, :, 1] << 4)).reshape(n, k // 2).contiguous()


def _block(d):
    return min(d & -d, 1024)


def _mix(z):
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


def _stream(key, i):
    with np.errstate(over="ignore"):
        return _mix(np.uint64(key) + (np.asarray(i, np.uint64) + np.uint64(1)) * np.uint64(0x9E3779B97F4A7C15))


def _rotation(d, h, seed):
    """Signs and gathers of the rotation's rounds, and the block's Hadamard matrix."""
    rounds, i = [], np.arange(d)
    for r in range(2 if h < 512 else 1):
        sign = np.where(_stream(_stream(seed, 2 * r), i) >> np.uint64(63), -1.0, 1.0)
        gather = np.argsort(_stream(_stream(seed, 2 * r + 1), i), kind="stable")
        rounds.append((torch.from_numpy(sign).float().cuda(), torch.from_numpy(gather).cuda()))
    bits = torch.arange(h, device="cuda")
    both, parity = bits[:, None] & bits[None, :], torch.zeros(h, h, dtype=torch.long, device="cuda")
    for b in range(10):
        parity ^= (both >> b) & 1
    return rounds, (1 - 2 * parity).float() / h ** 0.5


def _table(n, rot):
    """Cosines and sines of n positions, rot / 2 frequencies (base 10000)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return a.cos().float(), a.sin().float()


def _head_inputs(g, c):
    """Norm weights, the table of angles and the positions: decoding steps sit far into their
    sequences, and every eighth token of a longer one (text among image tokens) has none (-1)."""
    B, S, D = c["B"], c["S"], c["D"]
    n = 16384
    cos, sin = _table(n, c["rot"])
    if S == 1:
        pos = torch.randint(0, n, (B, 1), generator=g, device="cuda")
    else:
        pos = torch.arange(S, device="cuda")[None, :] + torch.randint(0, 16, (B, 1), generator=g, device="cuda")
        pos = torch.where(torch.arange(S, device="cuda") % 8 == 7, -1, pos)
    layer = c["norm"] == "layer"
    s = {"cos": cos, "sin": sin, "pos": pos.to(torch.int32), "eps": 1e-6,
         "qw": 1 + 0.2 * _normal(g, D), "kw": 1 + 0.2 * _normal(g, D),
         "qb": 0.2 * _normal(g, D) if layer else None, "kb": 0.2 * _normal(g, D) if layer else None}
    if own:
        import w4a8_ptq_linear_b200 as oq
        s["heads"] = oq.Heads(D, c["Hq"], c["Hk"], norm=c["norm"], eps=s["eps"], q_weight=s["qw"],
                              q_bias=s["qb"], k_weight=s["kw"], k_bias=s["kb"], rope=c["rope"],
                              cos=cos, sin=sin)
    return s


def _layer(s, seed, d, center):
    """The layer's rotation, and the library's plan for it."""
    h = _block(d)
    s["rounds"], s["H"] = _rotation(d, h, int(seed))
    if own:
        import w4a8_ptq_linear_b200 as oq
        s["plan"] = oq.Plan(d, h, len(s["rounds"]), seed=int(seed), center=center)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "gemm":
        s["a"] = torch.round(40 * _normal(g, c["T"], c["K"])).clamp_(-127, 127).to(torch.int8)
        s["scale"] = 0.02 + 0.02 * torch.rand(c["T"], generator=g, device="cuda")
        s["w"], s["ws"], s["w1"] = _weights(g, c["N"], c["K"], 127, c["mean"])
        s["mean"] = MEAN_STD * _normal(g, c["T"]) if c["mean"] else None
        s["bias"] = _normal(g, c["N"]).bfloat16() if c["bias"] else None
    elif c["op"] == "linear":
        s["x"] = _activations(g, c["T"], c["d"])
        s["w"], s["ws"], s["w1"] = _weights(g, c["N"], c["d"], 127, c["center"])
        s["bias"] = _normal(g, c["N"]).bfloat16() if c["bias"] else None
        _layer(s, seed, c["d"], c["center"])
    elif c["op"] == "heads":
        B, S, Hq, Hk, D = c["B"], c["S"], c["Hq"], c["Hk"], c["D"]
        s |= _head_inputs(g, c)
        if c["packed"]:  # slices of a projection's rows, values behind the keys
            rows = _normal(g, B, S, (Hq + 2 * Hk) * D).bfloat16()
            s["q"] = rows[..., :Hq * D].unflatten(-1, (Hq, D))
            s["k"] = rows[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        else:
            s["q"] = _normal(g, B, S, Hq, D).bfloat16()
            s["k"] = _normal(g, B, S, Hk, D).bfloat16()
    else:
        T, N = c["B"] * c["S"], (c["Hq"] + 2 * c["Hk"]) * c["D"]
        s |= _head_inputs(g, c)
        s["x"] = _activations(g, T, c["d"])
        codes, s["ws"], s["w1"] = _weights(g, N, c["d"], 127 if c["bits"] == 8 else 7, c["center"])
        s["w"] = codes if c["bits"] == 8 else _pack4(codes)
        s["bias"] = None
        _layer(s, seed, c["d"], c["center"])
    return s


# ---- the plain forms and the library's calls --------------------------------------------------

def _plain_linear(s, center):
    """The layer in float32, before the rounding of its result."""
    x, w = s["x"].float(), s["w"]
    if w.dtype == torch.uint8:
        b = w.view(w.shape[0], -1, 16)
        n = torch.cat([b & 15, b >> 4], -1).reshape(w.shape[0], -1).to(torch.int8)
        w = torch.where(n > 7, n - 16, n)
    mean = x.mean(1) if center else None
    z = x - mean[:, None] if center else x
    for sign, gather in s["rounds"]:
        z = ((z[:, gather] * sign).view(x.shape[0], -1, s["H"].shape[0]) @ s["H"]).view_as(x)
    alpha = z.abs().amax(1).clamp_min(EPS) / 127
    y = (torch.round(z / alpha[:, None]) @ w.float().T) * alpha[:, None] * s["ws"][None, :]
    if center:
        y = y + mean[:, None] * s["w1"][None, :]
    return y if s["bias"] is None else y + s["bias"].float()


def _plain_heads(x, c, s, weight, bias):
    """The norm and the rotation of [B, S, heads, D] in float32."""
    x = x.float()
    if c["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight
    if bias is not None:
        x = x + bias
    rot, pos = c["rot"], s["pos"].long()
    free = (pos < 0)[..., None, None]
    cos = torch.where(free, 1.0, s["cos"][pos.clamp_min(0)][:, :, None, :])
    sin = torch.where(free, 0.0, s["sin"][pos.clamp_min(0)][:, :, None, :])
    if c["rope"] == "pairs":
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def run(s):
    c = s["case"]
    if own:
        import w4a8_ptq_linear_b200 as oq
    if c["op"] == "gemm":
        if own:
            return oq.gemm_w8a8(s["a"], s["scale"], s["w"], s["ws"], mean=s["mean"],
                                w_rowsum=s["w1"], bias=s["bias"],
                                out_kind=oq.OUT_ACC if c["out"] == "acc" else oq.OUT_BF16)
        if c["out"] == "acc":  # whole numbers up to 2^31: exact in 64 bits
            return (s["a"].double() @ s["w"].double().T).to(torch.int32)
        y = (s["a"].float() @ s["w"].float().T) * s["scale"][:, None] * s["ws"][None, :]
        if c["mean"]:
            y = y + s["mean"][:, None] * s["w1"][None, :]
        return (y + s["bias"].float() if c["bias"] else y).bfloat16()
    if c["op"] == "linear":
        if own:
            return oq.linear_w8a8(s["plan"], s["x"], s["w"], s["ws"], s["w1"], s["bias"])
        return _plain_linear(s, c["center"]).bfloat16()
    if c["op"] == "heads":
        q, k = s["q"], s["k"]
        if own:
            outs = {}
            if c["heads_first"]:  # [B, heads, S, D] in memory, as an attention reads it
                outs = {n: torch.empty(c["B"], t.shape[2], c["S"], c["D"], dtype=torch.bfloat16,
                                       device=t.device).transpose(1, 2)
                        for n, t in (("q_out", q), ("k_out", k))}
            return oq.qk_norm_rope(s["heads"], q, k, positions=s["pos"], **outs)
        outs = (_plain_heads(q, c, s, s["qw"], s["qb"]), _plain_heads(k, c, s, s["kw"], s["kb"]))
        if c["heads_first"]:
            outs = [o.transpose(1, 2).bfloat16().contiguous().transpose(1, 2) for o in outs]
        return tuple(o.bfloat16() for o in outs)
    if own:
        return oq.linear_qkv(s["plan"], s["heads"], s["x"], s["w"], s["ws"], s["w1"], s["bias"],
                             positions=s["pos"])
    y = _plain_linear(s, c["center"])
    T, a, b = y.shape[0], c["Hq"] * c["D"], (c["Hq"] + c["Hk"]) * c["D"]
    q = _plain_heads(y[:, :a].view(c["B"], c["S"], c["Hq"], c["D"]), c, s, s["qw"], s["qb"])
    k = _plain_heads(y[:, a:b].view(c["B"], c["S"], c["Hk"], c["D"]), c, s, s["kw"], s["kb"])
    return torch.cat([q.reshape(T, a), k.reshape(T, b - a), y[:, b:]], 1).bfloat16()


# ---- work -------------------------------------------------------------------------------------

def _angles(c):
    """Bytes of the angles: a row for each position of a sequence, the sequences' are the same."""
    return 4 * c["rot"] * (c["S"] if c["S"] > 1 else c["B"])


def work(case):
    c = case
    if c["op"] == "gemm":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": T * K + N * K + T * N * (4 if c["out"] == "acc" else 2) + 8 * T + 10 * N,
                "flops": 2 * T * K * N}
    if c["op"] == "heads":
        T, H, D = c["B"] * c["S"], c["Hq"] + c["Hk"], c["D"]
        return {"bytes": 4 * T * H * D + 4 * T + _angles(c), "flops": 8 * T * H * D}
    if c["op"] == "linear":
        T, d, N, bits = c["T"], c["d"], c["N"], 8
        heads = 0
    else:
        T, d, N, bits = c["B"] * c["S"], c["d"], (c["Hq"] + 2 * c["Hk"]) * c["D"], c["bits"]
        heads = 4 * T + _angles(c)
    rounds = 2 if _block(d) < 512 else 1
    return {"bytes": 2 * T * d + N * d * bits // 8 + 2 * T * N + 10 * N + heads,
            "flops": 2 * T * d * N + rounds * T * d * (int(math.log2(_block(d))) + 1)}


# ---- the operators by definition, in 64 bits ------------------------------------------------------

MASK = (1 << 64) - 1


def _counter(key, i):
    """Output i of a SplitMix64 generator with the given key, in whole numbers."""
    z = (key + (i + 1) * 0x9E3779B97F4A7C15) & MASK
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & MASK
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & MASK
    return z ^ (z >> 31)


def _exact_rotate(z, h, seed):
    """The rotation by butterflies, one round after the other."""
    T, d = z.shape
    for r in range(2 if h < 512 else 1):
        ks, kp = _counter(seed, 2 * r), _counter(seed, 2 * r + 1)
        order = sorted(range(d), key=lambda i: _counter(kp, i))
        sign = [-1.0 if _counter(ks, i) >> 63 else 1.0 for i in range(d)]
        z = z[:, torch.tensor(order, device=z.device)] * torch.tensor(sign, dtype=torch.float64, device=z.device)
        step = 1
        while step < h:
            p = z.view(T, d // (2 * step), 2, step)
            z = torch.stack([p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]], 2).view(T, d)
            step *= 2
        z = z / math.sqrt(h)
    return z


def _exact_product(a, w):
    """sum over k of a[t, k] w[o, k], a slice of k at a time."""
    out = torch.zeros(a.shape[0], w.shape[0], dtype=torch.float64, device=a.device)
    for k in range(0, a.shape[1], 1024):
        out.addmm_(a[:, k:k + 1024].double(), w[:, k:k + 1024].double().t())
    return out


def _exact_linear(s, seed, d, center):
    x = s["x"].double()
    mean = x.sum(1, keepdim=True) / d
    z = _exact_rotate(x - mean if center else x, _block(d), int(seed))
    alpha = torch.clamp(z.abs().max(1, keepdim=True).values, min=EPS) / 127
    w = s["w"]
    if w.dtype == torch.uint8:
        full = torch.empty(w.shape[0], w.shape[1] // 16, 32, dtype=torch.float64, device=w.device)
        n = w.view(w.shape[0], -1, 16).long()
        full[:, :, :16], full[:, :, 16:] = n % 16, n // 16
        w = (full - 16 * (full >= 8)).view(w.shape[0], -1)
    y = _exact_product(torch.round(z / alpha), w) * alpha * s["ws"].double()
    if center:
        y += mean * s["w1"].double()
    if s["bias"] is not None:
        y += s["bias"].double()
    return y


def _exact_heads(x, c, s, weight, bias):
    x = x.double()
    D, rot = c["D"], c["rot"]
    if c["norm"] == "layer":
        x = x - x.sum(-1, keepdim=True) / D
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + s["eps"]) * weight.double()
    if bias is not None:
        x = x + bias.double()
    pos = s["pos"].long()
    turn = torch.complex(s["cos"].double(), s["sin"].double())[pos.clamp(min=0)]
    turn = torch.where((pos < 0)[..., None], torch.ones_like(turn), turn)[:, :, None, :]
    if c["rope"] == "pairs":
        i, j = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    else:
        i, j = torch.arange(rot // 2), torch.arange(rot // 2, rot)
    i, j = i.to(x.device), j.to(x.device)
    z = torch.complex(x[..., i], x[..., j]) * turn
    out = x.clone()
    out[..., i], out[..., j] = z.real, z.imag
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gemm":
        y = _exact_product(s["a"], s["w"])
        if c["out"] == "acc":
            return y.to(torch.int32)
        y *= s["scale"].double()[:, None] * s["ws"].double()[None, :]
        if c["mean"]:
            y += torch.outer(s["mean"].double(), s["w1"].double())
        if c["bias"]:
            y += s["bias"].double()
        return y
    if c["op"] == "linear":
        return _exact_linear(s, seed, c["d"], c["center"])
    if c["op"] == "heads":
        return (_exact_heads(s["q"], c, s, s["qw"], s["qb"]),
                _exact_heads(s["k"], c, s, s["kw"], s["kb"]))
    y = _exact_linear(s, seed, c["d"], c["center"])
    B, S, Hq, Hk, D = c["B"], c["S"], c["Hq"], c["Hk"], c["D"]
    q, k, v = y.split([Hq * D, Hk * D, Hk * D], 1)
    q = _exact_heads(q.reshape(B, S, Hq, D), c, s, s["qw"], s["qb"])
    k = _exact_heads(k.reshape(B, S, Hk, D), c, s, s["kw"], s["kb"])
    return torch.cat([q.reshape(B * S, -1), k.reshape(B * S, -1), v], 1)
