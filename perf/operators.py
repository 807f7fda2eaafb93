"""Work of the 4-bit training operators: microscaled quantisation and its reading back, the linear layer
on it (few tokens, whole prompts, and with its gradients), products over lists of experts, and dropout.

`run` computes each in its plain form, or with `own` by the calls that a training program makes of the
package.  Sizes are those of the package's matrix sets (width 768 and 2560 with 10240-wide feed-forward
matrices, experts of 2048 x 1408) and odd ones.

The number format: blocks of 32 consecutive elements along the contraction index share a scale 2^e, with e
the smallest integer >= -127 for which no element of the block exceeds 6 * 2^e; the elements are
sign * {0, 0.5, 1, 1.5, 2, 3, 4, 6} * 2^e.  A block that holds an infinity or a NaN is all NaN.
Nearest rounding takes ties to the even code; stochastic rounding goes up where 256 times the fraction
exceeds the element's random byte plus a half.  Random numbers are those of Philox 4x32 with ten rounds
(Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), keyed by a 64-bit seed.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}

# third counter word of the generator: what the numbers are for
TAG_DROPOUT, TAG_ROUND, TAG_ROUND_T = 0x44524F50, 0x53523430, 0x53523431


def listed():
    return [
        # one token's activations on their way into a 4-bit product: latency alone
        dict(name="quantize_token", op="quantize", rows=1, cols=2560, dtype="bf16", transpose="no", stochastic=False, count=1),
        # a micro-batch's activations, for the product and (transposed) for the weight gradient
        dict(name="quantize_activations", op="quantize", rows=16384, cols=2560, dtype="bf16", transpose="both", stochastic=False, count=1),
        # output gradients of a feed-forward matrix, rounded stochastically, both ways
        dict(name="quantize_gradients", op="quantize", rows=8192, cols=10240, dtype="bf16", transpose="both", stochastic=True, count=1),
        # a layer for one token, and for a few
        dict(name="linear_token", op="linear", tokens=1, cols=2560, outs=10240, dtype="bf16"),
        dict(name="linear_few_tokens", op="linear", tokens=13, cols=10240, outs=2560, dtype="bf16"),
        # a prompt of odd length through the same layer
        dict(name="linear_prompt", op="linear", tokens=8191, cols=2560, outs=10240, dtype="bf16"),
        # a small layer of sizes that divide nothing, fp32 activations, with its gradients
        dict(name="train_odd", op="train", tokens=1001, cols=333, outs=777, dtype="f32", dropout=0.1),
        # a micro-batch through a feed-forward matrix and back
        dict(name="train_large", op="train", tokens=16384, cols=2560, outs=10240, dtype="bf16", dropout=0.1),
        # 64 experts, each with its own tokens (some with none): forward products of one layer
        dict(name="experts_forward", op="experts", count=64, tokens=16384, cols=2048, outs=1408, dtype="bf16", gradient=False, spread=1),
        # weight gradients of twelve attention matrices, kept in fp32 for the optimizer
        dict(name="weight_gradients", op="experts", count=12, tokens=98304, cols=768, outs=768, dtype="bf16", gradient=True, spread=2),
        # dropout of a short odd batch, and of a micro-batch's residual stream, with the gradient's
        dict(name="dropout_small", op="dropout", rows=37, cols=333, dtype="f32", dropout=0.1),
        dict(name="dropout_stream", op="dropout", rows=16384, cols=2560, dtype="bf16", dropout=0.1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "train", "experts", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "quantize":
        cols, count = _log(rng, 8, 10240), rng.choice([1, 1, 2, 5])
        return dict(op=op, rows=_log(rng, 1, min(16384, 8192 * 10240 // (cols * count))), cols=cols, dtype=dtype,
                    transpose=rng.choice(["no", "yes", "both"]), stochastic=rng.random() < 0.5, count=count)
    if op == "linear":
        return dict(op=op, tokens=_log(rng, 1, 8192), cols=_log(rng, 64, 10240), outs=_log(rng, 64, 2560), dtype=dtype)
    if op == "train":
        return dict(op=op, tokens=_log(rng, 16, 16384), cols=_log(rng, 64, 2560), outs=_log(rng, 64, 10240), dtype=dtype,
                    dropout=rng.choice([0.0, 0.1, 0.25]))
    if op == "experts":
        count = rng.randint(2, 64)
        return dict(op=op, count=count, tokens=_log(rng, count, 16384), cols=_log(rng, 64, 2048), outs=_log(rng, 64, 2048),
                    dtype=dtype, gradient=rng.random() < 0.5, spread=rng.randrange(1000))
    return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 8, 2560), dtype=dtype, dropout=round(rng.uniform(0.02, 0.5), 3))


def _token_counts(case):
    """Tokens per expert: uneven, some experts with none; their sum is the case's."""
    g = np.random.default_rng(case["spread"])
    share = g.gamma(1.0, size=case["count"])
    if case["count"] > 8 and not case["gradient"]:
        share[g.choice(case["count"], 2, replace=False)] = 0
    edges = np.floor(np.cumsum(share) / share.sum() * case["tokens"] + 0.5).astype(np.int64)
    return np.diff(np.concatenate([[0], edges])).tolist()


def _inputs(case, seed):
    """The case's tensors and seeds."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def activations(rows, cols):   # channels of very different size, as a network's are
        size = torch.exp(torch.randn(cols, generator=g, device="cuda"))
        return (torch.randn(rows, cols, generator=g, device="cuda") * size).to(dt)

    def gradients(rows, cols):
        return (torch.randn(rows, cols, generator=g, device="cuda") * 1e-3).to(dt)

    def weights(rows, cols):
        return (torch.randn(rows, cols, generator=g, device="cuda") * 0.02).to(BF16)

    op, s = case["op"], {"seed": int(seed) * 1000003 + 17, "round_seed": int(seed) * 7919 + 5}
    if op == "quantize":
        make = gradients if case["stochastic"] else activations
        s["x"] = [make(case["rows"], case["cols"]) for _ in range(case["count"])]
    elif op == "linear":
        s["x"], s["weight"] = activations(case["tokens"], case["cols"]), weights(case["outs"], case["cols"])
    elif op == "train":
        s["x"], s["weight"] = activations(case["tokens"], case["cols"]), weights(case["outs"], case["cols"])
        s["dy"] = gradients(case["tokens"], case["outs"])
    elif op == "experts":
        n = _token_counts(case)
        s["x"] = [activations(t, case["cols"]) for t in n]
        if case["gradient"]:
            s["dy"] = [gradients(t, case["outs"]) for t in n]
        else:
            s["weight"] = [weights(case["outs"], case["cols"]) for _ in n]
    else:
        s["x"], s["dy"] = activations(case["rows"], case["cols"]), gradients(case["rows"], case["cols"])
    return s


def prepare(case, seed):
    """Inputs, and the weights as a program keeps them: in 4 bits (codes and scale bytes, or the package's handle)."""
    s = {"case": dict(case), **_inputs(case, seed)}
    if "weight" in s:
        w = s.pop("weight")
        if own:
            import orthogonalising_matrix_optimizer_amd as mo
            s["w"] = mo.mx_quantize(w, transpose="both" if case["op"] == "train" else False)
        else:
            s["w"] = [_encode(v) for v in w] if case["op"] == "experts" else _encode(w)
            s["wt"] = _encode(w.t()) if case["op"] == "train" else None
    return s


# ---------------------------------------------------------------- plain forms
def _philox(c0, c1, tag, c3, seed):
    """The four words (as int64 tensors in [0, 2^32)) of the counters (c0, c1, tag, c3)."""
    m = 0xFFFFFFFF
    x = [c0, c1, torch.full_like(c0, tag), torch.full_like(c0, c3)]
    k0, k1 = seed & m, (seed >> 32) & m
    for r in range(10):
        p0, p1 = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [((p1 >> 32) & m) ^ x[1] ^ k0, p1 & m, ((p0 >> 32) & m) ^ x[3] ^ k1, p0 & m]
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return x


def _randoms(rows, cols, bits, tag, which, seed, device):
    """Random integers of `bits` bits for a rows x cols array: 128 / bits consecutive elements of a row share a counter
    (group in the row, row, tag, index in the list)."""
    per = 128 // bits
    groups = -(-cols // per)
    c1, c0 = torch.meshgrid(torch.arange(rows, device=device), torch.arange(groups, device=device), indexing="ij")
    words = torch.stack(_philox(c0, c1, tag, which, seed), dim=-1)
    shifts = torch.arange(0, 32, bits, device=device)
    return ((words.unsqueeze(-1) >> shifts) & ((1 << bits) - 1)).reshape(rows, groups * per)[:, :cols]


def _power(byte):
    """2^(byte - 127) in fp32, exactly."""
    return torch.where(byte > 0, byte << 23, torch.full_like(byte, 1 << 22)).to(torch.int32).view(F32)


def _quantized(x, r8=None):
    """(magnitude code, negative, scale byte as int64 with 255 for NaN) of the blocks of a 2-D x: [rows, blocks, 32]."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    pad = (0, 32 * nb - cols)
    v = torch.nn.functional.pad(x.to(F32), pad).reshape(rows, nb, 32)
    top = v.abs().amax(-1)
    byte = torch.clamp(((top.view(torch.int32).to(torch.int64) + 0x3FFFFF) >> 23) - 2, min=0)
    a = v.abs() * _power(254 - torch.clamp(byte, max=253)).unsqueeze(-1)
    octave = (a >= 2).to(F32) + (a >= 4).to(F32)
    q = a * torch.where(a >= 4, 0.5, torch.where(a >= 2, 1.0, 2.0))
    if r8 is None:
        m = torch.round(q)
    else:
        low = torch.floor(q)
        r = torch.nn.functional.pad(r8, pad).reshape(rows, nb, 32).to(F32)
        m = low + ((q - low) * 256 > r + 0.5).to(F32)
    bad = ~torch.isfinite(top)
    code = torch.where(bad.unsqueeze(-1), 0.0, m + 2 * octave)
    return code.to(torch.int64), v < 0, torch.where(bad, 255, byte)


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(code, negative, byte, cols):
    """The fp32 values that codes and scales stand for."""
    rows, width = code.shape[0], 32 * code.shape[1]
    grid = torch.tensor(_GRID, device=code.device)
    scale = torch.where(byte == 255, math.nan, _power(torch.clamp(byte, max=254)))
    v = grid[code] * torch.where(negative, -1.0, 1.0) * scale.unsqueeze(-1)
    return v.reshape(rows, width)[:, :cols]


def _rounded(x, seed=None, tag=TAG_ROUND, which=0):
    """fp32 values of x after quantisation along its rows."""
    r8 = None if seed is None else _randoms(x.shape[0], x.shape[1], 8, tag, which, seed, x.device)
    return _values(*_quantized(x, r8), x.shape[1])


def _encode(x):
    """4-bit storage of x: packed codes, scale bytes, columns."""
    code, negative, byte = _quantized(x)
    nibble = (code + 8 * negative.to(torch.int64)).reshape(x.shape[0], 16 * code.shape[1], 2)
    return (nibble[..., 0] + 16 * nibble[..., 1]).to(torch.uint8), byte.to(torch.uint8), x.shape[1]


def _decode(e):
    packed, byte, cols = e
    nibble = torch.stack([packed & 15, packed >> 4], dim=-1).to(torch.int64).reshape(*byte.shape, 32)
    return _values(nibble & 7, nibble >= 8, byte.to(torch.int64), cols)


def _dropped(x, p, seed):
    """x (fp32 values, unrounded) with its dropped elements zeroed and the others scaled by 1 / (1 - p), p in steps of 2^-16."""
    t = math.floor(p * 65536 + 0.5)
    keep = _randoms(x.shape[0], x.shape[1], 16, TAG_DROPOUT, 0, seed, x.device) >= t
    scale = torch.tensor(65536.0, device=x.device) / (65536 - t)
    return torch.where(keep, x.to(F32) * scale, 0.0)


def _run_plain(s):
    case, x = s["case"], s["x"]
    op = case["op"]
    if op == "quantize":
        out = []
        for i, v in enumerate(x):
            seed = s["round_seed"] if case["stochastic"] else None
            if case["transpose"] != "yes":
                out.append(_rounded(v, seed, TAG_ROUND, i).to(BF16))
            if case["transpose"] != "no":
                out.append(_rounded(v.t(), seed, TAG_ROUND_T, i).to(BF16))
        return out
    if op == "linear":
        return (_rounded(x) @ _decode(s["w"]).t()).to(x.dtype)
    if op == "train":
        p, dy = case["dropout"], s["dy"]
        xd = _dropped(x, p, s["seed"]).to(x.dtype) if p else x
        y = _rounded(xd) @ _decode(s["w"]).t()
        dx = _rounded(dy, s["round_seed"], TAG_ROUND) @ _decode(s["wt"]).t()
        dw = _rounded(dy.t(), s["round_seed"], TAG_ROUND_T) @ _rounded(xd.t()).t()
        dx = _dropped(dx, p, s["seed"]) if p else dx
        return y.to(x.dtype), dx.to(dy.dtype), dw
    if op == "experts":
        if case["gradient"]:
            return [_rounded(d.t(), s["round_seed"], TAG_ROUND_T, i) @ _rounded(v.t()).t()
                    for i, (v, d) in enumerate(zip(x, s["dy"]))]
        return [(_rounded(v) @ _decode(w).t()).to(v.dtype) for v, w in zip(x, s["w"])]
    p = case["dropout"]
    return _dropped(x, p, s["seed"]).to(x.dtype), _dropped(s["dy"], p, s["seed"]).to(x.dtype)


# ---------------------------------------------------------------- the package's calls
def _run_own(s):
    import orthogonalising_matrix_optimizer_amd as mo
    case, x = s["case"], s["x"]
    op = case["op"]
    if op == "quantize":
        q = mo.mx_quantize(x, transpose={"no": False, "yes": True, "both": "both"}[case["transpose"]],
                           seed=s["round_seed"] if case["stochastic"] else None)
        return mo.mx_dequantize([m for pair in q for m in pair] if case["transpose"] == "both" else q)
    if op == "linear":
        return mo.mx_linear(x, s["w"])
    if op == "train":
        w, wt = s["w"]
        y, saved = mo.mx_linear(x, w, save=True, dropout=case["dropout"], dropout_seed=s["seed"])
        dx, dw = mo.mx_linear_grad(s["dy"], wt, saved, seed=s["round_seed"])
        return y, dx, dw
    if op == "experts":
        if case["gradient"]:
            return mo.mx_matmul(mo.mx_quantize(s["dy"], transpose=True, seed=s["round_seed"]),
                                mo.mx_quantize(x, transpose=True), dtype=F32)
        return mo.mx_matmul(mo.mx_quantize(x), s["w"], dtype=DTYPES[case["dtype"]])
    return mo.dropout(x, case["dropout"], s["seed"]), mo.dropout(s["dy"], case["dropout"], s["seed"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def _held(rows, cols):
    """Bytes of a 4-bit matrix: half a byte an element and one a block."""
    return rows * (-(-cols // 32)) * 17


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("quantize", "dropout"):
        n = case["rows"] * case["cols"]
        if op == "dropout":
            return {"bytes": 4 * n * es, "flops": 0}
        n *= case["count"]
        return {"bytes": n * (es + (4 if case["transpose"] == "both" else 2)), "flops": 0}
    t, k, n = case["tokens"], case["cols"], case["outs"]
    if op == "linear":
        return {"bytes": es * t * (k + n) + _held(n, k), "flops": 2 * t * k * n}
    if op == "train":
        return {"bytes": 2 * es * t * (k + n) + _held(n, k) + _held(k, n) + 4 * n * k, "flops": 6 * t * k * n}
    if case["gradient"]:
        return {"bytes": es * t * (k + n) + 4 * case["count"] * n * k, "flops": 2 * t * k * n}
    return {"bytes": es * t * (k + n) + case["count"] * _held(n, k), "flops": 2 * t * k * n}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_random(rows, cols, bits, tag, which, seed):
    """The generator once more, on the host in unsigned 64-bit words, a strip of rows at a time."""
    per, low32 = 128 // bits, np.uint64(0xFFFFFFFF)
    groups = -(-cols // per)
    out = np.empty((rows, groups, 4), np.uint32)
    strip = max(1, (1 << 20) // max(1, groups))
    for r0 in range(0, rows, strip):
        r1 = min(rows, r0 + strip)
        w = [np.broadcast_to(np.arange(groups, dtype=np.uint64), (r1 - r0, groups)),
             np.broadcast_to(np.arange(r0, r1, dtype=np.uint64)[:, None], (r1 - r0, groups)), np.uint64(tag), np.uint64(which)]
        ka, kb = seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF
        for _ in range(10):
            left, right = w[0] * np.uint64(0xD2511F53), w[2] * np.uint64(0xCD9E8D57)
            w = [right >> np.uint64(32) ^ w[1] ^ np.uint64(ka), right & low32, left >> np.uint64(32) ^ w[3] ^ np.uint64(kb), left & low32]
            ka, kb = ka + 0x9E3779B9 & 0xFFFFFFFF, kb + 0xBB67AE85 & 0xFFFFFFFF
        for i in range(4):
            out[r0:r1, :, i] = w[i]
    kind = np.uint8 if bits == 8 else np.uint16
    v = out.reshape(rows, groups * 4).view(kind)[:, :cols]
    return torch.from_numpy(v.astype(np.int32)).cuda()


def _times_power(v, e):
    """v * 2^e in float64, exactly (|e| < 1000)."""
    return v * ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_rounded(x, random=None):
    """Values in float64 after quantisation along the rows, by looking the grid up."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    rows, cols = x.shape
    v = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    if v.numel() == 0:
        return v[:, :cols]
    v = v.view(rows, -1, 32)
    share, e = torch.frexp(v.abs().max(dim=2, keepdim=True).values / 6)
    e = torch.where(share == 0.5, e - 1, e).clamp(min=-127)
    e = torch.where(share == 0, -127, e)
    t = _times_power(v, -e)
    a = t.abs().contiguous()
    if random is None:
        middle = (grid[1:] + grid[:-1]) / 2
        i = torch.bucketize(a, middle)
        i = i + ((a == middle[i.clamp(max=6)]) & (i % 2 == 1)).long()
    else:
        r = torch.zeros(rows, v.shape[1] * 32, dtype=torch.float64, device=x.device)
        r[:, :cols] = random
        i = torch.bucketize(a, grid, right=True) - 1
        above = grid[(i + 1).clamp(max=7)]
        part = torch.where(i < 7, (a - grid[i]) / (above - grid[i]).clamp(min=0.5), 0)
        i = i + (part * 256 > r.view_as(a) + 0.5).long()
    return _times_power(torch.copysign(grid[i], t), e).view(rows, -1)[:, :cols]


def _exact_dropped(x, p, seed):
    gone = int(math.floor(p * 65536 + 0.5))
    random = _exact_random(x.shape[0], x.shape[1], 16, TAG_DROPOUT, 0, seed)
    return x.double() * (65536 / (65536 - gone)) * (random >= gone)


def exact(case, seed):
    s = _inputs(case, seed)
    x, op = s["x"], case["op"]
    if op == "quantize":
        out = []
        for i, v in enumerate(x):
            for turn, tag in ((False, TAG_ROUND), (True, TAG_ROUND_T)):
                if case["transpose"] in (("yes", "both") if turn else ("no", "both")):
                    u = v.t().contiguous() if turn else v
                    random = _exact_random(u.shape[0], u.shape[1], 8, tag, i, s["round_seed"]) if case["stochastic"] else None
                    out.append(_exact_rounded(u, random))
        return out
    if op == "linear":
        return torch.mm(_exact_rounded(x), _exact_rounded(s["weight"]).t().contiguous())
    if op == "train":
        p, dy, w = case["dropout"], s["dy"], s["weight"]
        xd = x.double()
        if p:   # the values are kept in the activations' type
            xd = _exact_dropped(x, p, s["seed"]).float().to(x.dtype).double()
        dyt, xt = dy.t().contiguous(), xd.t().contiguous()
        y = torch.mm(_exact_rounded(xd), _exact_rounded(w).t().contiguous())
        by_row = _exact_random(dy.shape[0], dy.shape[1], 8, TAG_ROUND, 0, s["round_seed"])
        dx = torch.mm(_exact_rounded(dy, by_row), _exact_rounded(w.t().contiguous()).t().contiguous())
        del by_row
        by_col = _exact_random(dyt.shape[0], dyt.shape[1], 8, TAG_ROUND_T, 0, s["round_seed"])
        dw = torch.mm(_exact_rounded(dyt, by_col), _exact_rounded(xt).t().contiguous())
        return y, _exact_dropped(dx, p, s["seed"]) if p else dx, dw
    if op == "experts":
        if case["gradient"]:
            return [torch.mm(_exact_rounded(d.t().contiguous(), _exact_random(d.shape[1], d.shape[0], 8, TAG_ROUND_T, i, s["round_seed"])),
                             _exact_rounded(v.t().contiguous()).t().contiguous()) for i, (v, d) in enumerate(zip(x, s["dy"]))]
        return [torch.mm(_exact_rounded(v), _exact_rounded(w).t().contiguous()) for v, w in zip(x, s["weight"])]
    return _exact_dropped(x, case["dropout"], s["seed"]), _exact_dropped(s["dy"], case["dropout"], s["seed"])
