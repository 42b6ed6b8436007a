"""Operators of a fine-tuned block's feed-forward part, as cases for measurement: the
product in 8-bit floating point with a scale for each block of 128, the gated block over
frozen NF4 weights with its backward pass, and the layer with dropout whose mask is
drawn from a counter and never stored, forward and backward.

``run`` computes each operator either in its plain form (elementary torch operations
in fp32) or, with ``own`` set, through the package's entry points.

The definitions both share:
  8-bit floats   a block's scale is the smallest power of two s = 2^e, e >= -127, with
                 max |x| <= 448 s; codes are x / s rounded to nearest even into e4m3 (4 exponent
                 bits, 3 mantissa bits, largest value 448).  Blocks are 128 consecutive columns
                 of one row of x, and 128 x 128 of the weight.
  product        y[i, j] = sum_k xq[i, k] wq[j, k] (+ bias[j]) over the values the codes stand for
  NF4 weight     W = round_cd(fl32(level[code] scale)), level the 16 normal quantiles, scale a
                 block's largest magnitude (blocks of 64), or q S with u8 q and one fp32 S for
                 each 256 blocks
  gated block    g = x Wg^T + s (x Ag^T) Bg^T (+ bias), u likewise, h = act(g) u
                 backward, from the saved g and u: dg = dh u act'(g), du = dh act(g), and the
                 gradients of the two projections with respect to x, A and B
  dropout        keep[i, k] = w >= round(65536 p), w the 16-bit half k % 8 (low halves first) of the four
                 words that Philox 4x32-10 (Salmon et al., SC 2011) gives for the counter
                 (k // 8, i, offset low, offset high) and the key (seed low, seed high);
                 y = x W^T + s / (1 - p) (x keep A^T) B^T (+ bias), with p a multiple of 1 / 65536
"""
import math
import random
import statistics

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_ACTS = ("silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------------- cases
def _fp8(m, rows, cols, cd, bias=False):
    return {"op": "fp8", "m": m, "rows": rows, "cols": cols, "cd": cd, "bias": bias}


def _gated(way, m, rows, cols, r, cd, act="silu", dq=True, bias=False, save=False):
    return {"op": "gated_" + way, "m": m, "rows": rows, "cols": cols, "r": r, "cd": cd, "act": act, "dq": dq,
            "bias": bias, "save": save}


def _dropout(way, m, rows, cols, r, cd, p, dq=True, bias=False):
    return {"op": "dropout_" + way, "m": m, "rows": rows, "cols": cols, "r": r, "cd": cd, "p": p, "dq": dq,
            "bias": bias}


def listed():
    cases = [
        # one token through a merged attention projection: the weight's read, and latency
        ("fp8_one_token", _fp8(1, 4096, 4096, "bf16")),
        # one token each of 16 sequences through an MLP projection
        ("fp8_decode_batch", _fp8(16, 14336, 4096, "bf16", bias=True)),
        # a short prompt through a layer whose sizes suit no tile and end inside a block
        ("fp8_odd", _fp8(333, 1003, 2047, "f16", bias=True)),
        # a long prompt through the widest projection
        ("fp8_prompt", _fp8(4096, 14336, 4096, "bf16")),
        # one token of an adapter that is not merged
        ("gated_one_token", _gated("fwd", 1, 14336, 4096, 16, "bf16")),
        # a short training sequence, another activation, sizes that suit no tile
        ("gated_odd", _gated("fwd", 300, 1000, 704, 12, "f16", act="gelu", dq=False, bias=True, save=True)),
        # the MLP of a training step
        ("gated_train", _gated("fwd", 4096, 14336, 4096, 64, "bf16", save=True)),
        # fp32 training of a small model
        ("gated_bwd_small", _gated("bwd", 77, 512, 256, 8, "f32", act="gelu_tanh", dq=False)),
        # the MLP of a training step, backward
        ("gated_bwd_train", _gated("bwd", 4096, 14336, 4096, 64, "bf16")),
        # one GPU's share of a batch, an attention projection
        ("dropout_share", _dropout("fwd", 512, 4096, 4096, 16, "bf16", 0.05)),
        # sizes that suit no tile, heavy dropout
        ("dropout_bwd_odd", _dropout("bwd", 333, 1000, 704, 8, "f16", 0.5, dq=False)),
        # the down projection of a training step, backward
        ("dropout_bwd_train", _dropout("bwd", 4096, 4096, 14336, 64, "bf16", 0.1)),
    ]
    return [dict(c, name=name) for name, c in cases]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v > 64:  # half of the sizes are whole tiles, half are odd
        v = max(64, v // 64 * 64)
    return max(lo, min(hi, v))


def draw(rng):
    limit = {}
    for c in listed():
        w = work(c)
        limit[c["op"]] = max(limit.get(c["op"], 0), w["flops"] + 200 * w["bytes"])
    while True:
        op = rng.choice(["fp8", "fp8", "gated_fwd", "gated_bwd", "dropout_fwd", "dropout_bwd"])
        cd = rng.choice(["bf16", "bf16", "f16", "f32"])
        m, rows, cols = _log_int(rng, 1, 4096), _log_int(rng, 64, 14336), _log_int(rng, 64, 14336)
        bias = rng.random() < 0.4
        if op == "fp8":
            case = _fp8(m, rows, cols, cd, bias)
        else:
            if rng.random() < 0.7:
                cols = max(64, cols // 64 * 64)
            if cols % 64:  # whole blocks of 64 in all
                rows = max(64, rows // 64 * 64)
            r, dq = rng.choice([4, 8, 16, 32, 64, _log_int(rng, 1, 64)]), rng.random() < 0.5
            if op == "gated_fwd":
                case = _gated("fwd", m, rows, cols, r, cd, rng.choice(_ACTS), dq, bias, rng.random() < 0.7)
            elif op == "gated_bwd":
                case = _gated("bwd", m, rows, cols, r, cd, rng.choice(_ACTS), dq)
            else:
                case = _dropout(op[8:], m, rows, cols, r, cd, rng.choice([0.05, 0.1, 0.25, 0.5]), dq,
                                bias and op == "dropout_fwd")
        w = work(case)
        if w["flops"] + 200 * w["bytes"] <= limit[op]:
            return case


def work(case):
    b, m, n, k = _BYTES[case["cd"]], case["m"], case["rows"], case["cols"]
    bias = n * b if case.get("bias") else 0
    if case["op"] == "fp8":
        return {"bytes": m * k * b + n * k + -(-n // 128) * -(-k // 128) + m * n * b + bias, "flops": 2 * m * n * k}
    r = case["r"]
    weight = n * k // 2 + (n * k // 64 * (1 + 4 / 256) if case["dq"] else n * k // 64 * 4) + r * (n + k) * b
    if case["op"] == "gated_fwd":
        saved = 2 * m * n * b + 2 * m * r * 4 if case["save"] else 0
        return {"bytes": m * k * b + 2 * (weight + bias) + m * n * b + saved, "flops": 4 * m * (n * k + r * (n + k))}
    if case["op"] == "gated_bwd":
        return {"bytes": 2 * m * k * b + 3 * m * n * b + 2 * m * r * 4 + 2 * (weight + r * (n + k) * b),
                "flops": 4 * m * (n * k + 2 * r * (n + k))}
    if case["op"] == "dropout_fwd":
        return {"bytes": m * k * b + weight + bias + m * n * b + m * r * 4, "flops": 2 * m * (n * k + r * (n + k))}
    return {"bytes": 2 * m * k * b + m * n * b + m * r * 4 + weight + r * (n + k) * b,
            "flops": 2 * m * (n * k + 2 * r * (n + k))}


# ------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _hidden(g, m, k, cd):
    # hidden states after a norm: unit variance, a few channels much larger than the rest
    gain = torch.ones(k, device="cuda")
    gain[torch.randperm(k, generator=g, device="cuda")[: max(1, k // 200)]] = 12.0
    return (_randn(g, m, k) * gain).to(_TYPES[cd])


def _levels():
    """The 16 NF4 levels: evenly spaced probabilities of the normal distribution, 8 positive
    ones and 7 negative ones beside zero, the outermost at a mean tail offset, scaled to 1."""
    inv = statistics.NormalDist().inv_cdf
    off = 0.5 * (1 - 1 / 30) + 0.5 * (1 - 1 / 32)
    up = [inv(off - j * (off - 0.5) / 8) for j in range(8)]
    down = [-inv(off - j * (off - 0.5) / 7) for j in range(7)]
    return torch.tensor([v / inv(off) for v in sorted(down + [0.0] + up)], dtype=torch.float64).float().cuda()


def _nf4(g, rows, cols, dq):
    """Packed codes and scales of a weight N(0, 0.02^2): what a program keeps after quantizing."""
    levels = _levels()
    middle = (levels[1:].double() + levels[:-1].double()) / 2
    blocks = _randn(g, rows * cols // 64, 64) * 0.02
    absmax = blocks.abs().amax(dim=1)
    blocks = blocks / absmax[:, None]
    code = torch.empty(blocks.shape, dtype=torch.uint8, device="cuda")
    for i in range(0, blocks.shape[0], 1 << 18):
        code[i:i + (1 << 18)] = torch.bucketize(blocks[i:i + (1 << 18)], middle.float()).to(torch.uint8)
    code = code.view(-1, 2)
    w = {"rows": rows, "cols": cols, "dq": dq, "levels": levels, "codes": code[:, 0] * 16 + code[:, 1]}
    if not dq:
        return dict(w, absmax=absmax)
    pad = torch.nn.functional.pad(absmax, (0, -absmax.numel() % 256)).view(-1, 256)
    scale = pad.amax(dim=1) / torch.tensor(255.0, device="cuda")
    q = torch.round(pad / scale[:, None]).clamp(0, 255).to(torch.uint8).view(-1)[: absmax.numel()].contiguous()
    return dict(w, absmax_q=q, absmax_scale2=scale)


def _handle(w):
    if not own:
        return w
    import bit_nf4_quantized_nibble_amd as qn

    return qn.NF4Weight(w["rows"], w["cols"], 64, w["dq"], 256, w["codes"], w.get("absmax"), w.get("absmax_q"),
                        w.get("absmax_scale2"))


def _adapter(g, rows, cols, r, cd):
    return ((_randn(g, r, cols) / math.sqrt(r)).to(_TYPES[cd]), (_randn(g, rows, r) * 0.01).to(_TYPES[cd]))


def prepare(case, seed):
    g = _generator(seed)
    cd = _TYPES[case["cd"]]
    m, n, k, two = case["m"], case["rows"], case["cols"], 2 if case["op"].startswith("gated") else 1
    st = {"case": case, "x": _hidden(g, m, k, case["cd"])}
    st["bias"] = (_randn(g, two * n) * 0.1).to(cd) if case.get("bias") else None
    if case["op"] == "fp8":
        w = (_randn(g, n, k) * (0.01 + 0.02 * torch.rand(n, 1, generator=g, device="cuda"))).to(cd)
        if own:
            import bit_nf4_quantized_nibble_amd as qn

            st["w"] = qn.quantize_fp8(w)
        else:
            st["w"] = _to_fp8(w, 128)
        return st
    r = case["r"]
    plain = [_nf4(g, n, k, case["dq"]) for _ in range(two)]
    st["w"] = [_handle(w) for w in plain]
    st["a"], st["b"] = (list(t) for t in zip(*(_adapter(g, n, k, r, case["cd"]) for _ in range(two))))
    st["alpha"] = 2.0 * r
    if "dropout" in case["op"]:
        st["seed"] = torch.tensor([seed * 7919 + 12345, (seed << 33) + 5], dtype=torch.int64, device="cuda")
    if case["op"] == "gated_bwd":  # what the forward saved
        z, t = _project(plain, st["x"], st["a"], st["b"], 2.0, cd, None)
        st["pre"], st["t"] = z.to(cd), t
        st["dy"] = (_randn(g, m, n) * 0.5).to(cd)
    if case["op"] == "dropout_bwd":
        keep = _keep(m, k, st["seed"], _threshold(case["p"]))
        st["t"] = torch.matmul(torch.where(keep, st["x"].float(), torch.zeros((), device="cuda")), st["a"][0].float().t())
        st["dy"] = _randn(g, m, n).to(cd)
    return st


# --------------------------------------------------------------------- plain form
def _to_fp8(x, tall):
    """The values that the codes of blocks of `tall` rows by 128 columns stand for."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -cols % 128, 0, -rows % tall))
    blocks = x.view(x.shape[0] // tall, tall, x.shape[1] // 128, 128)
    amax = blocks.abs().amax(dim=(1, 3), keepdim=True)
    mantissa, exponent = torch.frexp(amax)  # amax = mantissa 2^exponent, mantissa in [1/2, 1): 448 = 7/8 2^9
    e = torch.where(mantissa <= 0.875, exponent - 9, exponent - 8).clamp(min=-127).long()
    powers = torch.tensor([2.0 ** i for i in range(-127, 128)], device=x.device)  # exact, as torch's pow need not be
    codes = (blocks * powers[127 - e]).to(torch.float8_e4m3fn).float()
    return (codes * powers[127 + e]).view(x.shape)[:rows, :cols].contiguous()


def _weight(w, cd):
    """The NF4 weight's values in the compute type, as fp32."""
    code = torch.stack([w["codes"] >> 4, w["codes"] & 15], dim=1).view(-1, 64)
    if w["dq"]:
        scale = w["absmax_q"].float() * w["absmax_scale2"].repeat_interleave(256)[: w["absmax_q"].numel()]
    else:
        scale = w["absmax"]
    return (w["levels"][code.long()] * scale[:, None]).to(cd).float().view(w["rows"], w["cols"])


def _project(ws, x, a, b, s, cd, bias, tx=None):
    """The projections' outputs side by side and their x A^T; tx: the low-rank branch's input."""
    x = x.float()
    tx = x if tx is None else tx
    t = [torch.matmul(tx, v.float().t()) for v in a]
    z = torch.cat([torch.matmul(x, _weight(w, cd).t()) + s * torch.matmul(t[i], b[i].float().t())
                   for i, w in enumerate(ws)], dim=1)
    return (z if bias is None else z + bias.float()), t


def _act(z, act):
    """The activation and its derivative."""
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return z * q, q * (1 + z * (1 - q))
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    q = 1 / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z * q, q + z * q * (1 - q) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def _threshold(p):
    return int(round(p * 65536))


def _keep(m, k, seed, threshold):
    """The keep mask [m, k] by Philox 4x32-10 on 64-bit integers."""
    low = 0xFFFFFFFF
    words = torch.stack([seed & low, (seed >> 32) & low])  # [low or high, seed or offset]
    key = [words[0, 0], words[1, 0]]
    c = [torch.arange(-(-k // 8), device=seed.device).expand(m, -1),
         torch.arange(m, device=seed.device)[:, None].expand(-1, -(-k // 8)), words[0, 1], words[1, 1]]
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((p1 >> 32) & low) ^ c[1] ^ key[0], p1 & low, ((p0 >> 32) & low) ^ c[3] ^ key[1], p0 & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    halves = [h for w in c for h in (w & 0xFFFF, w >> 16)]
    return (torch.stack(halves, dim=2).view(m, -1)[:, :k] >= threshold)


def _run_plain(st):
    case = st["case"]
    cd = _TYPES[case["cd"]]
    if case["op"] == "fp8":
        y = torch.matmul(_to_fp8(st["x"], 1), st["w"].t())
        return (y if st["bias"] is None else y + st["bias"].float()).to(cd)
    n, s = case["rows"], st["alpha"] / case["r"]
    if case["op"] == "gated_fwd":
        z, t = _project(st["w"], st["x"], st["a"], st["b"], s, cd, st["bias"])
        h = (_act(z[:, :n], case["act"])[0] * z[:, n:]).to(cd)
        return [h, z.to(cd)] + t if case["save"] else h
    x = st["x"].float()
    if case["op"] == "gated_bwd":
        z, dh = st["pre"].float(), st["dy"].float()
        value, slope = _act(z[:, :n], case["act"])
        dz = [dh * z[:, n:] * slope, dh * value]
        dx, grads = 0, []
        for i in range(2):
            dt = s * torch.matmul(dz[i], st["b"][i].float())
            dx = dx + torch.matmul(dz[i], _weight(st["w"][i], cd)) + torch.matmul(dt, st["a"][i].float())
            grads += [torch.matmul(dt.t(), x).to(cd), (s * torch.matmul(dz[i].t(), st["t"][i])).to(cd)]
        return [dx.to(cd)] + grads
    threshold = _threshold(case["p"])
    keep, s = _keep(*x.shape, st["seed"], threshold), s / (1 - threshold / 65536)
    xd = torch.where(keep, x, torch.zeros_like(x))
    if case["op"] == "dropout_fwd":
        y, t = _project(st["w"], st["x"], st["a"], st["b"], s, cd, st["bias"], xd)
        return [y.to(cd)] + t
    dy = st["dy"].float()
    dt = s * torch.matmul(dy, st["b"][0].float())
    low = torch.matmul(dt, st["a"][0].float())
    dx = torch.matmul(dy, _weight(st["w"][0], cd)) + torch.where(keep, low, torch.zeros_like(low))
    return [dx.to(cd), torch.matmul(dt.t(), xd).to(cd), (s * torch.matmul(dy.t(), st["t"])).to(cd)]


def run(st):
    case = st["case"]
    if not own:
        return _run_plain(st)
    import bit_nf4_quantized_nibble_amd as qn

    if case["op"] == "fp8":
        return qn.linear_fp8(st["w"], st["x"], bias=st["bias"])
    alphas = [st["alpha"]] * len(st["w"])
    if case["op"] == "gated_fwd":
        out = qn.linear_fwd_gated(st["w"], st["x"], st["a"], st["b"], alphas, act=case["act"], bias=st["bias"],
                                  save=case["save"])
        return [out[0], out[1]] + list(out[2]) if case["save"] else out
    if case["op"] == "gated_bwd":  # gradients in the adapters' own type
        dx, da, db = qn.linear_bwd_gated(st["w"], st["x"], st["dy"], st["a"], st["b"], alphas, st["pre"],
                                         act=case["act"], t_saved=st["t"], grad_dtype=st["x"].dtype)
        return [dx, da[0], db[0], da[1], db[1]]
    if case["op"] == "dropout_fwd":
        return list(qn.linear_fwd_dropout(st["w"][0], st["x"], st["a"][0], st["b"][0], st["alpha"], case["p"],
                                          st["seed"], bias=st["bias"], save_t=True))
    return list(qn.linear_bwd_dropout(st["w"][0], st["x"], st["dy"], st["a"][0], st["b"][0], st["alpha"], case["p"],
                                      st["seed"], t_saved=st["t"], grad_dtype=st["x"].dtype))


# -------------------------------------------------------------------------- exact
def _exact_fp8(x, tall):
    """The same values from the formats: exponents by logarithm-free comparison, codes on the
    grid of e4m3 (steps of 2^-3 of the leading power of two, 2^-9 below 2^-6)."""
    rows, cols = x.shape
    x = x.double()
    out = torch.empty_like(x)
    steps = torch.tensor([2.0 ** i for i in range(-127, 121)], dtype=torch.float64, device=x.device)  # the scales there are
    for k in range(0, cols, 128):
        part = x[:, k:k + 128]
        top = part.abs().max(dim=1).values
        if tall > 1:
            top = torch.stack([top[i:i + tall].max() for i in range(0, rows, tall)]).repeat_interleave(tall)[:rows]
        s = steps[torch.searchsorted(steps * 448.0, top.contiguous())][:, None]  # the first with top <= 448 s
        v = part / s
        grid = torch.full_like(v, 2.0 ** -9)
        for p in range(-5, 9):  # values of at least 2^p have steps of 2^(p - 3)
            grid = torch.where(v.abs() >= 2.0 ** p, torch.full_like(v, 2.0 ** (p - 3)), grid)
        out[:, k:k + 128] = torch.round(v / grid) * grid * s
    return out


def _exact_weight(w, cd):
    high, low = w["codes"] // 16, w["codes"] % 16
    value = w["levels"].double()[torch.stack((high, low), dim=-1).flatten().int()].view(-1, 64)
    if w["dq"]:
        i = torch.arange(value.shape[0], device=value.device)
        scale = (w["absmax_q"].double() * w["absmax_scale2"].double()[i // 256]).float().double()
    else:
        scale = w["absmax"].double()
    return (value * scale[:, None]).float().to(cd).double().view(w["rows"], w["cols"])


def _exact_keep(m, k, seed, p):
    """The mask from the generator's definition, in numpy's unsigned 64-bit integers."""
    import numpy as np

    s, o = (int(v) & ((1 << 64) - 1) for v in seed.tolist())
    key0, key1 = s & 0xFFFFFFFF, s >> 32
    groups = (k + 7) // 8
    shape = np.zeros((m, groups), dtype=np.uint64)
    x0, x1 = shape + np.arange(groups, dtype=np.uint64), shape + np.arange(m, dtype=np.uint64)[:, None]
    x2, x3 = shape + np.uint64(o & 0xFFFFFFFF), shape + np.uint64(o >> 32)
    word, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for rnd in range(10):
        k0, k1 = np.uint64((key0 + rnd * 0x9E3779B9) % (1 << 32)), np.uint64((key1 + rnd * 0xBB67AE85) % (1 << 32))
        a, b = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = (b >> half) ^ x1 ^ k0, b & word, (a >> half) ^ x3 ^ k1, a & word
    bits = np.empty((m, groups, 8), dtype=np.int32)
    for i, v in enumerate((x0, x1, x2, x3)):
        bits[:, :, 2 * i], bits[:, :, 2 * i + 1] = v & np.uint64(0xFFFF), v >> np.uint64(16)
    keep = bits.reshape(m, groups * 8)[:, :k] >= int(math.floor(p * 65536 + 0.5))
    return torch.from_numpy(keep.astype(np.float64)).cuda()


def _exact_act(z, act):
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * torch.sigmoid(-z)
    if act == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 0.134145 * z * z)


def exact(case, seed):
    global own
    kept, own = own, False  # the inputs alone, without the package
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    cd, x, n = _TYPES[case["cd"]], st["x"].double(), case["rows"]
    bias = 0.0 if st["bias"] is None else st["bias"].double()
    if case["op"] == "fp8":
        g = _generator(seed)  # the weight as prepare() made it, before it had 8 bits
        _hidden(g, case["m"], case["cols"], case["cd"])
        if st["bias"] is not None:
            _randn(g, n)
        w = (_randn(g, n, case["cols"]) * (0.01 + 0.02 * torch.rand(n, 1, generator=g, device="cuda"))).to(cd)
        return _exact_fp8(st["x"], 1) @ _exact_fp8(w, 128).t() + bias
    a, b = [v.double() for v in st["a"]], [v.double() for v in st["b"]]
    w = [_exact_weight(v, cd) for v in st["w"]]
    s = st["alpha"] / case["r"]
    if case["op"] == "gated_fwd":
        t = [x @ v.t() for v in a]
        z = torch.cat([x @ w[i].t() + (t[i] @ b[i].t()) * s for i in (0, 1)], dim=1) + bias
        h = _exact_act(z[:, :n], case["act"])[0] * z[:, n:]
        return [h, z] + t if case["save"] else h
    if case["op"] == "gated_bwd":
        z, dh = st["pre"].double(), st["dy"].double()
        value, slope = _exact_act(z[:, :n], case["act"])
        dg, du = dh * z[:, n:] * slope, dh * value
        dx = dg @ (w[0] + s * (b[0] @ a[0])) + du @ (w[1] + s * (b[1] @ a[1]))
        t = [x @ v.t() for v in a]
        return [dx, s * (dg @ b[0]).t() @ x, s * dg.t() @ t[0], s * (du @ b[1]).t() @ x, s * du.t() @ t[1]]
    p = int(math.floor(case["p"] * 65536 + 0.5)) / 65536
    keep, s = _exact_keep(*x.shape, st["seed"], case["p"]), s / (1 - p)
    t = (x * keep) @ a[0].t()
    if case["op"] == "dropout_fwd":
        return [x @ w[0].t() + s * (t @ b[0].t()) + bias, t]
    dy = st["dy"].double()
    dt = s * (dy @ b[0])
    return [dy @ w[0] + keep * (dt @ a[0]), dt.t() @ (x * keep), s * dy.t() @ t]
