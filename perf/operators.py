"""The operators around a fine-tuned layer, as cases for measurement: the 8-bit integer
product with a scale per token and per output channel, the same product grouped by
expert, and the distillation loss against a teacher's top logits with its gradient.

``run`` computes each operator either in its plain form (elementary torch operations
in fp32) or, with ``own`` set, through the package's entry points.

The definitions both share:
  rows to 8 bits   s = fl32(max |x| / 127) for each row, c = round-half-even(fl32(x / s))
                   limited to +-127 (0 where s is 0); a weight [rows, cols] has one scale
                   per row (output channel), activations one per token
  int8 product     y[i, j] = s_i t_j sum_k c[i, k] d[j, k] (+ bias[j])
  experts          rows offsets[e] .. offsets[e + 1] - 1 of x take expert e's weight; rows
                   from offsets[E] on are left as they were
  distillation     p = softmax(u / T) over a row's present slots, q = softmax(z / T) over the
                   vocabulary, kl = T^2 sum_j p_j (log p_j - log q[index_j]);
                   loss = sum_i w_i kl_i, dz_i = w_i T (q - p); a slot is absent when its index
                   lies outside the vocabulary or its value is -inf; a row of weight 0 or
                   without a present slot contributes nothing and has a zero gradient
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------- cases
def _int8(m, rows, cols, cd, bias=False):
    return {"op": "int8", "m": m, "rows": rows, "cols": cols, "cd": cd, "bias": bias}


def _experts(m, experts, rows, cols, cd, skew, routing, bias=False, tail=0):
    return {"op": "experts", "m": m, "experts": experts, "rows": rows, "cols": cols, "cd": cd, "skew": skew,
            "routing": routing, "bias": bias, "tail": tail}


def _distill(n, vocab, k, cd, temperature, weights=False, absent=False, masked=0, pad=0, grad=True, index="i64"):
    return {"op": "distill", "n": n, "vocab": vocab, "k": k, "cd": cd, "temperature": temperature,
            "weights": weights, "absent": absent, "masked": masked, "pad": pad, "grad": grad, "index": index}


def listed():
    cases = [
        # one token through an attention projection: bound by reading the weight, and by latency
        ("int8_one_token", _int8(1, 4096, 4096, "bf16")),
        # a batch of 16 sequences, one token each, through an MLP projection
        ("int8_decode_batch", _int8(16, 14336, 4096, "bf16", bias=True)),
        # a short prompt through a layer whose sizes suit no tile
        ("int8_odd", _int8(333, 1003, 2047, "f16", bias=True)),
        # a long prompt through the widest projection
        ("int8_prompt", _int8(4096, 14336, 4096, "bf16")),
        # one token each for 8 sequences, two of eight experts per token
        ("experts_decode", _experts(16, 8, 4096, 4096, "bf16", 1.0, 1)),
        # many small experts of unequal load, some without a row; a buffer with room behind the last row
        ("experts_many", _experts(4096, 64, 1024, 2048, "f16", 1.5, 2, tail=37)),
        # a prompt's tokens over eight wide experts
        ("experts_prompt", _experts(8192, 8, 14336, 4096, "bf16", 0.5, 3)),
        # fp32 activations, sizes that suit no tile, a bias for each expert
        ("experts_odd", _experts(700, 5, 515, 1111, "f32", 1.0, 4, bias=True)),
        # a handful of answer tokens in fp32: latency
        ("distill_few", _distill(8, 32000, 16, "f32", 2.0)),
        # an ordinary micro-batch; prompt tokens carry weight 0
        ("distill_batch", _distill(1024, 32000, 32, "bf16", 1.0, weights=True)),
        # a long batch over a wide vocabulary
        ("distill_wide", _distill(4096, 128000, 64, "bf16", 1.0)),
        # an odd vocabulary inside a padded buffer, teacher lists of differing lengths, forbidden tokens
        ("distill_odd", _distill(509, 50257, 100, "f16", 0.7, weights=True, absent=True, masked=97, pad=47,
                                 index="i32")),
    ]
    return [dict(c, name=name) for name, c in cases]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v > 64:  # half of the sizes are whole tiles, half are odd
        v = max(64, v // 64 * 64)
    return max(lo, min(hi, v))


def draw(rng):
    limit = {c["op"]: max(work(d)["flops"] + 200 * work(d)["bytes"] for d in listed() if d["op"] == c["op"])
             for c in listed()}
    while True:
        op = rng.choice(["int8", "experts", "distill"])
        cd = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op == "int8":
            case = _int8(_log_int(rng, 1, 4096), _log_int(rng, 64, 14336), _log_int(rng, 64, 14336), cd,
                         bias=rng.random() < 0.5)
        elif op == "experts":
            case = _experts(_log_int(rng, 1, 8192), _log_int(rng, 2, 128), _log_int(rng, 64, 14336),
                            _log_int(rng, 64, 8192), cd, rng.choice([0.0, 0.5, 1.0, 2.0]), rng.randrange(1 << 20),
                            bias=rng.random() < 0.3, tail=rng.choice([0, 0, 1, 130]))
            if case["experts"] * case["rows"] * case["cols"] > 8 * 14336 * 4096:
                continue
        else:
            vocab = _log_int(rng, 1000, 200000)
            case = _distill(_log_int(rng, 1, 4096), vocab, _log_int(rng, 1, 256), cd,
                            rng.choice([0.5, 1.0, 2.0, 4.0]), weights=rng.random() < 0.5,
                            absent=rng.random() < 0.5, masked=rng.choice([0, vocab // 50]),
                            pad=rng.choice([0, 0, 1, 24]), grad=rng.random() < 0.8, index=rng.choice(["i32", "i64"]))
        w = work(case)
        if w["flops"] + 200 * w["bytes"] <= limit[op]:
            return case


def _sizes(case):
    """Rows of each expert: shares of the total by a random weight to the power skew,
    dealt row by row; a skewed routing leaves experts without a row."""
    rng = random.Random(case["routing"])
    shares = [rng.expovariate(1.0) ** case["skew"] for _ in range(case["experts"])]
    sizes = [0] * case["experts"]
    for e in rng.choices(range(case["experts"]), weights=shares, k=case["m"]):
        sizes[e] += 1
    return sizes


def work(case):
    b = _BYTES[case["cd"]]
    if case["op"] == "int8":
        m, n, k = case["m"], case["rows"], case["cols"]
        return {"bytes": m * k * b + n * k + 4 * n + m * n * b + (n * b if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if case["op"] == "experts":
        m, n, k = case["m"], case["rows"], case["cols"]
        live = sum(1 for s in _sizes(case) if s)
        return {"bytes": m * k * b + live * (n * k + 4 * n + (n * b if case["bias"] else 0)) + m * n * b
                + 4 * (case["experts"] + 1), "flops": 2 * m * n * k}
    n, v, k = case["n"], case["vocab"], case["k"]
    live = n * 3 // 4 if case["weights"] else n  # rows of weight 0 need no reading
    slots = live * k * (4 + (4 if case["index"] == "i32" else 8))
    return {"bytes": live * v * b + (n * v * b if case["grad"] else 0) + slots + 4 * n + 4,
            "flops": live * v * (8 if case["grad"] else 4)}


# ------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, m, k, cd):
    # hidden states after a norm: unit variance, a few channels much larger than the rest
    x = torch.randn(m, k, generator=g, device="cuda")
    gain = torch.ones(k, device="cuda")
    gain[torch.randperm(k, generator=g, device="cuda")[: max(1, k // 200)]] = 12.0
    return (x * gain).to(_TYPES[cd])


def _weight(g, shape, cd):
    # a merged projection: N(0, 0.02^2), rows of differing size
    w = torch.empty(shape, dtype=_TYPES[cd], device="cuda")
    rows = 0.01 + 0.02 * torch.rand(shape[:-1], generator=g, device="cuda")
    for part, size in zip(w.view(-1, shape[-1]).split(8192), rows.view(-1).split(8192)):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * size[:, None])
    return w


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case}
    cd = _TYPES[case["cd"]]
    if case["op"] in ("int8", "experts"):
        lead = () if case["op"] == "int8" else (case["experts"],)
        w = _weight(g, lead + (case["rows"], case["cols"]), case["cd"])
        m = case["m"] + case.get("tail", 0)
        st["x"] = _activations(g, m, case["cols"], case["cd"])
        st["bias"] = (torch.randn(lead + (case["rows"],), generator=g, device="cuda") * 0.1).to(cd) \
            if case["bias"] else None
        if case["op"] == "experts":
            st["sizes"] = _sizes(case)
            ends = [0]
            for s in st["sizes"]:
                ends.append(ends[-1] + s)
            st["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
            # the buffer that receives y: rows behind the last expert's keep what they hold
            st["out"] = torch.randn(m, case["rows"], generator=g, device="cuda").to(cd)
        if own:
            import bit_nf4_quantized_nibble_amd as qn

            st["w"] = qn.quantize_int8(w)
        else:
            st["codes"], st["scale"] = _rows_to_int8(w)
        return st
    n, v, k = case["n"], case["vocab"], case["k"]
    buf = torch.empty(n, v + case["pad"], dtype=cd, device="cuda")
    st["logits"] = buf[:, :v]
    st["top_values"] = torch.empty(n, k, device="cuda")
    index = torch.empty(n, k, dtype=torch.int64, device="cuda")
    forbidden = torch.randperm(v, generator=g, device="cuda")[: case["masked"]]
    for i in range(0, n, 512):
        # the teacher's logits, and a student that follows them with noise
        t = torch.randn(min(512, n - i), v, generator=g, device="cuda") * 3.0
        t[:, forbidden] = float("-inf")
        st["top_values"][i:i + 512], index[i:i + 512] = torch.topk(t, k, dim=1)
        buf[i:i + 512, :v] = (t + torch.randn(t.shape, generator=g, device="cuda") * 0.5).to(cd)
        buf[i:i + 512, v:] = 0
    if case["absent"]:  # lists that end early; now and then an empty one
        length = torch.randint(0, k + 1, (n, 1), generator=g, device="cuda")
        index[torch.arange(k, device="cuda")[None, :] >= length] = -1
    st["top_index"] = index.to(torch.int32) if case["index"] == "i32" else index
    st["weight"] = None
    if case["weights"]:
        live = (torch.arange(n, device="cuda") % 4) != 0
        st["weight"] = live.float() * (0.5 + torch.rand(n, generator=g, device="cuda")) / n
    return st


# --------------------------------------------------------------------- plain form
def _rows_to_int8(x):
    x = x.float()
    scale = x.abs().amax(dim=-1) / torch.tensor(127.0, device=x.device)
    codes = torch.round(x / scale[..., None]).clamp(-127.0, 127.0)
    codes = torch.where(scale[..., None] > 0, codes, torch.zeros_like(codes))
    return codes.to(torch.int8), scale


def _plain_product(codes, scale, x, bias, cd):
    c, s = _rows_to_int8(x)
    y = torch.matmul(c.float(), codes.float().t()) * s[:, None] * scale[None, :]
    if bias is not None:
        y = y + bias.float()
    return y.to(cd)


def _plain_distill(st):
    case = st["case"]
    n, v, temp = case["n"], case["vocab"], case["temperature"]
    cd = _TYPES[case["cd"]]
    z = st["logits"].float() / temp
    u = st["top_values"].float() / temp
    idx = st["top_index"].long()
    present = (idx >= 0) & (idx < v) & (u > float("-inf"))
    weight = st["weight"] if st["weight"] is not None else torch.full((n,), 1.0 / n, device=z.device)
    live = (weight != 0) & present.any(dim=1)
    u = torch.where(present, u, torch.full_like(u, float("-inf")))
    u = torch.where(live[:, None], u, torch.zeros_like(u))
    u = u - u.amax(dim=1, keepdim=True)
    p = torch.exp(u)
    total = p.sum(dim=1, keepdim=True)
    p = p / total
    log_p = u - torch.log(total)
    z = z - z.amax(dim=1, keepdim=True)
    lse = torch.log(torch.exp(z).sum(dim=1, keepdim=True))
    slot = torch.where(present, idx, torch.zeros_like(idx))
    term = p * (log_p - (z.gather(1, slot) - lse))
    term = torch.where(present & (p > 0) & live[:, None], term, torch.zeros_like(term))
    kl = temp * temp * term.sum(dim=1)
    loss = torch.where(live, weight * kl, torch.zeros_like(kl)).sum().reshape(1)
    if not case["grad"]:
        return loss
    q = torch.exp(z - lse)
    q.scatter_add_(1, slot, torch.where(present, -p, torch.zeros_like(p)))
    dz = q * (weight * temp)[:, None]
    dz = torch.where(live[:, None], dz, torch.zeros_like(dz)).to(cd)
    return loss, dz


def run(st):
    case = st["case"]
    if own:
        import bit_nf4_quantized_nibble_amd as qn

        if case["op"] == "int8":
            return qn.linear_int8(st["w"], st["x"], bias=st["bias"])
        if case["op"] == "experts":
            return qn.linear_int8_experts(st["w"], st["x"], st["offsets"], bias=st["bias"], out=st["out"])
        out = qn.distill_loss_grad(st["logits"], st["top_values"], st["top_index"], temperature=case["temperature"],
                                   weight=st["weight"], need_grad=case["grad"])
        return out if case["grad"] else out[0]
    cd = _TYPES[case["cd"]]
    if case["op"] == "int8":
        return _plain_product(st["codes"], st["scale"], st["x"], st["bias"], cd)
    if case["op"] == "experts":
        at = 0
        for e, size in enumerate(st["sizes"]):
            if size:
                rows = slice(at, at + size)
                st["out"][rows] = _plain_product(st["codes"][e], st["scale"][e], st["x"][rows],
                                                 None if st["bias"] is None else st["bias"][e], cd)
            at += size
        return st["out"]
    return _plain_distill(st)


# -------------------------------------------------------------------------- exact
def _exact_rows(x):
    """Codes and scales by the definition: quotients formed in 64 bits, rounded to
    binary32 where the definition holds them in binary32."""
    x = x.double()
    scale = (x.abs().max(dim=-1, keepdim=True).values / 127.0).float().double()
    safe = torch.where(scale == 0, torch.ones_like(scale), scale)
    code = (x / safe).float().round().double().clamp(-127, 127)
    return code * (scale != 0), scale.squeeze(-1)


def exact(case, seed):
    global own
    kept, own = own, False  # the inputs alone, without the package
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    if case["op"] in ("int8", "experts"):
        x, m = st["x"], case["m"]
        codes = st["codes"] if case["op"] == "experts" else st["codes"][None]
        scale = st["scale"] if case["op"] == "experts" else st["scale"][None]
        sizes = st["sizes"] if case["op"] == "experts" else [m]
        bias = st["bias"] if case["op"] == "experts" or st["bias"] is None else st["bias"][None]
        y = st["out"].double() if case["op"] == "experts" \
            else torch.empty(m, case["rows"], dtype=torch.float64, device=x.device)
        end = 0
        for e, size in enumerate(sizes):
            start, end = end, end + size
            if not size:
                continue
            c, s = _exact_rows(x[start:end])
            acc = c @ codes[e].double().t().contiguous()  # whole numbers below 2^53: exact
            y[start:end] = torch.outer(s, scale[e].double()) * acc
            if bias is not None:
                y[start:end] += bias[e].double()
        return y
    n, v, temp = case["n"], case["vocab"], float(case["temperature"])
    loss = torch.zeros(1, dtype=torch.float64, device="cuda")
    grad = torch.zeros(n, v, dtype=torch.float64, device="cuda") if case["grad"] else None
    for i in range(0, n, 256):
        z = st["logits"][i:i + 256].double() / temp
        idx = st["top_index"][i:i + 256].long()
        u = st["top_values"][i:i + 256].double() / temp
        w = st["weight"][i:i + 256].double() if st["weight"] is not None \
            else torch.full((z.shape[0],), 1.0 / n, dtype=torch.float64, device="cuda")
        absent = (idx < 0) | (idx >= v) | (u == float("-inf"))
        rows = ((w != 0) & (~absent).any(dim=1)).nonzero().flatten()
        if rows.numel() == 0:
            continue
        z, idx, absent, w = z[rows], idx[rows], absent[rows], w[rows]
        u = u[rows].masked_fill(absent, float("-inf"))
        log_p = u - torch.logsumexp(u, dim=1, keepdim=True)
        log_q = z - torch.logsumexp(z, dim=1, keepdim=True)
        p = log_p.exp()
        at = idx.masked_fill(absent, 0)
        diff = (log_p - log_q.gather(1, at)).masked_fill(absent | (p == 0), 0.0)
        loss += (w * temp * temp * (p * diff).sum(dim=1)).sum()
        if grad is not None:
            d = log_q.exp()
            d.scatter_add_(1, at, -p.masked_fill(absent, 0.0))
            grad[i + rows] = d * (w * temp)[:, None]
    return loss if grad is None else (loss, grad)
