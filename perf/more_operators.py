"""The 8-bit verify layers and the sampled verify: the cases that are measured.

Three operators are listed, each in a plain form (elementary torch operations)
and as a user of the library calls it:

* ``norm``    rows of the residual stream: the residual's addition, the RMS
              norm and the result in 8 bits with a power-of-two scale per row,
              and the values read back; without the norm, rows of an activation
              quantised as they are;
* ``linear``  8-bit rows times 8-bit weights with bias, activation (plain or
              gated) and residual in the epilogue;
* ``sample``  a token from each row of logits with temperature, top-k, top-p and
              min-p, the noise keyed by (seed, position, stream).

An 8-bit row is e4m3 codes times one scale. Weights have one scale per output
channel. Rounding is to nearest even throughout.
"""
import math
import random

import torch

own = False
DEV = "cuda"
EPS = 1e-6
E4M3_MAX = 448.0


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token between two layers: latency
        dict(name="norm 1 row", op="norm", M=1, d=4096, dtype="bf16", norm=True),
        # a long prompt between two layers, an odd number of rows
        dict(name="norm prompt", op="norm", M=16383, d=4096, dtype="bf16", norm=True),
        # the MLP's activation before its down projection, quantised as it is
        dict(name="norm activation rows", op="norm", M=4097, d=12288, dtype="bf16", norm=False),
        # query, key and value projection of one token
        dict(name="linear qkv 1 row", op="linear", M=1, K=4096, N=6144, gated=False, act="none", bias=False,
             residual=False, out="bf16"),
        # the attention output's projection of a verify round's 64 packed rows, into the residual stream
        dict(name="linear o 64 rows", op="linear", M=64, K=4096, N=4096, gated=False, act="none", bias=False,
             residual=True, out="bf16"),
        # gate and up projection of the same rows
        dict(name="linear gated 64 rows", op="linear", M=64, K=4096, N=12288, gated=True, act="silu", bias=False,
             residual=False, out="bf16"),
        # a tower's MLP on an image's patches: odd sizes, bias, GELU
        dict(name="linear patches", op="linear", M=777, K=1040, N=4152, gated=False, act="gelu_tanh", bias=True,
             residual=False, out="bf16"),
        # the LM head's logits of a verify round
        dict(name="linear logits 64 rows", op="linear", M=64, K=4096, N=151936, gated=False, act="none", bias=False,
             residual=False, out="f32"),
        # gate and up projection of a long prompt: the largest case
        dict(name="linear gated prompt", op="linear", M=8191, K=4096, N=12288, gated=True, act="silu", bias=False,
             residual=False, out="bf16"),
        # the next token of one chat request: latency
        dict(name="sample 1 row", op="sample", M=1, V=151936, dtype="f32", params="chat", shape="mixed", masked=0.0),
        # a verify round's rows under nucleus sampling, 16-bit logits with many ties
        dict(name="sample 64 rows nucleus", op="sample", M=64, V=151936, dtype="bf16", params="nucleus",
             shape="mixed", masked=0.0),
        # a full batch of verify rows, every request with its own parameters
        dict(name="sample 512 rows mixed", op="sample", M=512, V=151936, dtype="f32", params="mixed", shape="mixed",
             masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "sample"))
    if op == "norm":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        d = 16 * _log_int(rng, 4, 1024)
        most = 16383 * 4096 // (2 if dtype == "f32" else 1)
        return dict(op=op, M=_log_int(rng, 1, max(1, min(16383, most // d))), d=d, dtype=dtype, norm=rng.random() < 0.7)
    if op == "linear":
        K = 16 * _log_int(rng, 4, 768)
        gated = rng.random() < 0.35
        N = 8 * _log_int(rng, 1, 1536 if gated else 4096)
        M = _log_int(rng, 1, max(1, min(8191, 8191 * 4096 * 24576 // (K * N * (2 if gated else 1)))))
        return dict(op=op, M=M, K=K, N=N, gated=gated, act=rng.choice(("silu", "gelu", "gelu_tanh") if gated else
                                                                      ("none", "none", "silu", "gelu", "gelu_tanh")),
                    bias=rng.random() < 0.4, residual=not gated and rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "f32")))
    V = _log_int(rng, 500, 151936)
    return dict(op=op, M=_log_int(rng, 1, 512), V=V, dtype=rng.choice(("f32", "bf16")),
                params=rng.choice(("chat", "nucleus", "mixed", "mixed", "pure", "minp")),
                shape=rng.choice(("mixed", "flat", "peaked")), masked=rng.choice((0.0, 0.0, 0.5, 0.99)))


# --------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _codes(gen, rows, width):
    """Weights or activations in 8 bits as a checkpoint or an earlier call leaves them: (codes, scales)."""
    codes = torch.empty(rows, width, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(rows, device=DEV)
    step = max(1, (1 << 26) // width)
    for i in range(0, rows, step):
        x = _randn(gen, min(step, rows - i), width)
        s = x.abs().amax(1) / E4M3_MAX
        codes[i:i + step] = (x / s[:, None]).to(torch.float8_e4m3fn)
        scales[i:i + step] = s
    return codes, scales


def prepare(case, seed):
    gen = _gen(seed)
    rng = random.Random(int(seed) * 1000003 + 29)
    op = case["op"]
    s = dict(case=case)
    if op == "norm":
        M, d = case["M"], case["d"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a residual stream has a few channels far above the others
        channel = torch.exp(0.5 * _randn(gen, d))
        channel[torch.randint(0, d, (3,), generator=gen, device=DEV)] *= 40
        s["x"] = (_randn(gen, M, d) * channel).to(dt)
        s["codes"] = torch.zeros(M, d, dtype=torch.float8_e4m3fn, device=DEV)
        s["scales"] = torch.zeros(M, device=DEV)
        s["back"] = torch.zeros(M, d, dtype=torch.bfloat16, device=DEV)
        if case["norm"]:
            s["residual"] = _randn(gen, M, d).to(dt)
            s["weight"] = 1 + 0.3 * _randn(gen, d)
            s["total"] = torch.zeros(M, d, dtype=dt, device=DEV)
    elif op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s["x"], s["x_scale"] = _codes(gen, M, K)
        # rows as the norm leaves them: power-of-two scales
        s["x_scale"] = torch.exp2(torch.ceil(torch.log2(s["x_scale"])))
        s["w"], s["w_scale"] = _codes(gen, N * (2 if case["gated"] else 1), K)
        s["w_scale"] *= 1.5 * K ** -0.5
        s["bias"] = 0.5 * _randn(gen, s["w"].shape[0]) if case["bias"] else None
        s["residual"] = _randn(gen, M, N).to(dt) if case["residual"] else None
        s["out"] = torch.zeros(M, N, dtype=dt, device=DEV)
    else:
        M, V = case["M"], case["V"]
        # a bulk of unlikely tokens and, row by row, a tail of likely ones above it
        x = _randn(gen, M, V).mul_(2.0)
        likely = min(V, 200)
        first, step = (torch.randint(0, n, (M, 1), generator=gen, device=DEV) for n in (V, V // likely))
        rank = torch.arange(likely, device=DEV)
        at = (first + rank * (step + 1)) % V
        lift = {"flat": 0.0, "mixed": 12.0, "peaked": 18.0}[case["shape"]]
        height = lift * torch.rand(M, 1, generator=gen, device=DEV) + 2
        x.scatter_(1, at, height * torch.exp(-rank / 25) + 0.7 * _randn(gen, M, likely) + 2)
        if case["masked"]:
            # tokens that a grammar forbids; the first likely one of each row stays
            stop = torch.rand(M, V, generator=gen, device=DEV) < case["masked"]
            stop.scatter_(1, at[:, :1], False)
            x.masked_fill_(stop, -math.inf)
        s["logits"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)

        def row(values, dtype=torch.float32):
            return torch.tensor([rng.choice(values) for _ in range(M)], dtype=dtype, device=DEV)

        p = case["params"]
        s["temperature"] = row({"chat": [0.7], "mixed": [0.0, 0.3, 0.7, 1.0, 1.5], "minp": [1.2]}.get(p, [1.0]))
        s["top_k"] = row({"chat": [20], "mixed": [0, 1, 20, 50, 1000]}.get(p, [0]), torch.int32)
        s["top_p"] = row({"chat": [0.8], "nucleus": [0.95], "mixed": [1.0, 0.95, 0.8, 0.5]}.get(p, [1.0]))
        s["min_p"] = row({"minp": [0.05], "mixed": [0.0, 0.0, 0.02, 0.1]}.get(p, [0.0]))
        s["seed"] = rng.getrandbits(63)
        s["position"] = torch.randint(0, 131072, (M,), generator=gen, device=DEV, dtype=torch.int32)
        s["stream"] = torch.randint(0, 16, (M,), generator=gen, device=DEV, dtype=torch.int32)
        s["tokens"] = torch.zeros(M, dtype=torch.int32, device=DEV)
        s["gap"] = torch.zeros(M, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _quantised_values(y):
    """What the 8-bit form of fp32 rows stands for."""
    top = y.abs().amax(1, keepdim=True)
    # least e with top <= 448 * 2^e, from the quotient's exponent (448 = 1.75 * 2^8)
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)
    scale = torch.ldexp(torch.ones_like(y[:, :1]), torch.where(top > 0, e, torch.zeros_like(e)))
    return ((y / scale).to(torch.float8_e4m3fn).float() * scale).to(torch.bfloat16)


def _plain_norm(s):
    if not s["case"]["norm"]:
        return [_quantised_values(s["x"].float())]
    s["total"].copy_(s["x"].float() + s["residual"].float())
    t = s["total"].float()
    y = t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * s["weight"]
    return [s["total"], _quantised_values(y)]


def _activation(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x)))
    return x


def _plain_linear(s):
    c = s["case"]
    y = torch.matmul(s["x"].float(), s["w"].float().t())
    y *= s["x_scale"][:, None]
    y *= s["w_scale"]
    if s["bias"] is not None:
        y += s["bias"]
    if c["gated"]:
        y = _activation(y[:, :c["N"]], c["act"]) * y[:, c["N"]:]
    else:
        y = _activation(y, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["out"].copy_(y)
    return s["out"]


def _noise(seed, position, stream, V):
    """Gumbel noise [M, V] in 64 bits from the ten-round Philox4x32 generator (Salmon et al., SC 2011):
    counter (v / 4, position, stream, 0), key the seed's halves, word v mod 4, its top 23 bits centred."""
    mask = 0xFFFFFFFF
    shape = (position.numel(), (V + 3) // 4)
    a = torch.arange(shape[1], device=DEV).expand(shape)
    b = (position.long() & mask)[:, None].expand(shape)
    c = (stream.long() & mask)[:, None].expand(shape)
    d = torch.zeros_like(a)
    k0, k1 = seed & mask, seed >> 32 & mask
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (q >> 32 & mask) ^ b ^ k0, q & mask, (p >> 32 & mask) ^ d ^ k1, p & mask
        k0, k1 = k0 + 0x9E3779B9 & mask, k1 + 0xBB67AE85 & mask
    words = torch.stack((a, b, c, d), 2).view(shape[0], -1)[:, :V]
    u = ((words >> 9).double() + 0.5) / (1 << 23)
    return -torch.log(-torch.log(u))


def _plain_sample(s):
    x = s["logits"].double()
    M, V = x.shape
    greedy = s["temperature"] == 0
    r = (1 / torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"])).double()[:, None]
    top, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((top - top[:, :1]) * r)
    k = torch.where(s["top_k"] > 0, s["top_k"], torch.full_like(s["top_k"], V))[:, None]
    keep = (torch.arange(V, device=DEV) < k) & (w >= s["min_p"].double()[:, None]) & (w > 0)
    w = w * keep
    upto = torch.cumsum(w, 1)
    p = s["top_p"].double()[:, None]
    keep &= (upto - w < p * upto[:, -1:]) | (p >= 1)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    z = x * r + _noise(s["seed"], s["position"], s["stream"], V)
    z = torch.where(greedy[:, None], x, torch.where(kept, z, torch.full_like(z, -math.inf)))
    best, at = z.max(1)
    rest = z.scatter(1, at[:, None], -math.inf).amax(1)
    s["tokens"].copy_((z == best[:, None]).int().argmax(1))
    s["gap"].copy_(best - rest)
    return [s["tokens"], s["gap"]]


# ------------------------------------------------------------------------ run

def run(s):
    c = s["case"]
    if not own:
        return {"norm": _plain_norm, "linear": _plain_linear, "sample": _plain_sample}[c["op"]](s)
    import tree_verified_block_gb300 as g
    if c["op"] == "norm":
        if c["norm"]:
            g.q8_norm_rows(s["x"], s["residual"], s["weight"], EPS, s["total"], s["codes"], s["scales"])
        else:
            g.q8_rows(s["x"], s["codes"], s["scales"])
        g.q8_read_rows(s["codes"], s["scales"], s["back"])
        return [s["total"], s["back"]] if c["norm"] else [s["back"]]
    if c["op"] == "linear":
        g.q8_linear(s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"], bias=s["bias"], act=c["act"],
                    gated=c["gated"], residual=s["residual"])
        return s["out"]
    g.sample(s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["seed"], s["position"], s["stream"],
             s["tokens"], s["gap"])
    return [s["tokens"], s["gap"]]


# ----------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["M"] * case["d"]
        # rows in (and the residual in, the sum out), codes out; codes in, values out
        return {"bytes": n * (e * (3 if case["norm"] else 1) + 1 + 3), "flops": n * (10 if case["norm"] else 4)}
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        rows = N * (2 if case["gated"] else 1)
        e = 2 if case["out"] == "bf16" else 4
        b = M * (K + 4) + rows * (K + 4 + (4 if case["bias"] else 0)) + M * N * e * (2 if case["residual"] else 1)
        return {"bytes": b, "flops": 2 * M * K * rows}
    M, V = case["M"], case["V"]
    return {"bytes": M * (V * (2 if case["dtype"] == "bf16" else 4) + 32), "flops": 4 * M * V}


# ---------------------------------------------------------------------- exact

def _grid():
    """The magnitudes of e4m3: (1 + f/8) 2^(e-7), and f/8 2^-6 where e is 0."""
    return torch.tensor([f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7) for e in range(16) for f in range(8)
                         if (e, f) != (15, 7)], dtype=torch.float64, device=DEV)


def _of_codes(codes):
    """The values of e4m3 codes in 64 bits, from their bits."""
    b = codes.view(torch.uint8).long()
    m = _grid()[b & 127]
    return torch.where(b > 127, -m, m)


def _nearest(x, grid):
    """The member of an ascending grid nearest to each x >= 0; between two, the one of even index."""
    i = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (i % 2 == 0))
    return torch.where(up, hi, lo)


def _exact_norm(s):
    c, grid, total, back = s["case"], _grid(), [], []
    step = max(1, (1 << 24) // c["d"])
    for i in range(0, c["M"], step):
        y = s["x"][i:i + step].double()
        if c["norm"]:
            y = y + s["residual"][i:i + step].double()
            total.append(y)
            y = y.to(s["x"].dtype).double()  # the stream holds the rounded sum
            y = y / torch.sqrt(y.pow(2).sum(1, keepdim=True) / c["d"] + EPS) * s["weight"].double()
        scale = torch.exp2(torch.ceil(torch.log2(y.abs().max(1, keepdim=True).values / E4M3_MAX)))
        scale = torch.where(torch.isfinite(scale), scale, torch.ones_like(scale))
        back.append(torch.sign(y) * _nearest(y.abs() / scale, grid) * scale)
    return [torch.cat(total), torch.cat(back)] if c["norm"] else [torch.cat(back)]


def _exact_linear(s):
    c = s["case"]
    x = _of_codes(s["x"]) * s["x_scale"].double().unsqueeze(1)
    out = torch.empty(c["M"], c["N"], dtype=torch.float64, device=DEV)

    def part(a, b):
        y = x @ (_of_codes(s["w"][a:b]) * s["w_scale"][a:b].double().unsqueeze(1)).t()
        return y if s["bias"] is None else y + s["bias"][a:b].double()

    def act(y):
        if c["act"] == "silu":
            return y * torch.special.expit(y)
        if c["act"] == "gelu":
            return y * torch.special.ndtr(y)
        if c["act"] == "gelu_tanh":  # (1 + tanh z) / 2 = 1 / (1 + e^-2z)
            return y * torch.special.expit(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y.pow(3)))
        return y

    for i in range(0, c["N"], 8192):
        j = min(i + 8192, c["N"])
        y = act(part(i, j))
        if c["gated"]:
            y = y * part(c["N"] + i, c["N"] + j)
        out[:, i:j] = y if s["residual"] is None else y + s["residual"][:, i:j].double()
    return out


def _words(seed, position, stream, V):
    """The generator's words of one row, with 32 x 32 bit products in 16-bit halves."""
    def product(m, x):
        low, mid = (m & 65535) * (x & 65535), (m >> 16) * (x & 65535)
        cross = (m & 65535) * (x >> 16) + (low >> 16) + (mid & 65535)
        return ((m >> 16) * (x >> 16) + (mid >> 16) + (cross >> 16)) & 0xFFFFFFFF, ((cross & 65535) << 16) | (low & 65535)

    x = torch.zeros(4, (V + 3) // 4, dtype=torch.int64, device=DEV)
    x[0] = torch.arange((V + 3) // 4, device=DEV)
    x[1], x[2] = position % (1 << 32), stream % (1 << 32)
    for i in range(10):
        hi0, lo0 = product(0xD2511F53, x[0])
        hi1, lo1 = product(0xCD9E8D57, x[2])
        x = torch.stack((hi1 ^ x[1] ^ (seed + i * 0x9E3779B9) % (1 << 32), lo1,
                         hi0 ^ x[3] ^ ((seed >> 32) + i * 0xBB67AE85) % (1 << 32), lo0))
    return x.t().reshape(-1)[:V]


def _exact_sample(s):
    tokens, gaps = [], []
    V = s["case"]["V"]
    for i in range(s["case"]["M"]):
        x = s["logits"][i].double()
        T, k, p, floor = (s[n][i].item() for n in ("temperature", "top_k", "top_p", "min_p"))
        if T == 0:
            z = x
        else:
            r = (torch.ones(1) / torch.tensor([T], dtype=torch.float32)).double().item()
            value = torch.sort(x).values.flip(0)
            n = min(k, V) if k > 0 else V
            weight = torch.exp((value - value[0]) * r)
            n = min(n, int((weight >= max(floor, 1e-323)).sum()))
            if p < 1:
                upto = torch.cumsum(weight[:n], 0)
                n = max(1, int((upto < p * upto[-1]).sum()) + 1)
            border = value[n - 1]
            tied = x == border
            kept = (x > border) | (tied & (torch.cumsum(tied, 0) <= n - (x > border).sum()))
            word = _words(s["seed"], int(s["position"][i]), int(s["stream"][i]), V)
            u = ((word >> 9) * 2 + 1).double() * 2.0 ** -24
            z = torch.where(kept, x * r - torch.log(torch.log(1 / u)), -math.inf)
        two = torch.topk(z, 2).values
        tokens.append(int((z == two[0]).nonzero()[0]))
        gaps.append((two[0] - two[1]).item())
    return [torch.tensor(tokens, dtype=torch.int32, device=DEV), torch.tensor(gaps, dtype=torch.float64, device=DEV)]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "sample": _exact_sample}[case["op"]](s)
