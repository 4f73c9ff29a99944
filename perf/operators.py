"""The operators beside the plain products, as a user's program calls them:
tensors kept in microscaled 4-bit floating point, linear layers with 4-bit
weights, and a mixture-of-experts layer for a few tokens.

Microscaled 4-bit floating point ("MX4" here): blocks of 32 consecutive
elements of a row share a power-of-two scale, held as one byte (exponent plus
127; 255 is NaN), and each element is a 4-bit float of values 0, 0.5, 1, 1.5,
2, 3, 4, 6 and a sign, the even element of a pair in the low half of a byte.
With m the largest magnitude of a block the scale is 2^(floor(log2 m) - 2);
elements round to nearest, ties to the even code, and saturate at 6.

  store   a tensor brought into 4 bits and back (weights at load time, a
          gradient or an activation set aside)
  linear  y = q(x) . w^T: 16-bit activations quantised on the fly, 4-bit
          weights; prefill and training's forward products
  decode  y = x . w^T: 16-bit activations as they are, 4-bit weights; a few
          rows, where reading the weights is all the time
  moe     y_t = sum over the top_k experts e of token t, by its logits, of
          p_te . w_down[e] (silu(g) * u), (g, u) = w_gate_up[e] x_t; expert
          weights in 16 bits or in MX4; the decode step of a
          mixture-of-experts model

listed() and draw() give cases, prepare() a case's inputs, run() one pass,
exact() the same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32

# The hidden and intermediate sizes of the expert products of this
# repository's own benchmark.
HIDDEN, INTER = 7168, 2048


def _store(name, rows, k, dtype, order):
    return {"name": name, "op": "store", "rows": rows, "k": k, "type": dtype, "order": order}


def _linear(name, m, n, k, dtype):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "type": dtype}


def _decode(name, m, n, k, dtype):
    return {"name": name, "op": "decode", "m": m, "n": n, "k": k, "type": dtype}


def _moe(name, tokens, experts, top_k, hidden, inter, dtype, weights, renormalize=True, logits="f32"):
    return {"name": name, "op": "moe", "tokens": tokens, "experts": experts, "top_k": top_k,
            "hidden": hidden, "inter": inter, "type": dtype, "weights": weights,
            "renormalize": renormalize, "logits": logits}


def listed():
    return [
        # a decode step's activations set aside: latency
        _store("store_decode_rows", 16, HIDDEN, "bf16", "rows"),
        # a prefill's activations: memory
        _store("store_prefill_rows", 32768, HIDDEN, "bf16", "rows"),
        # an odd-sized weight held [K, N], quantised along K
        _store("store_odd_columns", 4099, 2051, "f16", "columns"),
        # a chunked prefill through an expert's down product
        _linear("linear_prefill", 32768, INTER, HIDDEN, "bf16"),
        # an ordinary batch through a square projection
        _linear("linear_square", 4096, 4096, 4096, "f16"),
        # a short ragged prompt, odd sizes
        _linear("linear_odd", 333, 1061, 2050, "bf16"),
        # one token through a projection: latency and weights
        _decode("decode_one", 1, INTER, HIDDEN, "f16"),
        # a small decode batch, wide output
        _decode("decode_batch", 16, HIDDEN, INTER, "bf16"),
        # one token, large experts: weights
        _moe("moe_one", 1, 64, 8, HIDDEN, INTER, "bf16", "16"),
        # four tokens of a small model: latency
        _moe("moe_small", 4, 16, 2, 2048, 768, "f16", "16", renormalize=False, logits="same"),
        # a full decode batch: nearly every expert is read
        _moe("moe_batch", 64, 64, 8, HIDDEN, INTER, "bf16", "16"),
        # a decode batch with experts in 4 bits
        _moe("moe_mx4", 16, 64, 8, HIDDEN, INTER, "bf16", "mx4"),
    ]


def _log_size(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm; half of them
    multiples of 32 where that fits, the rest as they fall (odd ones among
    them)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 0.5:
        v -= v % 32
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["store", "linear", "decode", "moe"])
    half = rng.choice(["f16", "bf16"])
    if op == "store":
        c = _store("", _log_size(rng, 1, 32768), _log_size(rng, 32, HIDDEN),
                   rng.choice(["f16", "bf16", "f32"]), rng.choice(["rows", "columns"]))
    elif op == "linear":
        c = _linear("", _log_size(rng, 1, 16384), _log_size(rng, 64, 8192), _log_size(rng, 64, 8192), half)
        while c["m"] * c["n"] * c["k"] > 32768 * INTER * HIDDEN:
            c["n"] = max(64, c["n"] // 2)
    elif op == "decode":
        c = _decode("", _log_size(rng, 1, 64), _log_size(rng, 64, 16384), _log_size(rng, 64, 8192), half)
    else:
        experts = _log_size(rng, 2, 64)
        c = _moe("", _log_size(rng, 1, 64), experts, rng.randint(1, min(8, experts)),
                 _log_size(rng, 256, HIDDEN), _log_size(rng, 128, INTER), half,
                 rng.choice(["16", "mx4"]), rng.random() < 0.5, rng.choice(["f32", "same"]))
    del c["name"]
    return c


# ---- inputs

def _blocks(k):
    return (k + BLOCK - 1) // BLOCK


def _weights(gen, n, k, dtype):
    """n rows of k weights, of about unit gain."""
    return torch.randn(n, k, generator=gen, device="cuda", dtype=dtype) * k ** -0.5


def _mx4_weights(gen, n, k):
    """The same in MX4: (data [n, 16 blocks], scales [n, blocks])."""
    w = torch.zeros(n, _blocks(k) * BLOCK, device="cuda")
    w[:, :k] = _weights(gen, n, k, torch.float32)
    codes, exps = _codes(w)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), exps


def _activations(gen, m, k, dtype):
    """Unit-variance rows, a few channels of which run larger, as hidden
    states have them."""
    x = torch.randn(m, k, generator=gen, device="cuda", dtype=torch.float32)
    gain = torch.ones(k, device="cuda")
    gain[torch.randint(0, k, (max(1, k // 128),), generator=gen, device="cuda")] = 8.0
    return (x * gain).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    dtype = TYPES[case["type"]]
    if case["op"] == "store":
        if case["order"] == "rows":
            s["x"] = _activations(gen, case["rows"], case["k"], dtype)
        else:
            s["x"] = _weights(gen, case["k"], case["rows"], torch.float32).to(dtype).t()
        return s
    if case["op"] in ("linear", "decode"):
        s["x"] = _activations(gen, case["m"], case["k"], dtype)
        s["w"] = _mx4_weights(gen, case["n"], case["k"])
        if own:
            s["w4"] = _mx4(s["w"], case["k"])
        return s
    T, E, H, I = case["tokens"], case["experts"], case["hidden"], case["inter"]
    s["x"] = _activations(gen, T, H, dtype) * 0.5
    s["logits"] = torch.randn(T, E, generator=gen, device="cuda").to(
        torch.float32 if case["logits"] == "f32" else dtype)
    for key, n, k in (("gate_up", 2 * I, H), ("down", H, I)):
        if case["weights"] == "16":
            w = torch.empty(E, n, k, device="cuda", dtype=dtype)
            for e in range(E):
                w[e] = _weights(gen, n, k, dtype)
            s[key] = w
        else:
            d = torch.empty(E, n, 16 * _blocks(k), device="cuda", dtype=torch.uint8)
            x = torch.empty(E, n, _blocks(k), device="cuda", dtype=torch.uint8)
            for e in range(E):
                d[e], x[e] = _mx4_weights(gen, n, k)
            s[key] = (d, x)
            if own:
                s[key + "4"] = _mx4((d, x), k)
    return s


def _mx4(w, k):
    import dense_tiled_gemm_fp16_amd as g
    return g.MX4(w[0], w[1], k)


# ---- the plain forms

def _codes(x):
    """float32 rows of whole blocks -> (4-bit codes, scale bytes)."""
    b = x.view(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(dim=2)
    e = torch.frexp(amax).exponent - 3            # floor(log2(amax)) - 2
    e = torch.where(amax > 0, e, -127).clamp(min=-127)
    y = torch.ldexp(b, -e.unsqueeze(2))
    a = y.abs()
    # round to nearest; a tie goes to the even code
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) +
         (a > 5.0))
    c = c + 8 * (y < 0).to(torch.uint8)
    return c.view(x.shape).to(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, exps):
    """4-bit codes and scale bytes -> float32."""
    e = ((codes & 6) >> 1).int()                  # exponent field; 0 is subnormal
    h = (codes & 1).float() * 0.5
    v = torch.where(e > 0, torch.ldexp(h + 1.0, e - 1), h)
    v = torch.where(codes > 7, -v, v).view(codes.shape[0], -1, BLOCK)
    return torch.ldexp(v, exps.int().unsqueeze(2) - 127).view(codes.shape)


def _unpack(w, k):
    data, exps = w
    codes = torch.stack((data & 15, data >> 4), dim=2).view(data.shape[0], -1)
    return _values(codes, exps)[:, :k]


def _through_mx4(x):
    rows, k = x.shape
    p = torch.zeros(rows, _blocks(k) * BLOCK, device=x.device)
    p[:, :k] = x
    return _values(*_codes(p))[:, :k]


def _expert(w, e, k):
    """Expert e's weights as float32 rows (e an index tensor of one element)."""
    if isinstance(w, tuple):
        return _unpack((w[0].index_select(0, e)[0], w[1].index_select(0, e)[0]), k)
    return w.index_select(0, e)[0].float()


def _plain_moe(s):
    case = s["case"]
    T, E, k, I = case["tokens"], case["experts"], case["top_k"], case["inter"]
    H = case["hidden"]
    x, logits = s["x"].float(), s["logits"].float()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    p = torch.exp(top - top[:, :1])
    if case["renormalize"]:
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = p / torch.exp(logits - top[:, :1]).sum(dim=1, keepdim=True)
    y = torch.zeros(T, H, device=x.device)
    if T * k < E:                                  # few pairs: one pair at a time
        for t in range(T):
            for r in range(k):
                e = idx[t, r:r + 1]
                gu = x[t:t + 1] @ _expert(s["gate_up"], e, H).t()
                g, u = gu[:, :I], gu[:, I:]
                y[t:t + 1] += p[t, r] * ((g / (1 + torch.exp(-g)) * u) @ _expert(s["down"], e, I).t())
        return y.to(s["x"].dtype)
    dense = torch.zeros(T, E, device=x.device).scatter_(1, idx, p)
    for i in range(E):                             # many: one expert at a time, all tokens
        e = torch.full((1,), i, device=x.device, dtype=torch.int64)
        gu = x @ _expert(s["gate_up"], e, H).t()
        g, u = gu[:, :I], gu[:, I:]
        y += dense[:, i:i + 1] * ((g / (1 + torch.exp(-g)) * u) @ _expert(s["down"], e, I).t())
    return y.to(s["x"].dtype)


def run(state):
    case, x = state["case"], state["x"]
    if own:
        import dense_tiled_gemm_fp16_amd as g
        if case["op"] == "store":
            return g.dequantize_mx4(g.quantize_mx4(x), x.dtype)
        if case["op"] == "linear":
            return g.gemm_mx4(g.quantize_mx4(x), state["w4"], dtype=x.dtype)
        if case["op"] == "decode":
            return g.gemm_mx4(x, state["w4"])
        up, down = ("gate_up", "down") if case["weights"] == "16" else ("gate_up4", "down4")
        return g.gemm_moe(x, state["logits"], state[up], state[down], case["top_k"],
                          renormalize=case["renormalize"])
    if case["op"] == "store":
        return _through_mx4(x.float()).to(x.dtype)
    if case["op"] == "linear":
        return (_through_mx4(x.float()) @ _unpack(state["w"], case["k"]).t()).to(x.dtype)
    if case["op"] == "decode":
        return (x.float() @ _unpack(state["w"], case["k"]).t()).to(x.dtype)
    return _plain_moe(state)


# ---- what a pass cannot do without

def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "store":
        n = case["rows"] * case["k"]
        packed = case["rows"] * _blocks(case["k"]) * 17
        return {"bytes": 2 * size * n + 2 * packed, "flops": 2 * n}
    if case["op"] in ("linear", "decode"):
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + 17 * n * _blocks(k) + 2 * m * n, "flops": 2 * m * n * k}
    T, E, k, H, I = (case[f] for f in ("tokens", "experts", "top_k", "hidden", "inter"))
    used = E * (1 - (1 - k / E) ** T)              # experts that T independent tokens reach
    if case["weights"] == "16":
        per = 2 * 3 * I * H
    else:
        per = 17 * (2 * I * _blocks(H) + H * _blocks(I))
    return {"bytes": int(used * per) + 4 * T * H + (4 if case["logits"] == "f32" else 2) * T * E,
            "flops": 6 * T * k * I * H}


# ---- the definition in 64 bits

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_through_mx4(x):
    """Each element of a block goes to the nearest multiple of the block's
    scale among the magnitudes; of two equally near ones, to the even code."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // max(1, x.shape[1]))
    for r0 in range(0, x.shape[0], step):
        v = x[r0:r0 + step].double()
        pad = (-v.shape[1]) % BLOCK
        b = torch.cat((v, v.new_zeros(v.shape[0], pad)), dim=1).reshape(v.shape[0], -1, BLOCK)
        m = b.abs().max(dim=2, keepdim=True).values
        exponent = ((m.contiguous().view(torch.int64) >> 52) & 0x7FF) - 1023 - 2
        scale = (exponent.clamp(min=-127) + 1023 << 52).view(torch.float64)
        best = torch.zeros_like(b)
        dist = b.abs().clone()
        for code in (2, 4, 6, 1, 3, 5, 7):         # even codes first: an odd one must be nearer
            d = (b.abs() - MAGNITUDES[code] * scale).abs()
            nearer = d < dist
            best = torch.where(nearer, MAGNITUDES[code] * scale, best)
            dist = torch.where(nearer, d, dist)
        q = torch.where(b < 0, -best, best).reshape(v.shape[0], -1)
        out[r0:r0 + step] = q[:, :v.shape[1]]
    return out


def _exact_unpack(data, exps, k):
    lut = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), dtype=torch.float64, device=data.device)
    out = torch.empty(data.shape[0], 2 * data.shape[1], dtype=torch.float64, device=data.device)
    out[:, 0::2] = lut[(data % 16).long()]
    out[:, 1::2] = lut[(data // 16).long()]
    scale = torch.pow(torch.full((), 2.0, dtype=torch.float64, device=data.device), exps.double() - 127)
    return (out * scale.repeat_interleave(BLOCK, dim=1))[:, :k]


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "store":
        return _exact_through_mx4(s["x"])
    if case["op"] in ("linear", "decode"):
        x = _exact_through_mx4(s["x"]) if case["op"] == "linear" else s["x"].double()
        return x @ _exact_unpack(*s["w"], case["k"]).t()
    T, k, H, I = case["tokens"], case["top_k"], case["hidden"], case["inter"]
    x, logits = s["x"].double(), s["logits"].double()
    rows = logits.tolist()
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    chosen = [sorted(range(len(r)), key=lambda e: (-r[e], e))[:k] for r in rows]
    for e in sorted({e for c in chosen for e in c}):
        tokens = [t for t in range(T) if e in chosen[t]]
        share = []
        for t in tokens:
            over = chosen[t] if case["renormalize"] else range(len(rows[t]))
            share.append(1.0 / math.fsum(math.exp(rows[t][j] - rows[t][e]) for j in over))
        up, down = s["gate_up"], s["down"]
        if case["weights"] == "16":
            up, down = up[e].double(), down[e].double()
        else:
            up = _exact_unpack(up[0][e], up[1][e], H)
            down = _exact_unpack(down[0][e], down[1][e], I)
        z = x[tokens] @ up.t()
        a = z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]
        y[tokens] += torch.tensor(share, dtype=torch.float64, device=x.device)[:, None] * (a @ down.t())
    return y
