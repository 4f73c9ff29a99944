"""Operators around the 8-bit and the grouped products, as a user's program calls
them: 8-bit linear layers with a scale for each block of 128, the norm that
feeds them, and a mixture-of-experts layer's tokens on their way to the
experts and back.

"8 bits" is OCP floating point E4M3 (largest value 448) or E5M2 (57344).  A
block of 128 consecutive elements of a row ("row block"), or of 128 rows x 128
elements ("square block"), shares a float32 scale: with m the largest magnitude
of the block, m / largest value, at least 2^-126.  Elements are divided by
m / largest value (not yet rounded to float32: 16-bit elements often lie midway
between two 8-bit ones) and rounded to nearest, ties to even.  The last block of
a row or column may be shorter.

  norm       h = x + residual, rounded to x's type; y = h / sqrt(mean(h^2) + eps)
             * weight, kept in E4M3 by row blocks: the input of a linear layer,
             and the residual stream
  norm_grad  the gradients of the norm's input and weight, given those of y and
             of the residual stream (the rounding to 8 bits passed straight)
  linear     y = q(x) . w^T: 16-bit activations kept in 8 bits by row blocks on
             the fly, weights in 8 bits by square blocks
  wgrad      dw = q(dy)^T . q(x), both in 8 bits by blocks of 128 tokens
  moe        tokens sorted by expert (stable), the rows each expert gets, and the
             experts' rows back to their tokens, with weights
  moe_grad   its gradients: of the experts' rows, of the weights, of the tokens

listed() and draw() give cases, prepare() a case's inputs, run() one pass,
exact() the same outputs from the definition in 64 bits.  A tensor in 8 bits is
returned as its elements (8-bit floating point) and its scales.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
BLOCK = 128
LEAST = 2.0 ** -126
EPS = 1e-6

# The hidden and intermediate sizes of the expert products of this
# repository's own benchmark.
HIDDEN, INTER = 7168, 2048


def _norm(name, rows, k, dtype, residual, weight="f32"):
    return {"name": name, "op": "norm", "rows": rows, "k": k, "type": dtype, "residual": residual, "weight": weight}


def _norm_grad(name, rows, k, dtype, residual, weight="f32"):
    return {"name": name, "op": "norm_grad", "rows": rows, "k": k, "type": dtype, "residual": residual,
            "weight": weight}


def _linear(name, m, n, k, dtype, f8="e4m3"):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "type": dtype, "f8": f8}


def _wgrad(name, tokens, n, k, dtype, out):
    return {"name": name, "op": "wgrad", "tokens": tokens, "n": n, "k": k, "type": dtype, "out": out}


def _moe(name, op, tokens, experts, top_k, hidden, dtype, weights="f32", padded=0):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden,
            "type": dtype, "weights": weights, "padded": padded}


def listed():
    return [
        # a decode batch's hidden states ahead of a linear layer: latency
        _norm("norm_decode", 16, HIDDEN, "bf16", True),
        # a long prefill's: memory
        _norm("norm_prefill", 32768, HIDDEN, "bf16", True),
        # a training step's backward pass through the same
        _norm_grad("norm_grad", 16384, HIDDEN, "bf16", True),
        # a small model, odd sizes, no residual stream
        _norm_grad("norm_grad_odd", 1031, 2051, "f16", False, "same"),
        # one token through a projection: latency and weights
        _linear("linear_one", 1, INTER, HIDDEN, "bf16"),
        # a decode batch, wide output
        _linear("linear_batch", 48, HIDDEN, INTER, "bf16"),
        # a short ragged prompt, odd sizes
        _linear("linear_odd", 333, 1061, 2050, "f16"),
        # a chunked prefill through an expert's down product
        _linear("linear_prefill", 32768, INTER, HIDDEN, "bf16"),
        # a training step's weight gradient over 8192 tokens
        _wgrad("wgrad", 8192, INTER, HIDDEN, "bf16", "f32"),
        # a padded decode batch of a mixture-of-experts model: latency
        _moe("moe_decode", "moe", 48, 64, 8, HIDDEN, "bf16", padded=5),
        # a prefill's tokens to 64 experts and back: memory
        _moe("moe_prefill", "moe", 16384, 64, 8, HIDDEN, "bf16"),
        # a training step's backward pass through the same, a smaller batch
        _moe("moe_grad", "moe_grad", 4096, 64, 8, HIDDEN, "bf16"),
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
    op = rng.choice(["norm", "norm_grad", "linear", "linear", "wgrad", "moe", "moe_grad"])
    half = rng.choice(["f16", "bf16"])
    if op == "norm":
        c = _norm("", _log_size(rng, 1, 32768), _log_size(rng, 64, HIDDEN), half, rng.random() < 0.5,
                  rng.choice(["f32", "same"]))
    elif op == "norm_grad":
        c = _norm_grad("", _log_size(rng, 1, 16384), _log_size(rng, 64, HIDDEN), half, rng.random() < 0.5,
                       rng.choice(["f32", "same"]))
    elif op == "linear":
        c = _linear("", _log_size(rng, 1, 32768), _log_size(rng, 64, 8192), _log_size(rng, 64, 8192), half,
                    rng.choice(["e4m3", "e4m3", "e5m2"]))
        while c["m"] * c["n"] * c["k"] > 32768 * INTER * HIDDEN:
            c["n"] = max(64, c["n"] // 2)
    elif op == "wgrad":
        c = _wgrad("", _log_size(rng, 32, 8192), _log_size(rng, 64, 4096), _log_size(rng, 64, 4096), half,
                   rng.choice(["f32", "same"]))
    else:
        experts = _log_size(rng, 2, 256)
        c = _moe("", op, _log_size(rng, 1, 16384 if op == "moe" else 4096), experts,
                 rng.randint(1, min(8, experts)), _log_size(rng, 64, HIDDEN), half, rng.choice(["f32", "same"]))
        if rng.random() < 0.5:
            c["padded"] = rng.randint(0, c["tokens"] // 4)
    del c["name"]
    return c


# ---- inputs

def _activations(gen, m, k, dtype):
    """Unit-variance rows, a few channels of which run larger, as hidden
    states have them."""
    x = torch.randn(m, k, generator=gen, device="cuda", dtype=torch.float32)
    gain = torch.ones(k, device="cuda")
    gain[torch.randint(0, k, (max(1, k // 128),), generator=gen, device="cuda")] = 8.0
    return (x * gain).to(dtype)


def _gradients(gen, m, k, dtype):
    """Rows of gradients, small and of different size from row to row."""
    x = torch.randn(m, k, generator=gen, device="cuda", dtype=torch.float32)
    return (x * torch.exp(torch.randn(m, 1, generator=gen, device="cuda") - 6)).to(dtype)


def _f8_rows(values, dtype):
    """8-bit elements in rows that start 16-byte aligned."""
    n, k = values.shape
    data = torch.zeros(n, -(-k // 16) * 16, dtype=torch.uint8, device=values.device).view(dtype)[:, :k]
    data.copy_(values)
    return data


def _routing(gen, T, E, k, padded):
    """Experts by logits that favour some, the last tokens without any."""
    logits = torch.randn(T, E, generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k].contiguous()
    p = torch.exp(top - top[:, :1])
    if padded:
        ids[T - padded:] = -1
    return ids, p / p.sum(dim=1, keepdim=True)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    dtype = TYPES[case["type"]]
    if case["op"] in ("norm", "norm_grad"):
        R, K = case["rows"], case["k"]
        w = 1 + 0.2 * torch.randn(K, generator=gen, device="cuda")
        s["w"] = w if case["weight"] == "f32" else w.to(dtype)
        s["x"] = _activations(gen, R, K, dtype)
        if case["op"] == "norm":
            s["residual"] = (2 * _activations(gen, R, K, torch.float32)).to(dtype) if case["residual"] else None
        else:
            s["dy"] = _gradients(gen, R, K, dtype)
            s["dh"] = _gradients(gen, R, K, dtype) if case["residual"] else None
        return s
    if case["op"] == "linear":
        s["x"] = _activations(gen, case["m"], case["k"], dtype)
        w = torch.randn(case["n"], case["k"], generator=gen, device="cuda") * case["k"] ** -0.5
        values, s["w_scales"] = _quantise(w, BLOCK, torch.float8_e4m3fn)
        s["w"] = _f8_rows(values, torch.float8_e4m3fn)
        return s
    if case["op"] == "wgrad":
        s["x"] = _activations(gen, case["tokens"], case["k"], dtype)
        s["dy"] = _gradients(gen, case["tokens"], case["n"], dtype)
        return s
    T, E, k, H = case["tokens"], case["experts"], case["top_k"], case["hidden"]
    s["ids"], p = _routing(gen, T, E, k, case["padded"])
    s["p"] = p if case["weights"] == "f32" else p.to(dtype)
    s["rows"] = torch.randn(T * k, H, generator=gen, device="cuda", dtype=dtype)   # the experts' outputs
    if case["op"] == "moe":
        s["x"] = _activations(gen, T, H, dtype)
    else:
        s["dy"] = _gradients(gen, T, H, dtype)
        s["drows"] = _gradients(gen, T * k, H, dtype)                              # gradients of their inputs
        s["order"] = _order(s["ids"], E)                                           # as the forward pass left it
    return s


# ---- the plain forms

def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _quantise(x, rows, dtype):
    """float32 x [R, K] in blocks of rows x 128 -> (quotients before they are
    rounded, in 64 bits so that ties stay ties, and scales)."""
    R, K = x.shape
    p = torch.zeros(-(-R // rows) * rows, _blocks(K) * BLOCK, device=x.device)
    p[:R, :K] = x
    b = p.view(-1, rows, _blocks(K), BLOCK)
    m = b.abs().amax(dim=(1, 3)).clamp(min=LARGEST[dtype] * LEAST)
    quotients = b.double() * LARGEST[dtype] / m.double()[:, None, :, None]
    return quotients.view(p.shape)[:R, :K], m / LARGEST[dtype]


def _values(q, scales):
    """8-bit elements and their scales -> float32."""
    n, k = q.shape
    s = scales if scales.shape[0] == n else scales.repeat_interleave(BLOCK, dim=0)[:n]
    return q.float() * s.repeat_interleave(BLOCK, dim=1)[:, :k]


def _through_f8(x, dtype):
    values, scales = _quantise(x, 1, dtype)
    return _values(values.to(dtype), scales)


def _plain_norm(s):
    case, h = s["case"], s["x"]
    dtype = F8["e4m3"]
    if case["residual"]:
        h = (h.float() + s["residual"].float()).to(h.dtype)
    v = h.float()
    y = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS) * s["w"].float()
    values, scales = _quantise(y, 1, dtype)
    return [values.to(dtype), scales] + ([h] if case["residual"] else [])


def _plain_norm_grad(s):
    v, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
    r = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    g = dy * w
    dx = r * (g - v * (r * r * (g * v).mean(dim=1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dw = (dy * v * r).sum(dim=0)
    return [dx.to(s["x"].dtype), dw.to(s["w"].dtype)]


def _order(ids, E):
    """(offsets [E + 1], rows [P], slots like ids): the pairs (token, choice)
    sorted by expert, in order within one; ids outside 0 .. E - 1 have no slot,
    and rows behind the last expert's are -1."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    key, rows = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=ids.device))
    at = torch.arange(flat.numel(), device=ids.device)
    slots = torch.empty_like(at).scatter_(0, rows, torch.where(key < E, at, -1))
    return offsets, torch.where(key < E, rows, -1), slots.view(ids.shape)


def _back(rows, slots, weights):
    """sum over a token's choices of weight times its row, in float32."""
    T, k = slots.shape
    w = torch.where(slots < 0, 0.0, 1.0 if weights is None else weights.float())
    return (rows[slots.clamp(min=0)].float() * w[:, :, None]).sum(dim=1)


def _plain_moe(s):
    case, k = s["case"], s["case"]["top_k"]
    offsets, rows, slots = _order(s["ids"], case["experts"])
    x = torch.where(rows[:, None] < 0, 0.0, s["x"].float()[rows.clamp(min=0) // k])
    return [offsets, rows, slots, x.to(s["x"].dtype), _back(s["rows"], slots, s["p"]).to(s["x"].dtype)]


def _plain_moe_grad(s):
    k = s["case"]["top_k"]
    offsets, rows, slots = s["order"]
    at = rows.clamp(min=0)
    dy = s["dy"].float()
    none = (rows < 0)[:, None]
    drows = torch.where(none, 0.0, dy[at // k] * s["p"].float().reshape(-1)[at][:, None])
    dots = (dy[:, None] * s["rows"][slots.clamp(min=0)].float()).sum(dim=2)
    dp = torch.where(slots < 0, 0.0, dots)
    return [drows.to(s["dy"].dtype), dp.to(s["p"].dtype), _back(s["drows"], slots, None).to(s["dy"].dtype)]


def run(state):
    case = state["case"]
    if own:
        import dense_tiled_gemm_fp16_amd as g
        if case["op"] == "norm":
            data, scales, h = g.rms_norm_f8(state["x"], state["w"], EPS, residual=state["residual"])
            return [data, scales, h] if case["residual"] else [data, scales]
        if case["op"] == "norm_grad":
            return list(g.rms_norm_backward(state["dy"], state["x"], state["w"], EPS, dh=state["dh"]))
        if case["op"] == "linear":
            x, scales = g.quantize_f8(state["x"], dtype=F8[case["f8"]])
            return g.gemm_f8_scaled(x, scales, state["w"], state["w_scales"], dtype=state["x"].dtype)
        if case["op"] == "wgrad":
            dy, dy_scales = g.quantize_f8(state["dy"].t(), dtype=torch.float8_e5m2)
            x, x_scales = g.quantize_f8(state["x"].t())
            return g.gemm_f8_scaled(dy, dy_scales, x, x_scales,
                                    dtype=torch.float32 if case["out"] == "f32" else state["x"].dtype)
        if case["op"] == "moe":
            order = g.moe_sort(state["ids"], case["experts"])
            x = g.moe_gather(state["x"], order)
            return [*order, x, g.moe_combine(state["rows"], order, state["p"])]
        order = g.MoeOrder(*state["order"])
        drows, dp = g.moe_combine_backward(state["dy"], state["rows"], order, state["p"])
        return [drows, dp, g.moe_combine(state["drows"], order)]
    if case["op"] == "norm":
        return _plain_norm(state)
    if case["op"] == "norm_grad":
        return _plain_norm_grad(state)
    if case["op"] == "linear":
        x = _through_f8(state["x"].float(), F8[case["f8"]])
        return (x @ _values(state["w"], state["w_scales"]).t()).to(state["x"].dtype)
    if case["op"] == "wgrad":
        dy = _through_f8(state["dy"].t().float(), torch.float8_e5m2)
        x = _through_f8(state["x"].t().float(), torch.float8_e4m3fn)
        return (dy @ x.t()).to(torch.float32 if case["out"] == "f32" else state["x"].dtype)
    return _plain_moe(state) if case["op"] == "moe" else _plain_moe_grad(state)


# ---- what a pass cannot do without

def work(case):
    if case["op"] in ("norm", "norm_grad"):
        n = case["rows"] * case["k"]
        if case["op"] == "norm":
            passes = 3 * 2 if case["residual"] else 2
            return {"bytes": passes * n + n + 4 * case["rows"] * _blocks(case["k"]), "flops": 8 * n}
        return {"bytes": 2 * n * (4 if case["residual"] else 3), "flops": 12 * n}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k + 4 * _blocks(n) * _blocks(k) + 2 * m * n, "flops": 2 * m * n * k}
    if case["op"] == "wgrad":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": 2 * t * (n + k) + (4 if case["out"] == "f32" else 2) * n * k, "flops": 2 * t * n * k}
    P, H = (case["tokens"] - case["padded"]) * case["top_k"], case["hidden"]
    row, p = 2 * H, (4 if case["weights"] == "f32" else 2) * case["tokens"] * case["top_k"]
    if case["op"] == "moe":                      # x once, rows out, rows in, y; ids, offsets, rows, slots
        return {"bytes": row * (2 * case["tokens"] + 2 * P) + p + 24 * case["tokens"] * case["top_k"],
                "flops": 2 * P * H}
    return {"bytes": row * (2 * case["tokens"] + 3 * P) + 2 * p + 16 * case["tokens"] * case["top_k"],
            "flops": 4 * P * H}


# ---- the definition in 64 bits

def _exact_quotients(x, dtype):
    """float64 rows brought to the 8-bit range by blocks: the values that 8 bits
    round, and the blocks' scales, unrounded."""
    R, K = x.shape
    pad = x.new_zeros(R, _blocks(K) * BLOCK - K)
    b = torch.cat((x, pad), dim=1).reshape(R, -1, BLOCK)
    m = torch.maximum(b.abs().max(dim=2).values, x.new_full((), LEAST * LARGEST[dtype]))
    return ((LARGEST[dtype] * b) / m.unsqueeze(2)).reshape(R, -1)[:, :K], m / LARGEST[dtype]


def _exact_round(v, dtype):
    """v to the nearest 8-bit value of |v| <= largest, ties to even."""
    bits, least = (3, -6) if dtype == torch.float8_e4m3fn else (2, -14)
    exponent = ((v.contiguous().view(torch.int64) >> 52) & 0x7FF) - 1023
    step = ((exponent.clamp(min=least) - bits + 1023) << 52).view(torch.float64)
    return (v / step).round() * step             # round(): ties to even


def _exact_through_f8(x, dtype):
    """Rows x of any type; a part of them at a time."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // x.shape[1])
    for r in range(0, x.shape[0], step):
        v, scales = _exact_quotients(x[r:r + step].double(), dtype)
        top = LARGEST[dtype]
        q = _exact_round(v.clamp(-top, top), dtype)
        out[r:r + step] = q * scales.float().double().repeat_interleave(BLOCK, dim=1)[:, :x.shape[1]]
    return out


def _exact_weights(q, scales):
    n, k = q.shape
    at = torch.arange(n, device=q.device) // BLOCK, torch.arange(k, device=q.device) // BLOCK
    return q.double() * scales.double()[at[0][:, None], at[1][None, :]]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:
            h = h + s["residual"].double()
        v = h.to(s["x"].dtype).double()
        y = v * s["w"].double() * ((v * v).sum(dim=1, keepdim=True) / case["k"] + EPS).rsqrt()
        quotients, scales = _exact_quotients(y, F8["e4m3"])
        return [quotients, scales] + ([h] if case["residual"] else [])
    if case["op"] == "norm_grad":
        K = case["k"]
        v, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        m = (v * v).sum(dim=1, keepdim=True) / K + EPS
        dx = dy * w * m.rsqrt() - v * (dy * w * v).sum(dim=1, keepdim=True) / (K * m * m.sqrt())
        if case["residual"]:
            dx = dx + s["dh"].double()
        return [dx, (dy * v * m.rsqrt()).sum(dim=0)]
    if case["op"] == "linear":
        return _exact_through_f8(s["x"], F8[case["f8"]]) @ _exact_weights(s["w"], s["w_scales"]).t()
    if case["op"] == "wgrad":
        return (_exact_through_f8(s["dy"].t(), torch.float8_e5m2) @
                _exact_through_f8(s["x"].t(), torch.float8_e4m3fn).t())
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    chosen = [[] for _ in range(E)]                # pairs of each expert
    flat = s["ids"].reshape(-1).tolist()
    for pair, e in enumerate(flat):
        if 0 <= e < E:
            chosen[e].append(pair)
    pairs = [p for c in chosen for p in c]
    offsets, slots = [0], [-1] * (T * k)
    for c in chosen:
        offsets.append(offsets[-1] + len(c))
    for slot, p in enumerate(pairs):
        slots[p] = slot
    dev = s["ids"].device
    P = len(pairs)
    rows = torch.tensor(pairs, dtype=torch.int64, device=dev)
    p = s["p"].double().reshape(-1)[rows].unsqueeze(1)
    if case["op"] == "moe":
        to = torch.zeros(T * k, case["hidden"], dtype=torch.float64, device=dev)
        to[:P] = s["x"][rows // k].double()
        y = torch.zeros(T, case["hidden"], dtype=torch.float64, device=dev)
        y.index_add_(0, rows // k, s["rows"][:P].double() * p)
        return [torch.tensor(offsets, device=dev), torch.tensor(pairs + [-1] * (T * k - P), device=dev),
                torch.tensor(slots, device=dev).view(T, k), to, y]
    dy = s["dy"].double()[rows // k]
    drows = torch.zeros(T * k, case["hidden"], dtype=torch.float64, device=dev)
    drows[:P] = dy * p
    dp = torch.zeros(T * k, dtype=torch.float64, device=dev)
    dp[rows] = (dy * s["rows"][:P].double()).sum(dim=1)
    dx = torch.zeros(T, case["hidden"], dtype=torch.float64, device=dev)
    dx.index_add_(0, rows // k, s["drows"][:P].double())
    return [drows, dp.view(T, k), dx]
