"""The 8-bit, norm and row-sort operators as a program calls them: on streams by
argument, captured in graphs and replayed beside other work, without a
workspace, two at a time, and on matrices larger than the caches or than 32-bit
offsets reach."""
import ctypes

import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
import f8_ref as ref
from dense_tiled_gemm_fp16_amd import _lib
from gpu_util import DEV, say
from test_streams import CYCLES, Elsewhere, dropped

pytestmark = pytest.mark.gpu
F16, BF16, F32, E4M3, E5M2 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2


def randn(*shape, dtype=BF16, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device=DEV).to(dtype)


def ids(T, k, E, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.randint(-1, E, (T, k), generator=gen, device=DEV)


def same(got, want):
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def weights8(N, K, rows, seed=1):
    return tuple(t.clone() for t in g.quantize_f8(randn(N, K, seed=seed), rows))


T, k, E, H = 3000, 3, 16, 500          # more pairs than one workgroup sorts
ORDER = lambda: tuple(g.moe_sort(ids(T, k, E), E))
CALLS = {
    "quantize": (lambda: (randn(700, 3000),), lambda x, stream: g.quantize_f8(x, stream=stream)),
    "quantize square": (lambda: (randn(700, 3000),), lambda x, stream: g.quantize_f8(x, 128, stream=stream)),
    "product strips": (lambda: (*weights8(20, 1008, 1), *weights8(700, 1008, 128)),
                       lambda a, s, b, t, stream: [g.gemm_f8_scaled(a, s, b, t, stream=stream)]),
    "product tiles": (lambda: (*weights8(1500, 1008, 1), *weights8(1700, 1008, 1)),
                      lambda a, s, b, t, stream: [g.gemm_f8_scaled(a, s, b, t, dtype=F32, stream=stream)]),
    "norm": (lambda: (randn(500, 3000), randn(3000, dtype=F32), randn(500, 3000, seed=1)),
             lambda x, w, r, stream: g.rms_norm_f8(x, w, residual=r, stream=stream)),
    "norm backward": (lambda: (randn(500, 3000), randn(3000, dtype=F32), randn(500, 3000, seed=1), randn(500, 3000, seed=2)),
                      lambda h, w, y, d, stream: g.rms_norm_backward(y, h, w, dh=d, stream=stream)),
    "sort": (lambda: (ids(T, k, E),), lambda e, stream: g.moe_sort(e, E, stream=stream)),
    "gather": (lambda: (randn(T, H), *ORDER()), lambda x, o, r, s, stream: [g.moe_gather(x, g.MoeOrder(o, r, s), stream=stream)]),
    "combine": (lambda: (randn(T * k, H), randn(T, k, dtype=F32), *ORDER()),
                lambda y, w, o, r, s, stream: [g.moe_combine(y, g.MoeOrder(o, r, s), w, stream=stream)]),
    "combine backward": (lambda: (randn(T, H), randn(T * k, H, seed=2), randn(T, k, dtype=F32), *ORDER()),
                         lambda d, y, w, o, r, s, stream: g.moe_combine_backward(d, y, g.MoeOrder(o, r, s), w, stream=stream)),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_inputs_of_a_stream_by_argument(name):
    make, call = CALLS[name]
    say(f"stream inputs {name}")
    want, got = dropped(torch.cuda.Stream(DEV), make, call)
    same(got, want)


@pytest.mark.parametrize("name", list(CALLS))
def test_results_take_no_memory_in_use(name):
    make, call = CALLS[name]
    side = torch.cuda.Stream(DEV)
    inputs = make()
    want = call(*inputs, stream=None)
    say(f"stream results {name}")
    torch.cuda.synchronize()
    held = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device=DEV) for t in want]
    torch.cuda._sleep(CYCLES)
    for t in held:
        t.fill_(9)
    del held, t
    got = call(*inputs, stream=side)
    torch.cuda.synchronize()
    same(got, want)


@pytest.mark.parametrize("name", list(CALLS))
def test_stream_of_another_device(name):
    make, call = CALLS[name]
    say(f"stream of another device {name}")
    inputs = make()
    with pytest.raises(ValueError):
        call(*inputs, stream=Elsewhere())


@pytest.mark.parametrize("name", list(CALLS))
def test_two_at_a_time(name):
    make, call = CALLS[name]
    say(f"two at a time {name}")
    inputs = make()
    want = call(*inputs, stream=None)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(DEV) for _ in range(2)]
    got = [call(*inputs, stream=s) for _ in range(5) for s in sides]
    torch.cuda.synchronize()
    for y in got:
        same(y, want)


# ---- graphs

def layer(x, r, wn, w8, w8t, dy):
    """Norm, projection, and their backward pass."""
    a, sa, h = g.rms_norm_f8(x, wn, residual=r)
    y = g.gemm_f8_scaled(a, sa, *w8, dtype=BF16)
    d, sd = g.quantize_f8(dy, dtype=E5M2)
    da = g.gemm_f8_scaled(d, sd, *w8t, dtype=BF16)
    dw = g.gemm_f8_scaled(*g.quantize_f8(dy.t(), dtype=E5M2), *g.quantize_f8(x.t()), dtype=F32)
    return [a, sa, h, y, da, dw, *g.rms_norm_backward(da, h, wn, dh=r)]


def experts(x, e, p, dy):
    order = g.moe_sort(e, E)
    rows = g.moe_gather(x, order)
    return [*order, rows, g.moe_combine(rows, order, p), *g.moe_combine_backward(dy, rows, order, p),
            g.moe_combine(rows, order)]


def layer_inputs(M, K, N, seed):
    w = randn(N, K, seed=seed + 1)
    return [randn(M, K, seed=seed), randn(M, K, seed=seed + 2), randn(K, dtype=F32, seed=seed + 3),
            g.quantize_f8(w, 128), g.quantize_f8(w.t(), 128), randn(M, N, seed=seed + 4)]


def experts_inputs(tokens, seed):
    return [randn(tokens, H, seed=seed), ids(tokens, k, E, seed), randn(tokens, k, dtype=F32, seed=seed + 1),
            randn(tokens, H, seed=seed + 2)]


def copy_into(to, new):
    for a, b in zip(to, new):
        if isinstance(a, torch.Tensor):
            a.copy_(b)
        else:
            copy_into(a, b)


RUNS = {"layer of one token": (layer, lambda s: layer_inputs(1, 700, 300, s)),
        "layer": (layer, lambda s: layer_inputs(400, 700, 300, s)),
        "large layer": (layer, lambda s: layer_inputs(1100, 1024, 1300, s)),
        "experts of few tokens": (experts, lambda s: experts_inputs(5, s)),
        "experts": (experts, lambda s: experts_inputs(T, s))}


@pytest.mark.parametrize("name", list(RUNS))
def test_graphs(name):
    """Two captured graphs of one kind replayed in turn, inputs changed and other
    work done between the replays."""
    fn, make = RUNS[name]
    say(f"graph {name}: eager")
    inputs = [make(10), make(20)]
    fn(*inputs[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        say(f"graph {name}: capture {i}")
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(fn(*inputs[i]))
    for turn in range(3):
        wants = []
        for i in range(2):
            copy_into(inputs[i], make(30 + 10 * turn + 5 * i))
            wants.append([t.clone() for t in fn(*inputs[i])])
            for t in outs[i]:
                t.view(torch.uint8).fill_(0xFF)
        say(f"graph {name}: replay {turn}")
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        junk = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        for i in range(2):
            same(outs[i], wants[i])


def test_graphs_beside_each_other():
    """Graphs of the calls that take workspaces, replayed on two streams at once."""
    say("graphs beside each other")
    make = [lambda s: experts_inputs(T, s), lambda s: layer_inputs(400, 700, 300, s)]
    fns, inputs = [experts, layer], [make[0](1), make[1](2)]
    wants = [[t.clone() for t in fn(*x)] for fn, x in zip(fns, inputs)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for fn, x in zip(fns, inputs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(fn(*x))
    sides = [torch.cuda.Stream(DEV) for _ in graphs]
    for turn in range(3):
        for o in outs:
            for t in o:
                t.view(torch.uint8).fill_(0xFF)
        torch.cuda.synchronize()
        for s, gr in zip(sides, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            same(o, w)


# ---- without a workspace

def test_norm_backward_without_a_workspace():
    R, K = 300, 2000
    dy, h, w = randn(R, K), randn(R, K, seed=1), randn(K, dtype=F32, seed=2)
    dx, dw = g.rms_norm_backward(dy, h, w)
    outs = [(torch.zeros_like(dx), torch.zeros_like(dw)) for _ in range(3)]
    say("norm backward without a workspace")
    stream = torch.cuda.current_stream().cuda_stream
    for a, b in outs:
        args = _lib.NormBackwardArgs(dy.data_ptr(), K, h.data_ptr(), K, w.data_ptr(), 0, 0, a.data_ptr(), K, b.data_ptr(), R,
                                     K, 1e-6, 1, 2)
        assert g.lib.gemm_rms_norm_backward(ctypes.byref(args), stream, 0, 0) == 0
    torch.cuda.synchronize()
    for out in outs:
        same(out, (dx, dw))


def test_sort_without_a_workspace():
    e = ids(T * 4, k, E)
    want = g.moe_sort(e, E)
    outs = [tuple(torch.zeros_like(t) for t in want) for _ in range(3)]
    say("sort without a workspace")
    stream = torch.cuda.current_stream().cuda_stream
    for o in outs:
        args = _lib.SortArgs(e.data_ptr(), k, T * 4, *(t.data_ptr() for t in o), 8, k, E)
        assert g.lib.gemm_moe_sort(ctypes.byref(args), stream, 0, 0) == 0
    torch.cuda.synchronize()
    for o in outs:
        same(o, want)


@pytest.mark.parametrize("K", [3, 7, 8, 9, 12, 15, 505, 506, 507, 508, 509, 510, 511, 1025, 1027, 1031, 2053, 4103, 8199])
@pytest.mark.parametrize("dtype,res", [(BF16, True), (F16, False)])
def test_norm_backward_of_rows_that_end_inside_an_octet(K, dtype, res):
    """Rows inside a field of NaN, on any side of them."""
    R = 70
    say(f"norm backward tails {K} {dtype}")
    rows = []
    for seed in range(3):
        field = torch.full((R + 2, K + 11), float("nan"), dtype=dtype, device=DEV)
        field[1:-1, 5:5 + K] = randn(R, K, dtype=dtype, seed=seed)
        rows.append(field[1:-1, 5:5 + K])
    dy, h, dh = rows
    dh, w = dh if res else None, randn(K, dtype=F32, seed=4)
    out = torch.full((R + 2, K + 11), 3.0, dtype=dtype, device=DEV)
    dx, dw = g.rms_norm_backward(dy, h, w, 1e-6, dh=dh, out=out[1:-1, 5:5 + K])
    wx, tx, ww, tw = ref.norm_grad(dy, h, w, 1e-6, dh)
    ref.assert_near(dx, wx, tx + ref.half_step(np.abs(wx) + tx, dtype), "dx")
    ref.assert_near(dw, ww, tw + ref.half_step(np.abs(ww) + tw, F32), "dw")
    assert (out[0] == 3).all() and (out[-1] == 3).all() and (out[:, :5] == 3).all() and (out[:, 5 + K:] == 3).all()


@pytest.mark.parametrize("R,K", [(300, 16384), (300, 16392), (290, 20001), (260, 65536)])
def test_norm_backward_of_wide_rows_in_place(R, K):
    """More rows than workgroups, and dx where dy or dh was."""
    say(f"wide norm backward {R}x{K}")
    dy, h, dh, w = randn(R, K), randn(R, K, seed=1), randn(R, K, seed=3), randn(K, dtype=F32, seed=2)
    dx, dw = g.rms_norm_backward(dy, h, w, dh=dh)
    hd, y = h.double(), dy.double()
    r = 1 / (hd.square().mean(dim=1, keepdim=True) + 1e-6).sqrt()
    yw = y * w.double()
    c = (yw * hd).mean(dim=1, keepdim=True) * r * r
    want, mag = r * (yw - hd * c) + dh.double(), r * (yw.abs() + (hd * c).abs()) + dh.double().abs()
    cmag = (yw * hd).abs().mean(dim=1, keepdim=True) * r * r * hd.abs() * r
    # dx: half a step of bfloat16; r and c within 100 float32 roundings of their terms
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -24 * (100 * cmag + 120 * mag)).all()
    terms = y * hd * r
    # dw: at most 2 rows of a workgroup and R workgroups added, 60 roundings in a term
    assert ((dw.double() - terms.sum(dim=0)).abs() <= (R + 60) * 2.0 ** -24 * terms.abs().sum(dim=0)).all()
    for i in range(2):
        a, b = dy.clone(), dh.clone()
        same(g.rms_norm_backward(a, h, w, dh=b, out=(a, b)[i]), (dx, dw))


# ---- larger than the caches: the same rows in parts have the same bits

def test_large_norm():
    R, K, part = 20001, 7168, 4000
    say("large norm")
    x, r, w = randn(R, K), randn(R, K, seed=1), randn(K, dtype=F32, seed=2)
    for res in (None, r):
        whole = g.rms_norm_f8(x, w, residual=res)
        for i in range(0, R, part):
            cut = slice(i, i + part)
            same([t[cut] for t in whole], g.rms_norm_f8(x[cut], w, residual=None if res is None else res[cut]))


def test_large_norm_backward():
    R, K, part = 14001, 7168, 3000
    say("large norm backward")
    dy, h, dh, w = randn(R, K), randn(R, K, seed=1), randn(R, K, seed=3), randn(K, dtype=F32, seed=2)
    for d in (None, dh):
        dx, dw = g.rms_norm_backward(dy, h, w, dh=d)
        sums, mags = torch.zeros(K, dtype=torch.float64, device=DEV), torch.zeros(K, dtype=torch.float64, device=DEV)
        for i in range(0, R, part):
            cut = slice(i, i + part)
            same([dx[cut]], g.rms_norm_backward(dy[cut], h[cut], w, dh=None if d is None else d[cut])[:1])
            hd = h[cut].double()
            terms = dy[cut].double() * hd / (hd.square().mean(dim=1, keepdim=True) + 1e-6).sqrt()
            sums, mags = sums + terms.sum(dim=0), mags + terms.abs().sum(dim=0)
        # at most 76 additions in a row (28 rows of a workgroup, 32 workgroups of a group of
        # lanes, 16 groups), and in each term 40 roundings at most, each 2^-24
        assert ((dw.double() - sums).abs() <= 120 * 2.0 ** -24 * mags).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_quantize(dtype):
    R, K, part = 24001, 7168, 6400
    say(f"large quantize {dtype}")
    x = randn(R, K, dtype=dtype)
    for rows in (1, 128):
        data, scales = g.quantize_f8(x, rows)
        for i in range(0, R, part):
            d, s = g.quantize_f8(x[i:i + part], rows)
            same([data[i:i + part], scales[i // rows:(i + part) // rows if i + part < R else None]], [d, s])


def test_large_rows_there_and_back():
    """More than the caches hold, and slots behind 4 GiB."""
    tokens, top, width = 41000, 8, 7168
    say("large rows")
    e = ids(tokens, top, E, 3)
    order = g.moe_sort(e, E)
    x, p = randn(tokens, width), randn(tokens, top, dtype=F32, seed=1)
    rows = g.moe_gather(x, order)
    assert rows.numel() * 2 > 1 << 32
    n = int(order.offsets[-1])
    for i in range(0, tokens * top, 50000):
        of = order.rows[i:i + 50000]
        want = torch.where(of[:, None] < 0, torch.zeros((), dtype=BF16, device=DEV), x[of.clamp(min=0) // top])
        assert torch.equal(rows[i:i + 50000], want)
    assert 0 < n < tokens * top and not rows[n:].any()
    # one token's rows are copies of it, so its sum is its weights' sum times it
    slots = order.slots
    y, (dy, dp) = g.moe_combine(rows, order, p), g.moe_combine_backward(x, rows, order, p)
    there = (slots >= 0).double()
    wsum, wmag = (p.double() * there).sum(dim=1, keepdim=True), (p.double().abs() * there).sum(dim=1, keepdim=True)
    for i in range(0, tokens, 10000):
        cut = slice(i, i + 10000)
        xd = x[cut].double()
        tol = 2.0 ** -8 * (wsum[cut] * xd).abs() * 1.01 + 10 * 2.0 ** -24 * wmag[cut] * xd.abs()
        assert ((y[cut].double() - wsum[cut] * xd).abs() <= tol).all()
        dots = (xd * xd).sum(dim=1, keepdim=True) * there[cut]
        # 4 octets of 8 products a lane, six exchanges, four waves
        assert ((dp[cut].double() - dots).abs() <= 50 * 2.0 ** -24 * dots).all()
        for j in range(top):
            s = slots[cut, j]
            live = s >= 0
            assert torch.equal(dy[s[live]], (x[cut][live].float() * p[cut, j][live, None]).to(BF16))
    assert not dy[n:].any()


@pytest.mark.parametrize("variant", ["tile64x128", "tile128x128", "tile256x256", "strip64x64"])
def test_product_behind_32_bit_offsets(variant):
    M, N, K, part = (1 << 20) + 300, 200, 4112, 700
    say(f"large product {variant}")
    a = torch.empty(M, K, dtype=torch.uint8, device=DEV)
    for i in range(0, M, 1 << 17):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(i)
        a[i:i + (1 << 17)] = torch.randint(0, 0x70, (min(1 << 17, M - i), K), generator=gen, device=DEV, dtype=torch.uint8)
    a = a.view(E4M3)
    assert a.numel() > 1 << 32
    sa = torch.rand(M, -(-K // 128), device=DEV) + 0.5
    b, sb = weights8(N, K, 128)
    c = g.gemm_f8_scaled(a, sa, b, sb, dtype=BF16, variant=variant)
    for i in (0, 1 << 19, M - part):
        same([c[i:i + part]], [g.gemm_f8_scaled(a[i:i + part], sa[i:i + part], b, sb, dtype=BF16, variant=variant)])


def test_norm_and_quantize_behind_32_bit_offsets():
    R, K, part = 530000, 8200, 900
    say("norm behind 32 bits")
    x = torch.empty(R, K, dtype=BF16, device=DEV).normal_()
    w = randn(K, dtype=F32, seed=2)
    assert x.numel() > 1 << 32
    data, scales, h = g.rms_norm_f8(x, w, residual=x)
    d8, s8 = g.quantize_f8(x)
    for i in (0, R // 2, R - part):
        cut = slice(i, i + part)
        same([data[cut], scales[cut], h[cut]], g.rms_norm_f8(x[cut], w, residual=x[cut]))
        same([d8[cut], s8[cut]], g.quantize_f8(x[cut]))
    del data, scales, d8, s8
    dx, _ = g.rms_norm_backward(x, h, w, dh=x)
    for i in (0, R // 2, R - part):
        cut = slice(i, i + part)
        same([dx[cut]], g.rms_norm_backward(x[cut], h[cut], w, dh=x[cut])[:1])


# ---- orders that no sort made

@pytest.mark.parametrize("end", [2 ** 63 - 1, -2 ** 63, 10 ** 12, 0])
def test_offsets_of_any_value_clear_nothing_outside(end):
    say(f"offsets {end}")
    tokens, top, width = 6, 2, 40
    slots = torch.arange(tokens * top, device=DEV).reshape(tokens, top)
    order = g.MoeOrder(torch.tensor([0, end], device=DEV), slots.reshape(-1), slots)
    x, p = randn(tokens, width), torch.ones(tokens, top, device=DEV)
    if end <= 0:
        slots.fill_(-1)
        order = order._replace(slots=slots)
    buf = torch.full((tokens * top + 2, width), 3.0, dtype=BF16, device=DEV)
    want = torch.zeros(tokens * top, width, dtype=BF16, device=DEV) if end <= 0 else x.repeat_interleave(top, 0)
    assert torch.equal(g.moe_gather(x, order, out=buf[1:-1]), want)
    assert (buf[0] == 3).all() and (buf[-1] == 3).all()
    rows = randn(tokens * top, width, seed=2)
    assert torch.equal(g.moe_combine_backward(x, rows, order, p, out=buf[1:-1])[0], want)
    assert (buf[0] == 3).all() and (buf[-1] == 3).all()
