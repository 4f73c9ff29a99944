"""MX FP4 on the GPU against its definition in 64 bits (mx4_ref).

Quantisation and its inverse are exact arithmetic followed by one rounding,
so they have to match bit for bit.  Products are compared with the tolerance
of mx4_ref.product_tolerance, which counts the fp32 sums and the output's
rounding, and bit for bit where every sum is exact."""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
import mx4_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def host64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def mx4(data, scales, K):
    return g.MX4(dev(data), dev(scales), K)


def inputs(rng, R, K, dtype):
    """Normal values over many binades, whole blocks of zeros, ties, and the
    type's extremes."""
    x = rng.standard_normal((R, K)) * np.exp2(rng.integers(-12, 8, (R, 1)))
    x[rng.random((R, K)) < 0.1] = 0
    ties = rng.random((R, K)) < 0.2
    x[ties] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -2.5, -7.0, -0.0], ties.sum())
    if K > 40:
        x[0, 32:] = 0
    t = torch.from_numpy(x).to(dtype)
    info = torch.finfo(dtype)
    t[-1, 0] = info.max
    if R > 2:
        t[1, :] = torch.tensor(info.smallest_normal, dtype=dtype)
        t[1, ::2] = torch.tensor(info.smallest_normal, dtype=dtype) * 0.5
    return t


def check_quantized(q, x):
    data, scales = ref.quantize(host64(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.data.cpu().numpy(), data)


@pytest.mark.parametrize("R,K", [(1, 1), (3, 31), (5, 32), (7, 33), (2, 64), (130, 96), (9, 255), (4, 257),
                                 (3, 2049), (17, 4096), (1, 70000), (300, 257), (40, 2048), (71, 1000), (133, 33)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_quantize(R, K, dtype):
    x = inputs(np.random.default_rng(R * 7919 + K), R, K, TYPES[dtype])
    say(f"quantize {R}x{K} {dtype}")
    d = x.to(DEV)
    check_quantized(g.quantize_mx4(d), x)
    # padded rows, an unaligned start, columns, every second column
    buf = torch.full((R * (K + 5) + 3,), float("nan"), dtype=x.dtype, device=DEV)
    v = buf[3:].view(R, K + 5)[:, :K]
    v.copy_(d)
    check_quantized(g.quantize_mx4(v), x)
    c = d.t().contiguous().t()
    check_quantized(g.quantize_mx4(c), x)
    wide = torch.full((R, 2 * K), float("nan"), dtype=x.dtype, device=DEV)
    wide[:, ::2] = d
    check_quantized(g.quantize_mx4(wide[:, ::2]), x)


@pytest.mark.parametrize("order", ["rows", "columns", "even columns", "padded"])
def test_quantize_stack(order):
    G, R, K = 3, 5 if order != "even columns" else 6, 70
    x = torch.stack([inputs(np.random.default_rng(i), R, K, torch.bfloat16) for i in range(G)])
    d = x.to(DEV)
    if "columns" in order:
        d = d.transpose(1, 2).contiguous().transpose(1, 2)
    elif order == "padded":
        d = torch.cat((d, torch.full_like(d, float("nan"))), dim=2)[:, :, :K]
    say(f"quantize stack {order}")
    out = g.MX4(torch.full((G, R, 48), 0x77, dtype=torch.uint8, device=DEV),
                torch.full((G, R, 3), 9, dtype=torch.uint8, device=DEV), K)
    q = g.quantize_mx4(d, out=out)
    assert q is out
    for i in range(G):
        check_quantized(q[i], x[i])
    y = g.dequantize_mx4(q, torch.float32)
    assert np.array_equal(host64(y[1]), ref.values(*(t.cpu().numpy() for t in (q[1].data, q[1].scales)), K))
    # a stack whose matrices are not adjacent
    y = g.dequantize_mx4(q[:, 1:4], torch.bfloat16)
    assert torch.equal(y, g.dequantize_mx4(q, torch.bfloat16)[:, 1:4])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_quantize_non_finite_blocks(dtype):
    x = inputs(np.random.default_rng(5), 6, 100, TYPES[dtype])
    x[0, 5] = float("inf")
    x[1, 40] = float("nan")
    x[2, 99] = float("-inf")
    x[3, :] = float("nan")
    say(f"quantize non-finite {dtype}")
    for d in (x.to(DEV), x.to(DEV).t().contiguous().t()):
        q = g.quantize_mx4(d)
        check_quantized(q, x)
        y = host64(g.dequantize_mx4(q, torch.float32))
        assert np.isnan(y[0, :32]).all() and np.isfinite(y[0, 32:]).all()
        assert np.isnan(y[1, 32:64]).all() and np.isnan(y[2, 96:]).all() and np.isnan(y[3]).all()
        assert np.isfinite(y[4:]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_dequantize_every_scale_and_code(dtype):
    data = np.tile(np.arange(16, dtype=np.uint8) * 17, (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    say(f"dequantize all codes {dtype}")
    got = g.dequantize_mx4(mx4(data, scales, 32), TYPES[dtype])
    want = torch.from_numpy(ref.values(data, scales, 32)).to(TYPES[dtype])
    assert torch.equal(torch.nan_to_num(got.cpu().double(), nan=-77.0),
                       torch.nan_to_num(want.double(), nan=-77.0))


@pytest.mark.parametrize("R,K", [(1, 1), (2, 7), (3, 33), (65, 64), (5, 255), (3, 2051), (33, 512), (300, 257), (41, 2046), (71, 1003), (90, 4)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_dequantize_shapes(R, K, dtype):
    rng = np.random.default_rng(R + K)
    data, scales = ref.random_codes(rng, R, K)
    want = torch.from_numpy(ref.values(data, scales, K)).to(TYPES[dtype])
    say(f"dequantize {R}x{K} {dtype}")
    assert torch.equal(g.dequantize_mx4(mx4(data, scales, K), TYPES[dtype]).cpu(), want)
    # padded on both sides; what lies between the rows stays
    B = ref.blocks(K)
    wd = torch.full((R, 16 * B + 32), 0x55, dtype=torch.uint8, device=DEV)
    ws = torch.full((R, B + 3), 255, dtype=torch.uint8, device=DEV)
    wd[:, :16 * B], ws[:, :B] = dev(data), dev(scales)
    out = torch.full((R, K + 3), 5.0, dtype=TYPES[dtype], device=DEV)
    g.dequantize_mx4(g.MX4(wd[:, :16 * B], ws[:, :B], K), TYPES[dtype], out=out[:, :K])
    assert torch.equal(out[:, :K].cpu(), want) and (out[:, K:] == 5.0).all()


# ---- products

def check_product(c, av, bv, what):
    """c against av . bv^T (float64 [M, K], [N, K])."""
    info = torch.finfo(c.dtype)
    want = av @ bv.T
    tol = ref.product_tolerance(want, np.abs(av) @ np.abs(bv.T), av.shape[1] + 8, info.eps,
                                info.smallest_normal * info.eps)
    err = np.abs(host64(c) - want)
    over = np.abs(want) > info.max       # past the format's range: infinite
    ok = (err <= tol) | over
    assert ok.all(), f"{what}: {(~ok).sum()} of {ok.size} outputs outside the tolerance, first at " \
                     f"{np.argwhere(~ok)[0]}: {host64(c)[tuple(np.argwhere(~ok)[0])]} for " \
                     f"{want[tuple(np.argwhere(~ok)[0])]}"


def guarded(M, N, dtype):
    buf = torch.full((M + 2, N + 7), 3.0, dtype=dtype, device=DEV)
    return buf, buf[1:M + 1, 3:N + 3]


def check_guard(buf, M, N):
    b = buf.clone()
    b[1:M + 1, 3:N + 3] = 3.0
    assert (b == 3.0).all(), "write outside the output"


SHAPES = [(1, 1, 1), (1, 16, 32), (3, 17, 33), (5, 70, 128), (16, 33, 130), (17, 16, 256), (31, 100, 511),
          (33, 31, 1000), (64, 48, 96), (65, 20, 700), (200, 130, 257), (1, 300, 7168), (130, 257, 2048),
          (300, 264, 1025), (257, 513, 640),
          # enough columns (on 256 compute units) for several strips a wave, K of less and of more than a group
          (16, 6150, 161), (1, 6200, 1000), (40, 6150, 289), (33, 3100, 513), (4, 6150, 600), (4, 70, 500), (100, 6200, 257), (100, 10300, 97),
          # enough rows and columns for 256 x 256 tiles: whole steps only, a partial one only, both, edges of
          # nearly empty tiles
          (1801, 1543, 640), (1801, 1543, 33), (1543, 1801, 1025), (130, 12500, 257), (12500, 130, 96),
          (300, 6200, 2050), (1793, 1537, 128)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_product_mx4(M, N, K, dtype):
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    a, b = ref.random_codes(rng, M, K, 120, 128), ref.random_codes(rng, N, K, 116, 126)
    av, bv = ref.values(*a, K), ref.values(*b, K)
    qa, qb = mx4(*a, K), mx4(*b, K)
    say(f"gemm_mx4 {M}x{N}x{K} {dtype}")
    buf, out = guarded(M, N, TYPES[dtype])
    out.fill_(float("nan"))
    c = g.gemm_mx4(qa, qb, out=out, dtype=TYPES[dtype])
    check_product(c, av, bv, "product")
    check_guard(buf, M, N)
    assert torch.equal(g.gemm_mx4(qa, qb, dtype=TYPES[dtype]), out)       # the same bits again


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_product_a16(M, N, K, dtype):
    rng = np.random.default_rng(M * 37 + N * 5 + K)
    b = ref.random_codes(rng, N, K, 112, 126)
    bv = ref.values(*b, K)
    # rows of A inside a buffer of NaN: nothing past K or M may enter
    wide = torch.full((M + 1, K + 9), float("nan"), dtype=TYPES[dtype], device=DEV)
    wide[:M, 1:K + 1] = torch.from_numpy(rng.standard_normal((M, K))).to(TYPES[dtype]).to(DEV)
    a = wide[:M, 1:K + 1]
    say(f"gemm_mx4 a16 {M}x{N}x{K} {dtype}")
    buf, out = guarded(M, N, TYPES[dtype])
    out.fill_(float("nan"))
    c = g.gemm_mx4(a, mx4(*b, K), out=out)
    check_product(c, host64(a), bv, "product")
    check_guard(buf, M, N)
    assert torch.equal(g.gemm_mx4(a, mx4(*b, K)), out)


@pytest.mark.parametrize("M,N,K", [(1, 40, 300), (16, 33, 1000), (70, 65, 700), (300, 300, 512),
                                   (1700, 1800, 1000)])
def test_products_exact_sums(M, N, K):
    """Scales of 1: every product is a multiple of 1/4 and every sum below
    2^22, so fp32 holds it exactly and one rounding remains."""
    rng = np.random.default_rng(K)
    a, b = ref.random_codes(rng, M, K, 127, 127), ref.random_codes(rng, N, K, 127, 127)
    av, bv = ref.values(*a, K), ref.values(*b, K)
    say(f"gemm_mx4 exact {M}x{N}x{K}")
    for dtype in (torch.float16, torch.bfloat16):
        want = torch.from_numpy(av @ bv.T).to(dtype)
        assert torch.equal(g.gemm_mx4(mx4(*a, K), mx4(*b, K), dtype=dtype).cpu(), want)
        assert torch.equal(g.gemm_mx4(torch.from_numpy(av).to(dtype).to(DEV), mx4(*b, K)).cpu(), want)


@pytest.mark.parametrize("scales", [(90, 96), (60, 104), (140, 146), (0, 30), (100, 141)])
@pytest.mark.parametrize("M,N", [(1, 48), (20, 48), (50, 48), (9, 6150), (40, 6150), (33, 3100)])
def test_product_a16_far_scales(scales, M, N):
    """Weight scales outside what binary16 holds: the weights stay exact.  A
    row of one block's weights alone shows any that were rounded away."""
    rng = np.random.default_rng(scales[0])
    K = 300
    b = ref.random_codes(rng, N, K, *scales)
    x = torch.from_numpy(rng.standard_normal((M, K)) * 2.0 ** (6 if scales[0] < 100 else -14))
    say(f"gemm_mx4 far scales {scales}")
    for dtype in (torch.float16, torch.bfloat16):
        a = x.to(dtype).to(DEV)
        check_product(g.gemm_mx4(a, mx4(*b, K)), host64(a), ref.values(*b, K), f"{scales} {dtype}")


@pytest.mark.parametrize("scale", [1, 30, 60, 61, 103, 104, 140, 141, 254])
def test_infinite_activations_at_any_scale(scale):
    """An infinity times a weight that is not zero is infinite, however small
    the weight."""
    N, K = 20, 160
    codes = np.full((N, 80), 0x11, dtype=np.uint8)      # 0.5 everywhere
    codes[3] = 0x99                                     # -0.5
    b = mx4(codes, np.full((N, 5), scale, dtype=np.uint8), K)
    want = torch.full((N,), float("inf"))
    want[3] = -float("inf")
    say(f"gemm_mx4 infinities at scale {scale}")
    for M in (1, 20):
        for dtype in (torch.float16, torch.bfloat16):
            a = torch.ones((M, K), dtype=dtype, device=DEV)
            a[-1, 70] = float("inf")
            assert torch.equal(g.gemm_mx4(a, b)[-1].float().cpu(), want)


@pytest.mark.parametrize("M,N,K", [(5, 40, 300), (1600, 1800, 300)])
def test_products_nan_scale_stays_in_its_row(M, N, K):
    rng = np.random.default_rng(3)
    a, b = ref.random_codes(rng, M, K), ref.random_codes(rng, N, K)
    b[1][7, 4] = 255
    say("gemm_mx4 NaN scale")
    for c in (g.gemm_mx4(mx4(*a, K), mx4(*b, K)),
              g.gemm_mx4(torch.from_numpy(ref.values(*a, K)).to(torch.float16).to(DEV), mx4(*b, K))):
        nan = torch.isnan(c).cpu()
        assert nan[:, 7].all() and nan.sum() == M
    a[1][2, 0] = 255
    nan = torch.isnan(g.gemm_mx4(mx4(*a, K), mx4(*b, K))).cpu()
    assert nan[2].all() and nan[:, 7].all() and nan.sum() == N + M - 1


@pytest.mark.parametrize("M,N,K", [(70, 50, 200), (1600, 1800, 200)])
def test_strided_mx4_operands(M, N, K):
    rng = np.random.default_rng(11)
    a, b = ref.random_codes(rng, 2 * M, K), ref.random_codes(rng, 3 * N, K)
    qa, qb = mx4(*a, K), mx4(*b, K)
    say("gemm_mx4 strided")
    c = g.gemm_mx4(qa[::2], qb[1::3])
    check_product(c, ref.values(*a, K)[::2], ref.values(*b, K)[1::3], "strided")
    x = torch.from_numpy(rng.standard_normal((2 * M, K))).to(torch.bfloat16).to(DEV)
    check_product(g.gemm_mx4(x[::2], qb[1::3]), host64(x[::2]), ref.values(*b, K)[1::3], "strided a16")


@pytest.mark.parametrize("M", [1, 24, 300])
def test_linear_layer_run(M):
    """Weights and activations quantised, multiplied and set aside again, as a
    program would: each step against the definition on the step's own input."""
    N, K = 130, 352
    rng = np.random.default_rng(M)
    w = torch.from_numpy(rng.standard_normal((K, N)) * K ** -0.5).to(torch.bfloat16).to(DEV)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16).to(DEV)
    say(f"linear run {M}")
    qw = g.quantize_mx4(w.t())                       # [N, K] from a [K, N] weight
    qx = g.quantize_mx4(x)
    y = g.gemm_mx4(qx, qw, dtype=torch.bfloat16)
    back = g.dequantize_mx4(g.quantize_mx4(y), torch.bfloat16)
    wq, xq = ref.quantize(host64(w).T), ref.quantize(host64(x))
    check_product(y, ref.values(*xq, K), ref.values(*wq, K), "linear")
    assert torch.equal(back.cpu(), torch.from_numpy(ref.values(*ref.quantize(host64(y)), N)).to(torch.bfloat16))
    y16 = g.gemm_mx4(x, qw)
    check_product(y16, host64(x), ref.values(*wq, K), "linear a16")


@pytest.mark.parametrize("M,N", [(3, 136), (300, 136), (1700, 1600)])
def test_graph_replays_and_other_stream(M, N):
    K = 352
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.float16).to(DEV)
    qw = mx4(*ref.random_codes(rng, N, K, 118, 124), K)

    def step():
        q = g.quantize_mx4(x)
        return g.gemm_mx4(q, qw), g.gemm_mx4(x, qw), g.dequantize_mx4(q, torch.float16)

    say(f"mx4 graph {M}")
    side = torch.cuda.Stream(DEV)
    eager = [t.clone() for t in step()]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    q = g.quantize_mx4(x, stream=side)               # a stream by argument
    side.synchronize()
    assert torch.equal(g.dequantize_mx4(q, torch.float16), eager[2])
    # results of a stream by argument may take no memory that work of the current stream still uses
    for _ in range(3):
        held = torch.full((1 << 22,), 7.0, device=DEV)
        busy = [held * i for i in range(20)]
        del held, busy
        side.wait_stream(torch.cuda.current_stream())
        y = g.gemm_mx4(g.quantize_mx4(x, stream=side), qw, stream=side)
        z = g.gemm_mx4(x, qw, stream=side)
        side.synchronize()
        assert torch.equal(y, eager[0]) and torch.equal(z, eager[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        x.mul_(0.5).add_(0.25)                       # other inputs, the same buffers
        want = [t.clone() for t in step()]
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


def test_workspace():
    M, N, K = 1700, 1800, 200
    rng = np.random.default_rng(12)
    a, b = mx4(*ref.random_codes(rng, M, K), K), mx4(*ref.random_codes(rng, N, K), K)
    need = g.gemm_mx4_workspace_bytes(M, N, K)
    assert need > 0 and g.gemm_mx4_workspace_bytes(64, 64, K) == 0
    buf = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
    say("mx4 workspace")
    c = g.gemm_mx4(a, b, workspace=buf[:need])
    assert (buf[need:] == 255).all() and torch.equal(c, g.gemm_mx4(a, b))
    for bad in (buf[:need - 1], buf[8:need + 8]):
        with pytest.raises(g.GemmError):
            g.gemm_mx4(a, b, workspace=bad)
    with pytest.raises(g.GemmError):                 # over the output
        g.gemm_mx4(a, b, out=c, workspace=c.view(torch.uint8))
    # two products at once, each with a workspace of its own
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(g.gemm_mx4(a, b))
    torch.cuda.synchronize()
    assert all(torch.equal(o, c) for o in outs)


def test_offsets_past_32_bits():
    """Elements, codes and outputs beyond 2^32 from the base."""
    R, K = 66000, 66560                              # 4.4e9 elements, 8.8 GB in bfloat16
    rng = np.random.default_rng(1)
    say("mx4 past 32 bits")
    x = torch.full((R, K), 0.5, dtype=torch.bfloat16, device=DEV)
    tail = inputs(rng, 3, K, torch.bfloat16)
    x[-3:] = tail.to(DEV)
    q = g.quantize_mx4(x)
    check_quantized(q[R - 3:], tail)
    y = g.dequantize_mx4(q, torch.bfloat16)
    want = torch.from_numpy(ref.values(*ref.quantize(host64(tail)), K)).to(torch.bfloat16)
    assert torch.equal(y[-3:].cpu(), want) and (y[R - 4] == 0.5).all()
    del x, y
    N = 65600                                        # C of 4.3e9 elements
    a, b = ref.random_codes(rng, R, 64, 120, 126), ref.random_codes(rng, N, 64, 120, 126)
    c = g.gemm_mx4(mx4(*a, 64), mx4(*b, 64), dtype=torch.bfloat16)
    check_product(c[-2:, -300:], ref.values(a[0][-2:], a[1][-2:], 64), ref.values(b[0][-300:], b[1][-300:], 64),
                  "last rows")


def test_more_rows_than_one_grid_axis_takes():
    """2^26 rows of 257: more waves than a launch has along x.  The rows of x
    overlap (row stride 1), so few bytes describe them."""
    R, K = (1 << 26) + 100, 257
    rng = np.random.default_rng(6)
    line = torch.from_numpy(rng.standard_normal(R + K - 1).astype(np.float32)).to(torch.bfloat16)
    x = line.to(DEV).as_strided((R, K), (1, 1))
    say("mx4 many rows")
    q = g.quantize_mx4(x)
    y = g.dequantize_mx4(q, torch.bfloat16)
    for r in (0, (1 << 24) - 2, R // 2, R - 4):
        host = line.as_strided((R, K), (1, 1))[r:r + 4].contiguous()
        check_quantized(q[r:r + 4], host)
        assert torch.equal(y[r:r + 4].cpu(), torch.from_numpy(ref.values(*ref.quantize(host64(host)), K)).to(torch.bfloat16))


def test_single_rows_of_far_strided_operands():
    """A single row has no next one: its row stride does not matter."""
    K, N = 96, 20
    rng = np.random.default_rng(2)
    a, b = ref.random_codes(rng, 1, K, 120, 126), ref.random_codes(rng, N, K, 120, 126)
    qa, qb = mx4(*a, K), mx4(*b, K)
    far = g.MX4(qa.data.as_strided((1, 48), (1 << 30, 1)), qa.scales.as_strided((1, 3), (1 << 30, 1)), K)
    say("mx4 single rows")
    assert torch.equal(g.gemm_mx4(far, qb), g.gemm_mx4(qa, qb))
    assert torch.equal(g.gemm_mx4(qb, far), g.gemm_mx4(qb, qa))
    x = torch.from_numpy(rng.standard_normal((1, K))).to(torch.float16).to(DEV)
    assert torch.equal(g.gemm_mx4(x.as_strided((1, K), (1 << 30, 1)), qb), g.gemm_mx4(x, qb))


def test_stack_of_single_rows_with_any_row_stride():
    """[G, 1, K]: the stride of an axis of one is free."""
    G, K = 5, 100
    data, scales = ref.random_codes(np.random.default_rng(4), G, K)
    d, s = dev(data).view(1, G, 64).transpose(0, 1), dev(scales).view(1, G, 4).transpose(0, 1)
    assert d.is_contiguous() and d.stride(1) == G * 64
    q = g.MX4(d, s, K)
    say("mx4 stack of single rows")
    out = torch.full((1, G, K), 3.0, device=DEV).transpose(0, 1)
    y = g.dequantize_mx4(q, torch.float32, out=out)
    assert np.array_equal(host64(y)[:, 0], ref.values(data, scales, K))


def test_gpu_refusals():
    x = torch.zeros(4, 64, dtype=torch.float16, device=DEV)
    q = g.quantize_mx4(x)
    with pytest.raises(ValueError):
        g.quantize_mx4(x[:0])
    with pytest.raises(ValueError):
        g.quantize_mx4(x[:1].expand(4, 64))
    with pytest.raises(ValueError):
        g.quantize_mx4(x, out=g.quantize_mx4(x[:3]))
    with pytest.raises(ValueError):
        g.gemm_mx4(x[:, :32], q)
    with pytest.raises(ValueError):
        g.gemm_mx4(x.t(), g.quantize_mx4(x.t()).__getitem__(slice(0, 4)))
    with pytest.raises(TypeError):
        g.gemm_mx4(x.float(), q)
    with pytest.raises(TypeError):
        g.gemm_mx4(x, q, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        g.gemm_mx4(x, q, out=torch.empty(4, 5, dtype=torch.float16, device=DEV))
    with pytest.raises(g.GemmError):                 # C over A
        g.gemm_mx4(x, q, out=x[:, :4])
    with pytest.raises(ValueError):
        g.gemm_mx4(x, g.MX4(q.data.cpu(), q.scales.cpu(), 64))
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(8, dtype=torch.uint8, device=DEV).expand(1 << 16, 8),
               torch.empty(1 << 21, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            g.gemm_mx4(q, q, workspace=ws)
