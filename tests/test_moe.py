"""The mixture-of-experts layer on the GPU against its definition in 64 bits
(moe_ref), with 16-bit and MX4 expert weights."""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
import moe_ref
import mx4_ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def host64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Layer:
    """Inputs of a layer on the GPU, and as float64 arrays."""

    def __init__(self, T, E, k, H, I, dtype, weights, logits="f32", seed=0, pad=0):
        rng = np.random.default_rng(seed + 1000 * T + E + H)
        self.k, self.dtype = k, TYPES[dtype]
        x = torch.full((T, H + pad), float("nan"), dtype=self.dtype, device=DEV)
        x[:, :H] = torch.from_numpy(rng.standard_normal((T, H))).to(self.dtype).to(DEV)
        self.x = x[:, :H]
        lg = torch.full((T, E + pad), float("nan"), dtype=TYPES[logits], device=DEV)
        lg[:, :E] = torch.from_numpy(rng.standard_normal((T, E)) * 2).to(TYPES[logits]).to(DEV)
        self.logits = lg[:, :E]
        if weights == "16":
            def make(n, kk):
                w = torch.full((E, n, kk + pad), float("nan"), dtype=self.dtype, device=DEV)
                w[:, :, :kk] = torch.from_numpy(rng.standard_normal((E, n, kk)) * kk ** -0.5).to(self.dtype).to(DEV)
                return w[:, :, :kk], host64(w[:, :, :kk])
        else:
            def make(n, kk):
                d, s = mx4_ref.random_codes(rng, E * n, kk, 118, 123)
                v = mx4_ref.values(d, s, kk).reshape(E, n, kk)
                q = g.MX4(torch.from_numpy(d).to(DEV).view(E, n, -1), torch.from_numpy(s).to(DEV).view(E, n, -1), kk)
                return q, v
        self.up, self.up64 = make(2 * I, H)
        self.down, self.down64 = make(H, I)

    def run(self, renormalize=True, **kw):
        return g.gemm_moe(self.x, self.logits, self.up, self.down, self.k, renormalize=renormalize, **kw)

    def check(self, y, renormalize=True, rows=None):
        info = torch.finfo(self.dtype)
        rows = range(self.x.shape[0]) if rows is None else rows
        want, tol = moe_ref.layer(host64(self.x)[list(rows)], host64(self.logits)[list(rows)], self.up64,
                                  self.down64, self.k, renormalize, info.eps, info.smallest_normal * info.eps)
        err = np.abs(host64(y)[list(rows)] - want)
        bad = ~(err <= tol)
        assert not bad.any(), f"{bad.sum()} of {bad.size} outside the tolerance, first at {np.argwhere(bad)[0]}: " \
                              f"error {err[bad][0]}, tolerance {tol[bad][0]}"


CASES = [  # T, E, k, H, I: by pair (T k < E) and by expert, one expert, all experts, odd sizes, many tokens
    (1, 8, 2, 64, 32), (1, 1, 1, 32, 16), (1, 100, 8, 200, 48), (3, 17, 3, 70, 33), (5, 64, 4, 129, 65),
    (2, 4, 4, 96, 40), (16, 8, 2, 256, 64), (17, 5, 1, 100, 50), (33, 2, 2, 64, 130), (64, 3, 2, 72, 24),
    (64, 1, 1, 130, 31), (40, 70, 6, 33, 17), (64, 16, 16, 48, 40), (7, 512, 5, 40, 24), (1, 3, 2, 1, 1),
    (4, 6, 2, 1030, 520),
    # enough columns of Y (on 256 compute units) for two strips a wave
    (3, 4, 2, 6150, 24), (40, 5, 2, 6150, 40), (64, 3, 2, 6200, 70),
    # long sequences of experts per column: split over 2, 4 and 8 workgroups
    (9, 64, 8, 4090, 210), (48, 64, 8, 2000, 300), (16, 64, 4, 1000, 333), (64, 64, 8, 36, 200), (30, 40, 6, 3000, 257),
    # enough strips of I for four, two and one part of H
    (12, 24, 4, 70, 272), (40, 24, 4, 70, 530), (40, 24, 4, 300, 1040), (12, 24, 4, 70, 1040), (12, 24, 4, 70, 2060)]


@pytest.mark.parametrize("T,E,k,H,I", CASES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("weights", ["16", "mx4"])
def test_layer(T, E, k, H, I, dtype, weights):
    la = Layer(T, E, k, H, I, dtype, weights, pad=3 if E % 2 else 0)
    say(f"moe T={T} E={E} k={k} H={H} I={I} {dtype} {weights}")
    y = la.run()
    la.check(y)
    buf = torch.full((T + 2, H + 5), 7.0, dtype=la.dtype, device=DEV)
    ws = torch.full((g.gemm_moe_workspace_bytes(T, E, k, H, I),), 255, dtype=torch.uint8, device=DEV)
    out = la.run(renormalize=False, out=buf[1:T + 1, 2:H + 2], workspace=ws)
    la.check(out, renormalize=False)
    buf[1:T + 1, 2:H + 2] = 7.0
    assert (buf == 7.0).all(), "write outside the output"
    assert torch.equal(la.run(), y)                    # the same bits again


@pytest.mark.parametrize("T,E,k,H,I", [(3, 4, 2, 6150, 1000), (16, 8, 4, 6150, 500), (20, 8, 2, 6150, 500),
                                       (20, 32, 4, 2000, 400), (2, 4, 2, 5000, 1200)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_layer_with_weights_past_the_cache(T, E, k, H, I, dtype):
    la = Layer(T, E, k, H, I, dtype, "16")
    say(f"moe T={T} E={E} k={k} H={H} I={I} {dtype}")
    y = la.run()
    la.check(y)
    assert torch.equal(la.run(), y)


@pytest.mark.parametrize("logits", ["f16", "bf16"])
@pytest.mark.parametrize("T,E", [(2, 40), (30, 12)])
def test_ties_and_logit_types(logits, T, E):
    la = Layer(T, E, 3, 64, 32, "bf16", "16", logits=logits)
    la.logits.copy_(torch.round(la.logits))            # many equal logits
    la.logits[0] = 0.0                                 # all equal
    la.logits[0, 1::2] = -0.0
    say(f"moe ties {logits} {T} {E}")
    la.check(la.run())


@pytest.mark.parametrize("weights", ["16", "mx4"])
@pytest.mark.parametrize("T,E,k", [(6, 40, 3), (20, 8, 3)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_experts(T, E, k, weights, renormalize):
    """-inf removes an expert; a token without experts gets zeros; the type's
    lowest value is an ordinary logit."""
    la = Layer(T, E, k, 72, 40, "bf16", weights)
    la.logits[0] = float("-inf")
    la.logits[1] = float("-inf")
    la.logits[1, 5] = 1.5
    la.logits[2, 2:] = float("-inf")
    la.logits[3] = torch.finfo(torch.float32).min
    la.logits[4, ::2] = float("-inf")
    say(f"moe masked {T} {E} {weights}")
    y = la.run(renormalize)
    assert (y[0] == 0).all()
    la.check(y, renormalize)
    la.logits[:] = float("-inf")                       # an empty batch
    assert (la.run(renormalize) == 0).all()


@pytest.mark.parametrize("T,E", [(4, 40), (20, 8)])
def test_non_finite_rows_stay_apart(T, E):
    la = Layer(T, E, 2, 64, 32, "f16", "16")
    good = [t for t in range(T) if t not in (0, 1, 2)]
    la.x[0, 3] = float("nan")
    la.logits[1, 2] = float("nan")
    la.logits[2, 1] = float("inf")
    say(f"moe non-finite {T} {E}")
    y = la.run()
    assert torch.isnan(y[:3]).all()
    la.check(y, rows=good)


def test_unused_experts_are_not_read_into_sums():
    la = Layer(3, 12, 2, 64, 32, "bf16", "16")
    la.logits[:, 4:] = -50.0
    la.up[4:] = float("nan")
    la.down[4:] = float("nan")
    la.up64[4:], la.down64[4:] = 0, 0
    say("moe unused experts")
    la.check(la.run())


@pytest.mark.parametrize("weights", ["16", "mx4"])
@pytest.mark.parametrize("T", [5, 8, 9, 13, 16, 48])
@pytest.mark.parametrize("H", [100, 6150])
def test_an_expert_of_all_tokens(T, H, weights):
    """Few tokens per expert on the average, one expert with all of them."""
    E = max(16, T)
    la = Layer(T, E, 2, H, 300, "bf16", weights)
    la.logits[:, 3] = 30.0
    la.logits[:, 3] += torch.arange(T, device=DEV)
    la.logits[: T // 2, 7] = 31.0
    say(f"moe one expert of all {T} {H} {weights}")
    y = la.run()
    la.check(y)
    assert torch.equal(la.run(), y)


def test_expert_views():
    """Every second expert of a larger stack, rows with a stride of their own."""
    la = Layer(4, 10, 2, 64, 48, "bf16", "16")
    up = torch.full((10, 96, 100), float("nan"), dtype=torch.bfloat16, device=DEV)
    up[:, :, 5:69] = la.up
    y = g.gemm_moe(la.x, la.logits[:, :5], up[::2, :, 5:69], la.down[::2], 2)
    la.logits, la.up64, la.down64 = la.logits[:, :5], la.up64[::2], la.down64[::2]
    say("moe expert views")
    la.check(y)
    lq = Layer(4, 10, 2, 64, 48, "bf16", "mx4")
    y = g.gemm_moe(lq.x, lq.logits[:, :5], lq.up[::2], lq.down[1::2], 2)
    lq.logits, lq.up64, lq.down64 = lq.logits[:, :5], lq.up64[::2], lq.down64[1::2]
    lq.check(y)


def test_far_scales_of_expert_weights():
    """binary16 activations with MX4 scales that binary16 does not hold."""
    la = Layer(3, 4, 2, 100, 64, "f16", "mx4")
    for q, v in ((la.up, la.up64), (la.down, la.down64)):
        shift = 30 if q is la.up else -30
        q.scales[:] = (q.scales.int() - shift).to(torch.uint8)
        v *= 2.0 ** -shift
    la.x *= 64.0
    say("moe far scales")
    la.check(la.run())


def test_router_product_into_layer():
    """As a decode step uses them: the router's logits by the library's own
    product, experts quantised by the library, the layer, twice over."""
    T, E, k, H, I = 9, 12, 3, 128, 96
    rng = np.random.default_rng(9)
    def rand(*shape):
        return torch.from_numpy(rng.standard_normal(shape) * shape[-1] ** -0.5).to(torch.bfloat16).to(DEV)
    x, router = rand(T, H) * H ** 0.5, rand(E, H) * 3
    up, down = rand(E, 2 * I, H), rand(E, H, I)
    qu, qd = g.quantize_mx4(up), g.quantize_mx4(down)
    say("moe after router")
    for _ in range(2):
        logits = g.gemm(x, router.t())
        for wu, wd, u64, d64 in ((up, down, host64(up), host64(down)),
                                 (qu, qd, host64(g.dequantize_mx4(qu, torch.float32)),
                                  host64(g.dequantize_mx4(qd, torch.float32)))):
            y = g.gemm_moe(x, logits, wu, wd, k)
            want, tol = moe_ref.layer(host64(x), host64(logits), u64, d64, k, True,
                                      torch.finfo(torch.bfloat16).eps, 0.0)
            assert (np.abs(host64(y) - want) <= tol).all()
        x = (x + y).contiguous()


@pytest.mark.parametrize("T,E,H,I", [(2, 40, 136, 72), (20, 8, 136, 72), (32, 64, 520, 333)])
@pytest.mark.parametrize("weights", ["16", "mx4"])
def test_graph_replays_and_other_stream(T, E, H, I, weights):
    la = Layer(T, E, 2, H, I, "bf16", weights)
    say(f"moe graph {T} {E} {H} {I} {weights}")
    eager = la.run()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = la.run()
    third = la.run(stream=side)
    side.synchronize()
    assert torch.equal(other, eager) and torch.equal(third, eager)
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = la.run()
    with torch.cuda.graph(second):
        z = la.run(renormalize=False)
    for _ in range(3):
        la.x.mul_(0.75).add_(0.1)
        la.logits.copy_(la.logits.flip(0) * 0.9)       # other routes through the same graph
        want, other = la.run(), la.run(renormalize=False)
        y.fill_(float("nan"))
        z.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, other)


def test_gpu_refusals():
    la = Layer(4, 6, 2, 64, 32, "f16", "16")
    with pytest.raises(ValueError):
        g.gemm_moe(la.x, la.logits, la.up, la.down, 7)
    with pytest.raises(ValueError):
        g.gemm_moe(la.x, la.logits, la.up, la.down, 0)
    with pytest.raises(ValueError):
        g.gemm_moe(la.x, la.logits[:, :5], la.up, la.down, 2)
    with pytest.raises(ValueError):
        g.gemm_moe(la.x, la.logits, la.up.transpose(1, 2).contiguous().transpose(1, 2), la.down, 2)
    with pytest.raises(ValueError):
        g.gemm_moe(la.x[:0], la.logits[:0], la.up, la.down, 2)
    big = torch.zeros(65, 64, dtype=torch.float16, device=DEV)
    with pytest.raises(ValueError):
        g.gemm_moe(big, torch.zeros(65, 6, device=DEV), la.up, la.down, 2)
    with pytest.raises(g.GemmError):
        la.run(out=la.x)
    with pytest.raises(g.GemmError):
        la.run(workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(8, dtype=torch.uint8, device=DEV).expand(1 << 16, 8),
               torch.empty(1 << 21, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            la.run(workspace=ws)
