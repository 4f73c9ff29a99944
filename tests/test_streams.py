"""A stream by argument: what the call reads there stays what it was until the
stream has read it, although the caller drops its last reference right after
the call, and what it writes is not handed out before it is written.  A stream
of another device is refused."""
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

CYCLES = 20_000_000      # the side stream is busy for ten milliseconds at least


def dropped(side, make, call):
    """call(*make(), stream=side) behind other work of `side`, the inputs
    dropped at once and their memory asked for again on the current stream."""
    want = call(*make(), stream=None)
    torch.cuda.synchronize()
    inputs = make()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    sizes = [t.numel() * t.element_size() for t in inputs]
    got = call(*inputs, stream=side)
    del inputs
    again = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    del again
    return want, got


def randn(*shape, dtype=torch.float16, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device=DEV) * shape[-1] ** -0.5).to(dtype)


def mx4(*shape, seed=1):
    return g.quantize_mx4(randn(*shape, seed=seed))


def as_mx4(data, scales, K):
    return g.MX4(data, scales, K)


K = 4096
CALLS = {
    "quantize": (lambda: (randn(600, K),), lambda x, stream: g.quantize_mx4(x, stream=stream).data),
    "dequantize": (lambda: tuple(t.clone() for t in (lambda q: (q.data, q.scales))(mx4(600, K))),
                   lambda d, s, stream: g.dequantize_mx4(as_mx4(d, s, K), torch.float16, stream=stream)),
    "product": (lambda: tuple(t.clone() for q in (mx4(600, K), mx4(512, K, seed=2)) for t in (q.data, q.scales)),
                lambda d, s, e, t, stream: g.gemm_mx4(as_mx4(d, s, K), as_mx4(e, t, K), stream=stream)),
    "product a16": (lambda: (randn(16, K),) + tuple(t.clone() for t in (lambda q: (q.data, q.scales))(mx4(512, K))),
                    lambda x, d, s, stream: g.gemm_mx4(x, as_mx4(d, s, K), stream=stream)),
    "experts": (lambda: (randn(8, 512), randn(8, 4, dtype=torch.float32), randn(4, 512, 512), randn(4, 512, 256)),
                lambda x, l, u, d, stream: g.gemm_moe(x, l, u, d, 2, stream=stream)),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_inputs_of_a_stream_by_argument(name):
    make, call = CALLS[name]
    say(f"stream inputs {name}")
    want, got = dropped(torch.cuda.Stream(DEV), make, call)
    assert torch.equal(got, want)


def test_outputs_and_workspaces_of_a_stream_by_argument():
    """An out that the caller drops while it is written has no reader, but its
    memory must not be handed out before the write; the same of a workspace."""
    side = torch.cuda.Stream(DEV)
    M, N = 1700, 1800
    a, b = mx4(M, 256), mx4(N, 256, seed=3)
    say("stream outputs")
    for give in ("out", "workspace"):
        out = torch.empty(M, N, dtype=torch.float16, device=DEV)
        ws = torch.empty(g.gemm_mx4_workspace_bytes(M, N, 256), dtype=torch.uint8, device=DEV)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(CYCLES)
        given = {give: out if give == "out" else ws}
        n = given[give].numel() * given[give].element_size()
        y = g.gemm_mx4(a, b, stream=side, **given)
        del out, ws, given
        if give == "out":
            del y
        again = [torch.full((n,), 9, dtype=torch.uint8, device=DEV) for _ in range(2)]
        torch.cuda.synchronize()
        assert all((t == 9).all() for t in again), give
        if give == "workspace":
            assert torch.equal(y, g.gemm_mx4(a, b))


class Elsewhere:
    """The handle of the default stream, said to be another device's."""
    device = torch.device("cuda:1")
    cuda_stream = 0


def test_stream_of_another_device():
    x = randn(8, 64)
    q = g.quantize_mx4(x)
    say("stream of another device")
    for call in (lambda s: g.quantize_mx4(x, stream=s), lambda s: g.dequantize_mx4(q, stream=s),
                 lambda s: g.gemm_mx4(q, q, stream=s), lambda s: g.gemm_mx4(x, q, stream=s),
                 lambda s: g.gemm_moe(x, randn(8, 2), randn(2, 32, 64), randn(2, 64, 16), 1, stream=s)):
        with pytest.raises(ValueError):
            call(Elsewhere())


# ---- the 16-bit and FP8 products, by the same rules

def offsets(*rows):
    return torch.tensor(rows, dtype=torch.int64, device=DEV)


SMALL, BIG = 512, 16384     # BIG: plans that pack B into a workspace of the library
OLDER = {
    "gemm": (lambda: (randn(600, K), randn(K, SMALL)), lambda a, b, stream: g.gemm(a, b, stream=stream)),
    "gemm f8": (lambda: (randn(64, K).to(torch.float8_e4m3fn), randn(SMALL, K).to(torch.float8_e4m3fn)),
                lambda a, b, stream: g.gemm(a, b.t(), stream=stream)),
    "gemm packing": (lambda: (randn(BIG, 256), randn(SMALL, 256)), lambda a, b, stream: g.gemm(a, b.t(), stream=stream)),
    "noalloc": (lambda: (randn(600, K), randn(K, SMALL)),
                lambda a, b, stream: g.gemm_noalloc(a, b, noalloc_out(stream), stream=stream)),
    "grouped": (lambda: (randn(600, K), randn(3, K, SMALL), offsets(0, 100, 400, 600)),
                lambda a, b, o, stream: g.gemm_grouped(a, b, o, stream=stream)),
    "pack": (lambda: (randn(K, SMALL),), lambda b, stream: g.pack_b(b, stream=stream).data),
    "packed": (lambda: (randn(300, K), g.pack_b(randn(K, SMALL)).data),
               lambda a, d, stream: g.gemm_packed(a, g.PackedB(d, K, SMALL), stream=stream)),
}


def noalloc_out(stream):
    with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
        return torch.empty(600, SMALL, dtype=torch.float16, device=DEV)


@pytest.mark.parametrize("name", list(OLDER))
def test_inputs_of_older_calls(name):
    make, call = OLDER[name]
    say(f"stream inputs {name}")
    want, got = dropped(torch.cuda.Stream(DEV), make, call)
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("name", [n for n in OLDER if n != "noalloc"])
def test_results_of_older_calls_take_no_memory_in_use(name):
    """The result is written by the side stream while the current one is still
    busy with what was freed there."""
    make, call = OLDER[name]
    side = torch.cuda.Stream(DEV)
    inputs = make()
    want = call(*inputs, stream=None)
    say(f"stream results {name}")
    torch.cuda.synchronize()
    held = torch.empty(want.numel() * want.element_size(), dtype=torch.uint8, device=DEV)
    torch.cuda._sleep(CYCLES)
    held.fill_(9)                        # after the sleep; the memory is free for the next caller at once
    del held
    got = call(*inputs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


def test_older_calls_on_a_stream_of_another_device():
    a, b = randn(64, 64), randn(64, 64)
    p = g.pack_b(b)
    say("older calls, stream of another device")
    for call in (lambda s: g.gemm(a, b, stream=s), lambda s: g.gemm_noalloc(a, b, torch.empty_like(a), stream=s),
                 lambda s: g.gemm_grouped(a, b[None], offsets(0, 64), stream=s), lambda s: g.pack_b(b, stream=s),
                 lambda s: g.gemm_packed(a, p, stream=s)):
        with pytest.raises(ValueError):
            call(Elsewhere())
