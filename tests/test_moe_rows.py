"""Tokens sorted by expert and back, with the gradients, against plain loops and
64-bit sums; and a whole mixture-of-experts layer through gemm_grouped."""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
from f8_ref import assert_near, f64, half_step
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def randn(*shape, dtype=BF16, seed=0, scale=1.0):
    gen = torch.Generator(device="cpu")
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(DEV)


def ids_of(T, k, E, seed, spare=1):
    """Experts with some numbers outside 0 .. E - 1 and repeated ones."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(-spare, E + spare, (T, k))
    if T > 3:
        ids[-1] = -1
        ids[1] = ids[1, 0]
    return torch.from_numpy(ids).to(DEV)


def sorted_pairs(ids, E):
    flat = ids.cpu().numpy().reshape(-1)
    chosen = [np.flatnonzero(flat == e) for e in range(E)]
    rows = np.concatenate(chosen) if chosen else np.zeros(0, np.int64)
    offsets = np.concatenate(([0], np.cumsum([len(c) for c in chosen])))
    slots = np.full(flat.size, -1)
    slots[rows] = np.arange(rows.size)
    return offsets, np.concatenate((rows, np.full(flat.size - rows.size, -1))), slots.reshape(ids.shape)


def check_order(order, ids, E):
    for got, want in zip(order, sorted_pairs(ids, E)):
        assert got.dtype == torch.int64 and np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (5, 2, 3), (64, 8, 64), (63, 1, 2), (512, 1, 7), (1000, 3, 1024),
                                   (1024, 8, 64), (1025, 8, 33), (5000, 6, 512), (20011, 7, 200), (70000, 2, 1)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, k, E, dtype):
    say(f"sort {T} {k} {E} {dtype}")
    ids = ids_of(T, k, E, T + E).to(dtype)
    check_order(g.moe_sort(ids, E), ids, E)


@pytest.mark.parametrize("T,k,E", [(40, 4, 8), (9000, 4, 16)])
def test_sort_of_one_expert_of_none_and_of_views(T, k, E):
    say(f"sort special {T}")
    for fill in (0, E - 1, -1, E, 2 ** 40):
        ids = torch.full((T, k), fill, dtype=torch.int64, device=DEV)
        check_order(g.moe_sort(ids, E), ids, E)
    ids = ids_of(T, k + 3, E, 1)[:, 2:2 + k]
    ws = torch.empty(max(1, g.moe_sort_workspace_bytes(T, k, E)), dtype=torch.uint8, device=DEV)
    check_order(g.moe_sort(ids, E, workspace=ws), ids, E)


ROWS = [(1, 1, 1, 1), (3, 2, 4, 7), (6, 9, 5, 130), (40, 8, 16, 1000), (33, 17, 8, 2050), (700, 4, 64, 264), (2, 3, 4, 20000)]


@pytest.mark.parametrize("T,k,E,H", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32, torch.float8_e4m3fn])
def test_gather(T, k, E, H, dtype):
    say(f"gather {T} {k} {E} {H} {dtype}")
    ids = ids_of(T, k, E, 3)
    order = g.moe_sort(ids, E)
    x = randn(T, H + 3, dtype=F32, seed=4).to(dtype)[:, 1:1 + H]
    rows = order.rows.cpu()
    want = torch.where(rows[:, None] < 0, torch.zeros(1), x.float().cpu()[rows.clamp(min=0) // k])
    assert torch.equal(g.moe_gather(x, order).float().cpu(), want)
    buf = torch.full((T * k, H + 5), 3.0, dtype=F32, device=DEV).to(dtype)
    got = g.moe_gather(x, order, out=buf[:, 2:2 + H])
    assert torch.equal(got.float().cpu(), want)
    assert (buf[:, :2].float() == 3).all() and (buf[:, 2 + H:].float() == 3).all()


def back(y, order, w):
    """(sum, its tolerance before the output's rounding), float64."""
    slots = order.slots.cpu().numpy()
    v = f64(y)[np.maximum(slots, 0)] * (slots >= 0)[:, :, None]
    t = v * f64(w)[:, :, None] if w is not None else v
    return t.sum(axis=1), (slots.shape[1] + 1) * 2.0 ** -24 * np.abs(t).sum(axis=1)


@pytest.mark.parametrize("T,k,E,H", ROWS)
@pytest.mark.parametrize("dtype,wt", [(BF16, F32), (F16, F16), (F32, F32), (BF16, None), (BF16, BF16)])
def test_combine(T, k, E, H, dtype, wt):
    say(f"combine {T} {k} {E} {H} {dtype} {wt}")
    order = g.moe_sort(ids_of(T, k, E, 5), E)
    y = randn(T * k, H + 2, dtype=dtype, seed=6)[:, 1:1 + H]
    w = None if wt is None else randn(T, k + 1, dtype=wt, seed=7)[:, :k]
    want, tol = back(y, order, w)
    buf = torch.full((T, H + 4), 3.0, dtype=dtype, device=DEV)
    got = g.moe_combine(y, order, w, out=buf[:, 2:2 + H])
    assert_near(got, want, tol + half_step(np.abs(want) + tol, dtype))
    assert torch.equal(got, g.moe_combine(y, order, w))
    assert (buf[:, :2] == 3).all() and (buf[:, 2 + H:] == 3).all()


@pytest.mark.parametrize("T,k,E,H", ROWS)
@pytest.mark.parametrize("dtype,wt", [(BF16, F32), (F16, F16), (F32, F32)])
def test_combine_backward(T, k, E, H, dtype, wt):
    say(f"combine backward {T} {k} {E} {H} {dtype} {wt}")
    order = g.moe_sort(ids_of(T, k, E, 8), E)
    y, w, d = randn(T * k, H, dtype=dtype, seed=9), randn(T, k, dtype=wt, seed=10), randn(T, H, dtype=dtype, seed=11)
    dy, dw = g.moe_combine_backward(d, y, order, w)
    assert dy.dtype == dtype and dw.dtype == wt and dw.shape == (T, k)
    rows, slots = order.rows.cpu().numpy(), order.slots.cpu().numpy()
    at = np.maximum(rows, 0)
    want = np.where(rows[:, None] < 0, 0.0, f64(d)[at // k] * f64(w).reshape(-1)[at][:, None])
    assert_near(dy, want, 2.0 ** -24 * np.abs(want) + half_step(np.abs(want), dtype), "dy")
    v = f64(y)[np.maximum(slots, 0)] * (slots >= 0)[:, :, None]
    dot, mag = (v * f64(d)[:, None]).sum(axis=2), np.abs(v * f64(d)[:, None]).sum(axis=2)
    tol = (H + 16) * 2.0 ** -24 * mag
    assert_near(dw, dot, tol + half_step(np.abs(dot) + tol, wt), "dw")
    # the gradient of gather is combine with ones; both against differences: the
    # calls are linear in each of their inputs
    u = randn(T, H, dtype=F32, seed=12)
    lhs = (f64(g.moe_gather(u, order)) * f64(dy)).sum()
    rhs = (f64(u) * f64(g.moe_combine(dy.float(), order))).sum()
    assert abs(lhs - rhs) <= 1e-5 * np.abs(f64(g.moe_gather(u, order)) * f64(dy)).sum()
    p = randn(T, k, dtype=F32, seed=13)
    slope = (f64(g.moe_combine(y.float(), order, p)) * f64(d)).sum()
    assert abs(slope - (f64(p) * dot).sum()) <= 1e-5 * (np.abs(f64(p)) * mag).sum()


def test_infinite_weights_of_absent_rows_count_nothing():
    say("absent rows")
    ids = torch.tensor([[0, -1], [-1, -1]], device=DEV)
    order = g.moe_sort(ids, 2)
    y, w = randn(4, 64, seed=1), torch.tensor([[1.0, float("inf")], [float("nan"), 1.0]], device=DEV)
    y[3] = float("nan")
    out = g.moe_combine(y, order, w)
    assert torch.equal(out[0], y[0]) and (out[1] == 0).all()
    dy, dw = g.moe_combine_backward(out, y, order, w)
    assert torch.isfinite(dy).all() and (dw[1] == 0).all() and dw[0, 1] == 0 and (dy[1:] == 0).all()


def test_slots_outside_the_rows_are_not_followed():
    """An order made by hand: what points past the rows counts as absent."""
    say("bad slots")
    slots = torch.tensor([[0, 4], [-5, 1 << 40]], device=DEV)
    order = g.MoeOrder(torch.tensor([0, 1, 2], device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV), slots)
    x, y = randn(2, 40, seed=1), randn(4, 40, seed=2)
    xs = g.moe_gather(x, order)
    assert torch.equal(xs[0], x[0]) and (xs[2:] == 0).all()
    w = torch.ones(2, 2, device=DEV)
    out = g.moe_combine(y, order, w)
    assert torch.equal(out[0], y[0]) and (out[1] == 0).all()
    _, dw = g.moe_combine_backward(x, y, order, w)
    assert (dw[1] == 0).all() and dw[0, 1] == 0
    order = order._replace(offsets=torch.tensor([0, 1, 1 << 40], device=DEV))
    g.moe_gather(x, order)
    torch.cuda.synchronize()


def silu(v):
    return v / (1 + torch.exp(-v))


def test_layer_of_many_tokens_with_gradients():
    """x -> sort, gather, gate/up product, activation, down product, combine; and
    back, against the same in 64 bits."""
    say("layer")
    T, k, E, H, I = 200, 3, 6, 192, 128
    x, w1, w2 = randn(T, H, seed=1), randn(E, H, 2 * I, seed=2, scale=H ** -0.5), randn(E, I, H, seed=3, scale=I ** -0.5)
    p = torch.softmax(randn(T, k, dtype=F32, seed=4), dim=1)
    ids = torch.from_numpy(np.argsort(np.random.default_rng(1).random((T, E)), axis=1)[:, :k].copy()).to(DEV)
    ids[-7:] = -1                               # a padded batch
    order = g.moe_sort(ids, E)
    a = g.moe_gather(x, order)
    n = int(order.offsets[-1])
    z = torch.zeros(T * k, 2 * I, dtype=BF16, device=DEV)
    g.gemm_grouped(a, w1, order.offsets, out=z)
    act = (silu(z[:, :I].float()) * z[:, I:].float()).to(BF16)
    y = torch.zeros(T * k, H, dtype=BF16, device=DEV)
    g.gemm_grouped(act, w2, order.offsets, out=y)
    out = g.moe_combine(y, order, p)
    # 64 bits, token by token
    X, W1, W2, Pw, I_ = f64(x), f64(w1), f64(w2), f64(p), ids.cpu().numpy()
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = I_[t, j]
            if e >= 0:
                zz = X[t] @ W1[e]
                want[t] += Pw[t, j] * ((zz[:I] / (1 + np.exp(-zz[:I])) * zz[I:]) @ W2[e])
    # four roundings to bfloat16 on the way (gate, up, activation, y) and the output's
    assert np.linalg.norm(f64(out) - want) <= 4 * 2.0 ** -8 * np.linalg.norm(want)
    assert (out[-7:] == 0).all() and n == (T - 7) * k
    # backward: the experts' part by the same grouped products with transposed weights
    d = randn(T, H, seed=5, scale=0.1)
    dy, dp = g.moe_combine_backward(d, y, order, p)
    da = torch.zeros(T * k, I, dtype=BF16, device=DEV)
    g.gemm_grouped(dy, w2.transpose(1, 2), order.offsets, out=da)
    zf = z.float()
    sg = 1 / (1 + torch.exp(-zf[:, :I]))
    dz = torch.cat((da.float() * zf[:, I:] * sg * (1 + zf[:, :I] * (1 - sg)), da.float() * zf[:, :I] * sg), dim=1).to(BF16)
    dxs = torch.zeros(T * k, H, dtype=BF16, device=DEV)
    g.gemm_grouped(dz, w1.transpose(1, 2), order.offsets, out=dxs)
    dx = g.moe_combine(dxs, order)

    def loss(xv, pv):
        total = 0.0
        for t in range(T):
            for j in range(k):
                e = I_[t, j]
                if e >= 0:
                    zz = xv[t] @ W1[e]
                    total += pv[t, j] * (((zz[:I] / (1 + np.exp(-zz[:I])) * zz[I:]) @ W2[e]) @ f64(d)[t])
        return total

    rng = np.random.default_rng(2)
    for _ in range(3):
        u, s = rng.standard_normal((T, H)), 1e-5
        slope = (loss(X + s * u, Pw) - loss(X - s * u, Pw)) / (2 * s)
        # seven roundings to bfloat16, random against u
        assert abs(slope - (f64(dx) * u).sum()) <= 7 * 2.0 ** -8 * np.linalg.norm(f64(dx)) * 4
        u = rng.standard_normal((T, k))
        slope = (loss(X, Pw + s * u) - loss(X, Pw - s * u)) / (2 * s)
        assert abs(slope - (f64(dp) * u).sum()) <= 4 * 2.0 ** -8 * np.linalg.norm(f64(dp)) * 4
