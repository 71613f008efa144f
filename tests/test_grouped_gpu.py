"""Linears over rows grouped by expert, against each group's own product.

INT8: the int32 sums are exact, so y is the fp32 dequantization of the exact
sum bit for bit.  E4M3: within the fp32 accumulator's bound of the dense call
((K/32 + 17) * 2^-23 of sum |x w|) and the two products of the dequantization
(2^-24 each).  Block scales: the bound of the dense block-scaled linear.
Rounding to the output type adds half a step.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import w8a8_post_quantization_channel_b200 as sq
from w8a8_post_quantization_channel_b200 import synth

from .test_block_gpu import B, DT, block_bound, blocks, check_block, dequantized, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
CALL = {"i8": sq.sq_w8a8_linear_grouped, "e4m3": sq.sq_w8a8_linear_grouped_e4m3,
        "block": sq.sq_w8a8_linear_grouped_e4m3_block}


def codes(T, E, N, K, scale, seed):
    """(xq, xs, wq, ws) on the device: codes of every value and scales of different sizes."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def one(*shape):
        if scale == "i8":
            return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
        v = torch.randn(shape, generator=g, device=DEV) * 100.0
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def scales(*shape):
        return torch.rand(shape, generator=g, device=DEV) * 0.01 + 1e-4
    xs = scales(T, blocks(K)) if scale == "block" else scales(T)
    ws = scales(E, blocks(N), blocks(K)) if scale == "block" else scales(E, N)
    return one(T, K), xs, one(E, N, K), ws


def offsets_of(sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]), dtype=torch.int32, device=DEV)


def check(y, xq, xs, wq, ws, off, scale, dt):
    """Every group's rows of y, on the host's copy of valid offsets."""
    off = off.tolist()
    for e in range(len(off) - 1):
        r = slice(off[e], off[e + 1])
        if r.start == r.stop:
            continue
        if scale == "block":
            check_block(y[r], xq[r], xs[r], wq[e], ws[e], dt)
            continue
        value = (lambda q: q.double()) if scale == "i8" else (lambda q: q.view(torch.float8_e4m3fn).double())
        x, w = value(xq[r]), value(wq[e])
        acc = x @ w.t()
        if scale == "i8":
            assert torch.equal(y[r], ((acc.float() * xs[r, None]) * ws[e]).to(DT[dt])), e
        else:
            s = xs[r, None].double() * ws[e].double()
            exact = acc * s
            bound = (xq.shape[1] / 32 + 17 + 2) * 2.0 ** -23 * (x.abs() @ w.abs().t()) * s
            bound = bound + half_step(exact.abs() + bound, dt)
            assert torch.all((y[r].double() - exact).abs() <= bound), e


GROUPS = {
    "one_row": [1],
    "one_row_of_many_experts": [0, 0, 1, 0],
    "single_rows": [1] * 24,
    "few_each": [3, 0, 17, 1, 16, 5, 0, 0, 33, 2],
    "around_tiles": [127, 1, 128, 0, 129, 255, 256, 257, 64, 65],
    "all_in_one": [0, 700, 0],
    "skewed": [900, 300, 120, 60, 30, 15, 7, 3, 1, 0],
}


@pytest.mark.parametrize("scale", ["i8", "e4m3", "block"])
@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("N,K,dt", [(272, 528, "bf16"), (1040, 128, "f32"), (128, 2064, "f16")])
def test_groups(scale, groups, N, K, dt):
    sizes = GROUPS[groups]
    T, E = sum(sizes), len(sizes)
    ops = codes(T, E, N, K, scale, seed=T + N + K)
    off = offsets_of(sizes)
    y = CALL[scale](*ops, off, DT[dt])
    assert y.shape == (T, N) and y.dtype == DT[dt]
    check(y, *ops, off, scale, dt)
    assert torch.equal(y, CALL[scale](*ops, off, DT[dt]))
    assert sq.sq_check_device_error() == sq.SQ_OK


@pytest.mark.parametrize("scale", ["i8", "e4m3", "block"])
@pytest.mark.parametrize("sizes,N,K", [([2, 0, 5, 1], 16, 16), ([40] * 64, 1408, 256), ([1, 0] * 512, 144, 144),
                                       ([1500, 2000, 800], 2064, 784), ([5, 3, 8, 0, 0, 0, 0, 0], 4096, 4096)])
def test_sizes(scale, sizes, N, K):
    ops = codes(sum(sizes), len(sizes), N, K, scale, seed=N)
    off = offsets_of(sizes)
    check(CALL[scale](*ops, off), *ops, off, scale, "bf16")
    assert sq.sq_check_device_error() == sq.SQ_OK


@pytest.mark.parametrize("scale", ["i8", "e4m3", "block"])
@pytest.mark.parametrize("sizes", [[5, 0, 9, 2], [130, 0, 300, 70]])
def test_rows_in_no_group_are_left_as_they_were(scale, sizes):
    # rows before the first group and behind the last, with codes and scales
    # that are not numbers; y is a window of a wider matrix
    N, K, first, behind = 272, 400, 19, 37
    T = first + sum(sizes) + behind
    xq, xs, wq, ws = codes(T, len(sizes), N, K, scale, seed=3)
    out = torch.ones(T, dtype=torch.bool, device=DEV)
    out[first:T - behind] = False
    if scale != "i8":
        xq[out] = 0x7f
    xs[out] = float("nan")
    off = offsets_of(sizes, first)
    wide = torch.full((T, 2 * N), -3.0, dtype=torch.float16, device=DEV)
    y = CALL[scale](xq, xs, wq, ws, off, y=wide[:, N:])
    check(y, xq, xs, wq, ws, off, scale, "f16")
    assert torch.all(wide[:, :N] == -3.0) and torch.all(wide[out] == -3.0)


@pytest.mark.parametrize("scale", ["i8", "block"])
@pytest.mark.parametrize("T", [24, 600])
def test_offsets_out_of_order_stay_inside(scale, T):
    # documented: clamped to [0, T], a falling offset raised to the largest before it
    E, N, K = 6, 272, 272
    ops = codes(T, E, N, K, scale, seed=9)
    bad = [-5, T // 3, T // 6, T // 2, -(2 ** 31), 2 ** 31 - 1, T // 4]
    top, good = 0, []
    for v in bad:
        top = max(top, min(max(v, 0), T))
        good.append(top)
    y = CALL[scale](*ops, torch.tensor(bad, dtype=torch.int32, device=DEV), torch.float32)
    off = torch.tensor(good, dtype=torch.int32, device=DEV)
    check(y, *ops, off, scale, "f32")
    assert sq.sq_check_device_error() == sq.SQ_OK


@pytest.mark.parametrize("scale", ["i8", "block"])
@pytest.mark.parametrize("T,E,K", [(5, 3, 1024), (500, 2, 4096)])
def test_no_rows_in_any_group(scale, T, E, K):
    ops = codes(T, E, 272, K, scale, seed=6)
    y = torch.full((T, 272), 5.0, dtype=torch.bfloat16, device=DEV)
    for first in (0, T // 2, T):
        CALL[scale](*ops, torch.full((E + 1,), first, dtype=torch.int32, device=DEV), y=y)
    assert torch.all(y == 5.0)
    assert sq.sq_check_device_error() == sq.SQ_OK


def test_int8_groups_equal_the_dense_call():
    N, K, sizes = 528, 1040, [70, 1, 0, 200, 33]
    xq, xs, wq, ws = codes(sum(sizes), len(sizes), N, K, "i8", seed=4)
    off = offsets_of(sizes)
    y = sq.sq_w8a8_linear_grouped(xq, xs, wq, ws, off)
    o = off.tolist()
    for e, n in enumerate(sizes):
        if n:
            r = slice(o[e], o[e + 1])
            assert torch.equal(y[r], sq.sq_w8a8_linear(xq[r].clone(), xs[r].clone(), wq[e].clone(), ws[e].clone()))


@pytest.mark.parametrize("scale", ["i8", "e4m3", "block"])
def test_one_graph_serves_changing_groups_and_streams(scale):
    T, E, N, K = 150, 8, 272, 528
    ops = codes(T, E, N, K, scale, seed=12)
    off = offsets_of([20, 0, 60, 10, 10, 50, 0, 0])
    CALL[scale](*ops, off)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = CALL[scale](*ops, off)
        graphs.append((graph, y))
    for sizes in ([150, 0, 0, 0, 0, 0, 0, 0], [0, 1, 2, 3, 4, 5, 6, 129], [0] * 7 + [150]):
        off.copy_(offsets_of(sizes))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for i, (graph, y) in enumerate(graphs):     # two at once, on two streams
            with torch.cuda.stream(side if i else torch.cuda.current_stream()):
                graph.replay()
        torch.cuda.synchronize()
        for graph, y in graphs:
            check(y, *ops, off, scale, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = CALL[scale](*ops, off, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(y, *ops, off, scale, "bf16")
    assert sq.sq_check_device_error() == sq.SQ_OK


def test_first_call_of_a_process_is_captured():
    # nothing that a call sets up on first use may need to run outside a capture
    code = """
import torch
import w8a8_post_quantization_channel_b200 as sq
x = torch.randn(40, 528, device="cuda")
w = torch.randn(3, 272, 528, device="cuda")
off = torch.tensor([0, 7, 7, 40], dtype=torch.int32, device="cuda")
def run():
    q, s = sq.sq_quant_act_e4m3_block(x)
    wq, ws, _, _ = sq.sq_smooth_quant_weight_e4m3_block(w)
    return sq.sq_w8a8_linear_grouped_e4m3_block(q, s, wq, ws, off, torch.float32)
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    y = run()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, run())
assert sq.sq_check_device_error() == sq.SQ_OK
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_outputs_past_two_gib_elements():
    # y of more than 2^31 elements: rows on both sides of the border
    T, N, K = 140000, 16384, 16
    ops = codes(T, 2, N, K, "i8", seed=2)
    assert T * N > 2 ** 31
    off = offsets_of([100, T - 100])
    y = sq.sq_w8a8_linear_grouped(*ops, off)
    xq, xs, wq, ws = ops
    for r in (slice(0, 50), slice(131000, 131200), slice(T - 50, T)):
        w, s = (wq[0], ws[0]) if r.start < 100 else (wq[1], ws[1])
        acc = xq[r].double() @ w.double().t()
        assert torch.equal(y[r], ((acc.float() * xs[r, None]) * s).to(torch.bfloat16))


def test_refusals():
    xq, xs, wq, ws = codes(8, 3, 256, 256, "i8", seed=1)
    off = offsets_of([2, 3, 3])
    f = sq.sq_w8a8_linear_grouped
    for bad in [(xq, xs, wq, ws, off.long()), (xq, xs, wq, ws, off[:3]), (xq, xs, wq, ws, off.cpu()),
                (xq, xs, wq[0], ws, off), (xq, xs, wq, ws[0], off), (xq, xs[:7], wq, ws, off),
                (xq.view(torch.uint8), xs, wq, ws, off), (xq, xs, wq.transpose(1, 2), ws, off),
                (xq, xs, wq, ws.double(), off)]:
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(ValueError):
        f(xq, xs, wq, ws, off, torch.float64)
    with pytest.raises(ValueError):
        f(xq, xs, wq, ws, off, y=torch.empty(8, 512, device=DEV))
    with pytest.raises(sq.SqError):
        f(xq[:, :24].contiguous(), xs, wq[:, :, :24].contiguous(), ws, off)     # K % 16
    with pytest.raises(sq.SqError):
        sq.sq_w8a8_linear_grouped_e4m3(*codes(8, 1025, 16, 16, "e4m3", 1), offsets_of([8] + [0] * 1024))
    assert f(xq[:0], xs[:0], wq, ws, offsets_of([0, 0, 0])).shape == (0, 256)


@pytest.mark.parametrize("T", [6, 300])
def test_a_mixture_layer_end_to_end(T):
    """Two experts of eight per token: rows sorted by expert, quantized with the
    experts' shared smoothing, multiplied up, quantized, multiplied down, and
    added back per token; each product within its bound of the 64-bit product
    of its own codes, the whole near the layer in 64 bits."""
    E, K, H, top = 8, 528, 1040, 2
    o = synth.outliers(K, frac=0.01, mult=60.0, seed=1)
    x = synth.activations(T, K, o, 2, torch.bfloat16).to(DEV)
    up = synth.weights(K, E * H, 3, torch.bfloat16).reshape(E, H, K).to(DEV)
    down = synth.weights(H, E * K, 4, torch.bfloat16).reshape(E, K, H).to(DEV)
    logits = torch.randn(T, E, generator=synth.gen(5)).to(DEV)
    gate, expert = logits.softmax(-1).topk(top)
    order = expert.flatten().argsort(stable=True)
    token = order // top
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV),
                     torch.bincount(expert.flatten(), minlength=E).cumsum(0)]).to(torch.int32)

    amax = torch.zeros(K, device=DEV)
    sq.sq_calib_absmax(x, amax)
    uq, us, _, inv = sq.sq_smooth_quant_weight_e4m3_block(up, amax, 0.5)
    dq, ds, _, _ = sq.sq_smooth_quant_weight_e4m3_block(down)
    xq, xs = sq.sq_quant_act_e4m3_block(x[token], inv)
    h = sq.sq_w8a8_linear_grouped_e4m3_block(xq, xs, uq, us, off)
    check(h, xq, xs, uq, us, off, "block", "bf16")
    a = torch.nn.functional.silu(h)
    aq, as_ = sq.sq_quant_act_e4m3_block(a)
    y = sq.sq_w8a8_linear_grouped_e4m3_block(aq, as_, dq, ds, off, torch.float32)
    check(y, aq, as_, dq, ds, off, "block", "f32")
    out = torch.zeros(T, K, device=DEV).index_add_(0, token, y * gate.flatten()[order, None])

    # the layer in 64 bits, and how far 4-bit significands (2^-4 relative per
    # operand, each product's errors added in magnitude) may move it
    src = expert.flatten()[order]
    xe, ue, de = x.double()[token], up.double(), down.double()
    hx = torch.stack([ue[e] @ v for e, v in zip(src.tolist(), xe)])
    hb = torch.stack([ue[e].abs() @ v.abs() for e, v in zip(src.tolist(), xe)])
    r = 2 * 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -7      # both operands, their product, underflowing codes and bf16
    ax = torch.nn.functional.silu(hx)
    ea = 1.1 * (hb * r + hx.abs() * 2.0 ** -8)     # |silu'| <= 1.1
    yx = torch.stack([de[e] @ v for e, v in zip(src.tolist(), ax)])
    yb = torch.stack([de[e].abs() @ (v.abs() * r + d * (1 + r)) for e, v, d in zip(src.tolist(), ax, ea)])
    g = gate.flatten()[order, None].double()
    want = torch.zeros(T, K, dtype=torch.float64, device=DEV).index_add_(0, token, yx * g)
    room = torch.zeros(T, K, dtype=torch.float64, device=DEV).index_add_(0, token, yb * g)
    assert torch.all((out.double() - want).abs() <= room + 1e-5 * want.abs())
    assert sq.sq_check_device_error() == sq.SQ_OK


@pytest.mark.parametrize("scale", ["i8", "e4m3", "block"])
@pytest.mark.parametrize("sizes", [[1, 5, 17, 31, 3, 29, 8, 23], [33, 63, 40, 1, 127, 97, 65, 100]])
def test_split_tiles_of_ragged_groups(scale, sizes):
    # 256 tiles of 32 blocks over clusters whose CTAs hold the end of one tile
    # and the beginning of another, of groups that end inside a warp's 32 rows
    N, K = 4096, 4096
    ops = codes(sum(sizes), len(sizes), N, K, scale, seed=31)
    off = offsets_of(sizes)
    y = CALL[scale](*ops, off, torch.float32)
    check(y, *ops, off, scale, "f32")
    for _ in range(5):
        assert torch.equal(y, CALL[scale](*ops, off, torch.float32))
    assert sq.sq_check_device_error() == sq.SQ_OK


@pytest.mark.parametrize("scale", ["i8", "e4m3"])
@pytest.mark.parametrize("T", [6, 300])
def test_experts_quantized_by_the_dense_calls(scale, T):
    """The documented way to the codes of INT8 and E4M3 experts: one dense
    quantizer call over the stacked weights, its results viewed per expert.
    Against the layer in 64 bits: an INT8 code is off by at most half a scale,
    an E4M3 code by 2^-4 of its value or, below 2^-6, by 2^-10; the fp32
    roundings of s, 1/s, x~, w~, their quotients and the dequantization are
    under 20 of 2^-23 together, and the E4M3 sum is off by K/32 + 17 of them."""
    E, K, N = 8, 528, 272
    x = synth.activations(T, K, synth.outliers(K, frac=0.01, mult=60.0, seed=1), 2, torch.bfloat16).to(DEV)
    w = synth.weights(K, E * N, 3, torch.bfloat16).reshape(E, N, K).to(DEV)
    expert = torch.randint(0, E, (T,), generator=synth.gen(4)).to(DEV).sort().values
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV),
                     torch.bincount(expert, minlength=E).cumsum(0)]).to(torch.int32)
    amax = torch.zeros(K, device=DEV)
    sq.sq_calib_absmax(x, amax)
    i8 = scale == "i8"
    quant_w, quant_x = ((sq.sq_smooth_quant_weight, sq.sq_quant_act) if i8 else
                        (sq.sq_smooth_quant_weight_e4m3, sq.sq_quant_act_e4m3))
    wq, ws, s, inv = quant_w(w.view(E * N, K), sq.SQ_W_NK, amax, 0.5)
    xq, xs = quant_x(x, inv)
    wq, ws = wq.view(E, N, K), ws.view(E, N)
    y = CALL[scale](xq, xs, wq, ws, off, torch.float32)
    check(y, xq, xs, wq, ws, off, scale, "f32")

    def size_and_error(v, d):
        v = v.abs()
        return (v, (d / 2).expand_as(v)) if i8 else (v, v * 2.0 ** -4 + d * 2.0 ** -10)
    ulps = ((0 if i8 else K / 32 + 17) + 20) * 2.0 ** -23
    o = off.tolist()
    for e in range(E):
        r = slice(o[e], o[e + 1])
        exact = x[r].double() @ w[e].double().t()
        xv, xe = size_and_error(x[r].double() * inv.double(), xs[r, None].double())
        wv, we = size_and_error(w[e].double() * s.double(), ws[e, :, None].double())
        room = xv @ we.t() + xe @ wv.t() + xe @ we.t() + ulps * ((xv + xe) @ (wv + we).t())
        assert torch.all((y[r].double() - exact).abs() <= room), e
    assert sq.sq_check_device_error() == sq.SQ_OK
