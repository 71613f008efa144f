"""Block-scaled E4M3: the quantizers bit for bit against the oracle, block by
block, and the linear against the product of the dequantized operands in 64
bits.

The linear's bound, relative to S = sum_j |x_j w_j| of the dequantized
values: the tensor cores' sum of one block of 128 channels takes 4
instructions, each at most one fp32 ulp (2^-23) on the accumulator and one
more for its own sum, so 5 * 2^-23; the scales' product and the multiply-add
of each of the KB blocks are one rounding of 2^-24 each, the first on that
block's part of S and the second on at most S; and at most 8 partial sums are
added when a tile's channels are split.  Together (5 + 1/2 + KB/2 + 4) * 2^-23,
below (KB + 12) * 2^-23.  Rounding to the output type adds half a step.
"""
import numpy as np
import pytest
import torch

import oracle
import w8a8_post_quantization_channel_b200 as sq
from w8a8_post_quantization_channel_b200 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
B = 128


def blocks(n):
    return -(-n // B)


def block_bound(K):
    return (blocks(K) + 12) * 2.0 ** -23


def half_step(y, dt):
    """Half a step of `dt` at |y| (64-bit tensor); fp32 included."""
    tiny = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}[dt]
    return y.abs() * (torch.finfo(DT[dt]).eps / 2) + tiny


def oracle_rows(v):
    """(codes, scales) of fp32 v [R, K] per row and 128 columns, from the oracle's row quantizer."""
    R, K = v.shape
    pad = np.zeros((R, blocks(K) * B), np.float32)
    pad[:, :K] = v
    q, s = oracle.quant_act_e4m3(pad.reshape(-1, B), np.ones(B, np.float32))
    return q.reshape(R, -1)[:, :K], s.reshape(R, -1)


def oracle_weight(v):
    """(codes, scales) of fp32 v [E, N, K] per 128 x 128 block."""
    E, N, K = v.shape
    pad = np.zeros((E, blocks(N) * B, blocks(K) * B), np.float32)
    pad[:, :N, :K] = v
    t = pad.reshape(E, blocks(N), B, blocks(K), B).transpose(0, 1, 3, 2, 4)
    q, s = oracle.quant_act_e4m3(np.ascontiguousarray(t).reshape(-1, B * B), np.ones(B * B, np.float32))
    q = q.reshape(E, blocks(N), blocks(K), B, B).transpose(0, 1, 3, 2, 4).reshape(pad.shape)[:, :N, :K]
    return q, s.reshape(E, blocks(N), blocks(K))


def hard_rows(M, K, dt, seed):
    """Activations with outlier channels, zero blocks, signed zeros and blocks of tiny values."""
    o = synth.outliers(K, frac=0.02, mult=80.0, seed=seed)
    x = synth.activations(M, K, o, seed + 1, torch.float32)
    if M > 3:
        x[1] = 0
        x[2, : K // 2] = -0.0
        x[3] *= 2.0 ** -12 if dt == "f16" else 2.0 ** -130
    return x.to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 16), (5, 112), (1, 4096), (37, 1040), (9, 8208), (300, 528)])
@pytest.mark.parametrize("smooth", [True, False])
def test_quant_act_block_bit_exact(dt, M, K, smooth):
    x = hard_rows(M, K, dt, seed=M + K)
    inv = torch.exp(torch.randn(K, generator=synth.gen(K))) if smooth else None
    q, s = sq.sq_quant_act_e4m3_block(x.to(DEV), None if inv is None else inv.to(DEV))
    v = x.float().numpy()
    q_ref, s_ref = oracle_rows(v * inv.numpy() if smooth else v)
    np.testing.assert_array_equal(s.cpu().numpy(), s_ref)
    np.testing.assert_array_equal(q.cpu().numpy(), q_ref)


def test_quant_act_block_strided_rows_and_given_outputs():
    M, K = 70, 1040
    wide = hard_rows(M, 2 * K, "bf16", seed=3).to(DEV)
    x = wide[:, 16:16 + K]          # row stride 2K, 32-byte offset
    q = torch.empty(M, K, dtype=torch.uint8, device=DEV)
    s = torch.empty(M, blocks(K), device=DEV)
    out = sq.sq_quant_act_e4m3_block(x, xq=q, x_scale=s)
    assert out[0] is q and out[1] is s
    q_ref, s_ref = oracle_rows(x.float().cpu().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), s_ref)
    np.testing.assert_array_equal(q.cpu().numpy(), q_ref)


def test_quant_act_block_many_rows():
    # more rows than one pass of the grid covers, and an empty batch
    M, K = 20011, 272
    x = hard_rows(M, K, "f16", seed=8)
    q, s = sq.sq_quant_act_e4m3_block(x.to(DEV))
    q_ref, s_ref = oracle_rows(x.float().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), s_ref)
    np.testing.assert_array_equal(q.cpu().numpy(), q_ref)
    q, s = sq.sq_quant_act_e4m3_block(torch.empty(0, 256, device=DEV))
    assert q.shape == (0, 256) and s.shape == (0, 2)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("E,N,K", [(1, 16, 16), (1, 528, 1040), (3, 144, 400), (2, 256, 512)])
@pytest.mark.parametrize("alpha", [None, 0.25, 0.5])
def test_smooth_quant_weight_block_bit_exact(dt, E, N, K, alpha):
    w = synth.weights(K, E * N, K + N, torch.float32, "nk").reshape(E, N, K)
    w[0, :, : K // 3] = 0
    if dt != "f16":
        w[E - 1, N // 2:] *= 2.0 ** -125      # block scales below the normal range
    w = w.to(DT[dt])
    amax = None if alpha is None else 4.0 * torch.exp(torch.randn(K, generator=synth.gen(K)))
    q, ws, s, inv = sq.sq_smooth_quant_weight_e4m3_block(w.to(DEV), None if amax is None else amax.to(DEV),
                                                         0.5 if alpha is None else alpha)
    v = w.float().numpy()
    if alpha is None:
        assert s is None and inv is None
    else:
        wmax = oracle.weight_absmax(v.reshape(E * N, K), oracle.LAYOUT_NK)
        s_ref, inv_ref = oracle.smooth_factor(amax.numpy(), wmax, alpha)
        np.testing.assert_array_equal(s.cpu().numpy(), s_ref)
        np.testing.assert_array_equal(inv.cpu().numpy(), inv_ref)
        v = v * s_ref
    q_ref, ws_ref = oracle_weight(v)
    np.testing.assert_array_equal(ws.cpu().numpy(), ws_ref)
    np.testing.assert_array_equal(q.cpu().numpy(), q_ref)


def test_smooth_quant_weight_block_more_block_rows_than_a_grid_has():
    # 65538 block rows: beyond a grid's second dimension
    N, K = 65537 * B + 16, 16
    w = torch.randn(N, K, generator=torch.Generator(DEV).manual_seed(9), device=DEV, dtype=torch.float16)
    wq, ws, _, _ = sq.sq_smooth_quant_weight_e4m3_block(w)
    pad = torch.zeros(blocks(N) * B, K, device=DEV)
    pad[:N] = w.float()
    top = pad.view(-1, B * K).abs().amax(1)
    d = top / torch.full_like(top, 448)      # (by a Python number torch multiplies with the reciprocal)
    assert torch.equal(ws[:, 0], d)
    want = (pad.view(-1, B * K) / d[:, None]).view(-1, K)[:N].to(torch.float8_e4m3fn)
    assert torch.equal(wq, want.view(torch.uint8))
    assert sq.sq_check_device_error() == sq.SQ_OK


def test_smooth_quant_weight_block_strided_and_dense_shapes():
    wide = synth.weights(512, 272, 5, torch.bfloat16, "nk").to(DEV)
    w = wide[:, 64:64 + 272]
    q, ws, _, _ = sq.sq_smooth_quant_weight_e4m3_block(w)
    assert q.shape == (272, 272) and ws.shape == (3, 3)
    q_ref, ws_ref = oracle_weight(w.float().cpu().numpy()[None])
    np.testing.assert_array_equal(q.cpu().numpy(), q_ref[0])
    np.testing.assert_array_equal(ws.cpu().numpy(), ws_ref[0])
    with pytest.raises(ValueError):          # experts that do not follow one another
        sq.sq_smooth_quant_weight_e4m3_block(torch.zeros(2, 32, 64, device=DEV)[:, :16])


def operands(M, N, K, seed):
    """Block-scaled codes of outlier activations and Gaussian weights, on the device."""
    o = synth.outliers(K, frac=0.01, mult=60.0, seed=seed)
    x = synth.activations(M, K, o, seed + 1, torch.float32).to(DEV)
    w = synth.weights(K, N, seed + 2, torch.float32, "nk").to(DEV)
    xq, xs = sq.sq_quant_act_e4m3_block(x)
    wq, ws, _, _ = sq.sq_smooth_quant_weight_e4m3_block(w)
    return xq, xs, wq, ws


def dequantized(q, s, rows):
    """64-bit values; `rows`: code rows per scale row (1 or 128)."""
    v = q.view(torch.float8_e4m3fn).to(torch.float64)
    s = s.double().repeat_interleave(B, -1)[..., :q.shape[-1]]
    if rows > 1:
        s = s.repeat_interleave(rows, -2)[..., :q.shape[-2], :]
    return v * s


def check_block(y, xq, xs, wq, ws, dt):
    x, w = dequantized(xq, xs, 1), dequantized(wq, ws, B)
    exact, size = x @ w.t(), x.abs() @ w.abs().t()
    bound = block_bound(xq.shape[1]) * size
    bound = bound + half_step(exact.abs() + bound, dt)
    err = (y.double() - exact).abs()
    assert torch.all(err <= bound), f"worst error / bound: {float((err / bound.clamp_min(1e-300)).max()):.3g}"


SHAPES = [(1, 16, 16), (1, 4096, 4096), (2, 272, 1040), (16, 1024, 11008), (17, 528, 256), (33, 2048, 400),
          (64, 640, 2064), (65, 1024, 512), (128, 384, 1040), (129, 272, 128), (300, 1040, 2064), (256, 512, 16),
          (1000, 2064, 272), (2048, 1536, 1024)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_linear_block(M, N, K, dt):
    ops = operands(M, N, K, seed=M + N + K)
    y = sq.sq_w8a8_linear_e4m3_block(*ops, out_dtype=DT[dt])
    assert y.dtype == DT[dt] and y.shape == (M, N)
    check_block(y, *ops, dt)
    assert torch.equal(y, sq.sq_w8a8_linear_e4m3_block(*ops, out_dtype=DT[dt]))
    assert sq.sq_check_device_error() == sq.SQ_OK


def test_linear_block_scales_far_apart():
    # neighbouring blocks whose scales differ by 2^40, rows of zero scale, and
    # an infinite scale: only the rows and columns that it belongs to see it
    M, N, K = 40, 272, 784
    xq, xs, wq, ws = operands(M, N, K, seed=5)
    xs = xs * torch.exp2(torch.randint(-20, 21, xs.shape, generator=synth.gen(1)).to(DEV).float())
    ws = ws * torch.exp2(torch.randint(-20, 21, ws.shape, generator=synth.gen(2)).to(DEV).float())
    xs[7] = 0
    y = sq.sq_w8a8_linear_e4m3_block(xq, xs, wq, ws, torch.float32)
    check_block(y, xq, xs, wq, ws, "f32")
    assert torch.all(y[7] == 0)
    xs[9, 2] = float("inf")
    xq[11, 5] = 0x7f                      # an E4M3 NaN
    z = sq.sq_w8a8_linear_e4m3_block(xq, xs, wq, ws, torch.float32)
    keep = [r for r in range(M) if r not in (9, 11)]
    assert torch.equal(z[keep], y[keep])
    assert torch.all(~torch.isfinite(z[9])) and torch.all(torch.isnan(z[11]))


@pytest.mark.parametrize("M", [3, 200])
def test_linear_block_into_a_wider_matrix(M):
    N, K = 272, 528
    ops = operands(M, N, K, seed=17)
    wide = torch.full((M, 3 * N), 7.0, dtype=torch.bfloat16, device=DEV)
    y = sq.sq_w8a8_linear_e4m3_block(*ops, y=wide[:, N:2 * N])
    assert y.data_ptr() == wide.data_ptr() + 2 * N
    check_block(y, *ops, "bf16")
    assert torch.all(wide[:, :N] == 7.0) and torch.all(wide[:, 2 * N:] == 7.0)


def test_linear_block_refusals():
    xq, xs, wq, ws = operands(4, 256, 256, seed=1)
    f = sq.sq_w8a8_linear_e4m3_block
    for bad in [(xq.to(torch.int8), xs, wq, ws), (xq, xs[:, :1], wq, ws), (xq, xs, wq[:, :128], ws),
                (xq, xs, wq, ws.double()), (xq.t(), xs, wq, ws), (xq, xs.t().contiguous().t(), wq, ws),
                (xq, xs.cpu(), wq, ws)]:
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(ValueError):
        f(xq, xs, wq, ws, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        f(xq, xs, wq, ws, y=torch.empty(5, 256, device=DEV))
    with pytest.raises(ValueError):
        sq.sq_quant_act_e4m3_block(torch.zeros(4, 256, device=DEV), torch.ones(255, device=DEV))
    with pytest.raises(sq.SqError):
        sq.sq_quant_act_e4m3_block(torch.zeros(4, 24, device=DEV))       # K % 16
    assert f(xq[:0], xs[:0], wq, ws).shape == (0, 256)


def test_block_calls_on_another_stream_and_in_a_graph():
    M, N, K = 130, 528, 1040
    x = synth.activations(M, K, synth.outliers(K, frac=0.01, seed=3), 4, torch.bfloat16).to(DEV)
    wq, ws, _, _ = sq.sq_smooth_quant_weight_e4m3_block(synth.weights(K, N, 6, torch.float32).to(DEV))

    def chain(stream=None):
        q, s = sq.sq_quant_act_e4m3_block(x, stream=stream)
        return sq.sq_w8a8_linear_e4m3_block(q, s, wq, ws, stream=stream)

    y = chain()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = chain(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3 = chain()
    x.copy_(synth.activations(M, K, synth.outliers(K, frac=0.01, seed=3), 9, torch.bfloat16).to(DEV))
    graph.replay()
    y = chain()
    assert torch.equal(y, y3)
    assert sq.sq_check_device_error() == sq.SQ_OK


def _e4m3_midpoints():
    v = oracle.e4m3_decode(np.arange(256, dtype=np.uint8)).astype(np.float64)
    v = np.unique(np.abs(v[~np.isnan(v)]))
    return (v[1:] + v[:-1]) / 2


@pytest.mark.parametrize("kind", ["bf16_ties", "few_bits", "next_to_few_bits", "small"])
def test_codes_next_to_e4m3_midpoints(kind):
    # values within a few ulps of (E4M3 midpoint) * scale.  Scales: of bf16
    # maxima (exact ties), of four significant bits, within 20 ulps of those
    # (where only a division decides), and around 2^-90 and 2^-126
    rng = np.random.default_rng(7)
    R, K = 256, 512
    mids = _e4m3_midpoints()
    x = np.zeros((R, K), np.float32)
    for r in range(R):
        for b in range(K // B):
            if kind == "bf16_ties":
                d = rng.integers(128, 256) * 2.0 ** rng.integers(-12, 4) / 448.0
            elif kind == "small":
                d = rng.uniform(1, 2) * 2.0 ** rng.choice([-91, -90, -89, -125, -126, -127, -140])
            else:
                d = rng.integers(8, 16) / 8.0 * 2.0 ** rng.integers(-12, 4)
                if kind == "next_to_few_bits":
                    d *= 1 + rng.integers(-20, 21) * 2.0 ** -23
            m = np.float32(448.0 * d)
            d = np.float64(m / np.float32(448.0))
            v = (rng.choice(mids, B) * d).astype(np.float32)
            v = (v.view(np.int32) + np.where(v > 1e-37, rng.integers(-2, 3, B), 0).astype(np.int32)).view(np.float32)
            v *= rng.choice([-1, 1], B)
            v[rng.integers(0, B, 4)] = -0.0
            v = np.clip(v, -m, m)
            v[0] = m
            x[r, b * B:(b + 1) * B] = v
    t = torch.from_numpy(x)
    if kind == "bf16_ties":
        t = t.to(torch.bfloat16)
        x = t.float().numpy()
    q, s = sq.sq_quant_act_e4m3_block(t.to(DEV))
    q_ref, s_ref = oracle_rows(x)
    np.testing.assert_array_equal(s.cpu().numpy(), s_ref)
    np.testing.assert_array_equal(q.cpu().numpy(), q_ref)
    q, s, _, _ = sq.sq_smooth_quant_weight_e4m3_block(t.to(DEV))
    q_ref, s_ref = oracle_weight(x[None])
    np.testing.assert_array_equal(s.cpu().numpy(), s_ref[0])
    np.testing.assert_array_equal(q.cpu().numpy(), q_ref[0])


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (40, 272, 784), (333, 1040, 2064), (2048, 1536, 1024)])
def test_linear_block_scale_products_at_the_ends_of_the_range(M, N, K):
    # scale products below 2^-126 and up to 2^100 between ordinary ones.  A
    # subnormal product is within 2^-150 of the exact one, times a block's sum
    # of at most 128 * 448^2 < 2^25; adding below the normal range is off by
    # 2^-150 per block: together under KB * 2^-125
    xq, xs, wq, ws = operands(M, N, K, seed=23)
    ws, xs = ws / ws.max(), xs / xs.max()
    r = torch.arange(M, device=DEV) % 3
    for dt in ("f32", "bf16"):
        for w_shift, x_shift in ((-66, (-70, 0, 40)), (50, (50, -40, 0)), (-100, (-40, -49, -26))):
            x_scale = xs * torch.exp2(torch.tensor(x_shift, device=DEV, dtype=torch.float32))[r][:, None]
            w_scale = ws * 2.0 ** w_shift
            y = sq.sq_w8a8_linear_e4m3_block(xq, x_scale, wq, w_scale, DT[dt])
            x, w = dequantized(xq, x_scale, 1), dequantized(wq, w_scale, B)
            bound = block_bound(K) * (x.abs() @ w.abs().t()) + blocks(K) * 2.0 ** -125
            bound = bound + half_step((x @ w.t()).abs() + bound, dt)
            assert torch.all((y.double() - x @ w.t()).abs() <= bound), (dt, w_shift)
    assert sq.sq_check_device_error() == sq.SQ_OK
