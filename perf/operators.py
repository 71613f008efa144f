"""Workloads of the block-scaled FP8 and the expert-grouped linears.

Blocks of 128: an E4M3 code matrix carries one fp32 scale for each token and
128 input channels (activations, [M, ceil(K/128)]) or for each 128 x 128
block (weights, [N, K] -> [ceil(N/128), ceil(K/128)]); a block's largest
magnitude maps to 448.  Groups: the rows of X are sorted by expert, expert e
owns rows offsets[e] .. offsets[e+1], and has weights of its own.

  quant_act      codes and scales of X * inv_smooth, per token and block
  quant_weight   smoothing factors, codes and scales of diag(s) W, per block
  linear_block   Y = dequantized X times dequantized W, block scales
  grouped        the same per expert; "scale" says how codes are scaled:
                 i8 / e4m3 (per token and per output channel) or block

With `own` false, run() computes them with elementary torch operations in
fp32; with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

B = 128
_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_DEV = "cuda"


def listed():
    return [
        # one decoded token's hidden state: latency of a launch
        dict(name="act_1x4096", op="quant_act", M=1, K=4096, dt="bf16", smooth=True),
        # a long prompt batch at the widest input of a 70B-sized block
        dict(name="act_16384x8192", op="quant_act", M=16384, K=8192, dt="bf16", smooth=True),
        # one dense layer with odd widths (last blocks ragged both ways), no smoothing
        dict(name="weight_1040x2000", op="quant_weight", E=1, N=2000, K=1040, dt="f32", alpha=0.0),
        # the experts of one projection of a mixture layer, smoothed over their shared input
        dict(name="weight_8x11008x4096", op="quant_weight", E=8, N=11008, K=4096, dt="bf16", alpha=0.5),
        # single-token decode, attention output projection: streams the weight
        dict(name="block_1x4096x4096", op="linear_block", M=1, N=4096, K=4096, out="bf16"),
        # a small ragged prefill chunk, fp32 output
        dict(name="block_333x4096x11008", op="linear_block", M=333, N=4096, K=11008, out="f32"),
        # a full prefill batch of a 7B-sized gate projection
        dict(name="block_4096x11008x4096", op="linear_block", M=4096, N=11008, K=4096, out="bf16"),
        # decode with 8 sequences, two experts each, of 8
        dict(name="i8_16r_8e_4096x4096", op="grouped", scale="i8", T=16, E=8, N=4096, K=4096, skew=0.0, out="bf16"),
        # a mid-sized ragged batch over small experts of odd width
        dict(name="e4m3_1000r_16e_1360x2064", op="grouped", scale="e4m3", T=1000, E=16, N=1360, K=2064, skew=0.5,
             out="f16"),
        # prefill of 4096 tokens, two experts each, of 8
        dict(name="i8_8192r_8e_11008x4096", op="grouped", scale="i8", T=8192, E=8, N=11008, K=4096, skew=0.2,
             out="bf16"),
        # decode with 32 sequences over many small experts
        dict(name="block_192r_64e_1408x2048", op="grouped", scale="block", T=192, E=64, N=1408, K=2048, skew=0.3,
             out="bf16"),
        # prefill of 4096 tokens, six experts each, of 64 small ones
        dict(name="block_24576r_64e_1408x2048", op="grouped", scale="block", T=24576, E=64, N=1408, K=2048, skew=0.3,
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _16(v):
    return max(16, v // 16 * 16)


def draw(rng):
    op = rng.choice(["quant_act", "quant_weight", "linear_block", "grouped", "grouped"])
    while True:
        K = _16(_log(rng, 256, 16384))
        if op == "quant_act":
            c = dict(op=op, M=_log(rng, 1, 16384), K=K, dt=rng.choice(["bf16", "f16", "f32"]),
                     smooth=rng.random() < 0.5)
            if c["M"] * K <= 16384 * 8192:
                return c
        elif op == "quant_weight":
            c = dict(op=op, E=_log(rng, 1, 16), N=_16(_log(rng, 128, 16384)), K=K,
                     dt=rng.choice(["bf16", "f16", "f32"]), alpha=rng.choice([0.0, 0.25, 0.5, 0.75]))
            if c["E"] * c["N"] * K * (2 if c["dt"] == "f32" else 1) <= 8 * 11008 * 4096:
                return c
        elif op == "linear_block":
            c = dict(op=op, M=_log(rng, 1, 8192), N=_16(_log(rng, 128, 16384)), K=K,
                     out=rng.choice(["bf16", "f16", "f32"]))
            if c["M"] * c["N"] * K <= 4096 * 11008 * 4096 and c["N"] * K >= 1 << 18:
                return c
        else:
            c = dict(op=op, scale=rng.choice(["i8", "e4m3", "block", "block"]), T=_log(rng, 1, 24576),
                     E=_log(rng, 2, 128), N=_16(_log(rng, 256, 11008)), K=K,
                     skew=round(rng.uniform(0.0, 0.8), 2), out=rng.choice(["bf16", "f16", "f32"]))
            if (c["T"] * c["N"] * K <= 8192 * 11008 * 4096 // 2 and c["E"] * c["N"] * K <= 8 * 11008 * 4096
                    and c["T"] * max(c["N"], K) <= 1 << 28):
                return c


def _shares(E, skew):
    """Each expert's share of the routed rows."""
    p = np.arange(1, E + 1, dtype=np.float64) ** -skew
    return p / p.sum()


def _blocks(x):
    """x [..., R, K] -> fp32 view of it in whole blocks of 128 columns, zero-padded."""
    K = x.shape[-1]
    x = x.to(torch.float32)
    if K % B:
        x = torch.nn.functional.pad(x, (0, B - K % B))
    return x.reshape(*x.shape[:-1], -1, B)


def _codes(v, scale):
    """E4M3 codes of v / scale, +0 where the scale is 0."""
    return torch.where(scale > 0, v / scale, torch.zeros_like(v)).to(torch.float8_e4m3fn)


def _quant_rows(x):
    """Per row and 128 columns: (codes uint8 [R, K], scales [R, ceil(K/128)])."""
    v = _blocks(x)
    s = v.abs().amax(-1) / 448.0
    q = _codes(v, s.unsqueeze(-1)).reshape(x.shape[0], -1)[:, :x.shape[1]]
    return q.contiguous(), s


def _quant_weight(w):
    """Per 128 x 128 block: w [E, N, K] -> (codes [E, N, K], scales [E, ceil(N/128), ceil(K/128)])."""
    E, N, K = w.shape
    v = _blocks(torch.nn.functional.pad(w.to(torch.float32), (0, 0, 0, -N % B)))
    v = v.reshape(E, -1, B, v.shape[-2], B)
    s = v.abs().amax((2, 4)) / 448.0
    q = _codes(v, s[:, :, None, :, None]).reshape(E, v.shape[1] * B, -1)[:, :N, :K]
    return q.contiguous(), s


def _quant_plain(x, scale):
    """Per row (int8 or E4M3 codes over the whole row): x [..., R, K] -> (codes, scales [..., R])."""
    x = x.to(torch.float32)
    s = x.abs().amax(-1) / (127.0 if scale == "i8" else 448.0)
    v = x / s.unsqueeze(-1)
    return v.round().to(torch.int8) if scale == "i8" else v.to(torch.float8_e4m3fn), s


def _u8(q):
    """Codes as the library takes them: int8, or E4M3 patterns in uint8."""
    return q if q.dtype == torch.int8 else q.view(torch.uint8)


def _activations(g, M, K):
    """Rows of N(0, 1) with 0.5% of the channels 50 times larger, as such inputs have."""
    x = torch.randn(M, K, generator=g, device=_DEV)
    n = max(1, K // 200)
    x[:, torch.randperm(K, generator=g, device=_DEV)[:n]] *= 50.0
    return x


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 11)
    op, K = case["op"], case["K"]
    if op == "quant_act":
        x = _activations(g, case["M"], K).to(_DT[case["dt"]])
        inv = torch.exp(0.5 * torch.randn(K, generator=g, device=_DEV)) if case["smooth"] else None
        return dict(case=case, x=x, inv=inv)
    if op == "quant_weight":
        w = torch.randn(case["E"], case["N"], K, generator=g, device=_DEV, dtype=_DT[case["dt"]]) * 0.02
        amax = 4.0 * torch.exp(torch.randn(K, generator=g, device=_DEV)) if case["alpha"] > 0 else None
        return dict(case=case, w=w, amax=amax)
    out = _DT[case["out"]]
    if op == "linear_block":
        xq, xs = _quant_rows(_activations(g, case["M"], K))
        wq, ws = _quant_weight(0.02 * torch.randn(1, case["N"], K, generator=g, device=_DEV))
        return dict(case=case, xq=_u8(xq), xs=xs, wq=_u8(wq[0]), ws=ws[0], out=out)
    T, E = case["T"], case["E"]
    sizes = np.random.RandomState(int(seed) * 977 % (1 << 32)).multinomial(T, _shares(E, case["skew"]))
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=_DEV)
    x = _activations(g, T, K)
    w = 0.02 * torch.randn(E, case["N"], K, generator=g, device=_DEV)
    if case["scale"] == "block":
        (xq, xs), (wq, ws) = _quant_rows(x), _quant_weight(w)
    else:
        (xq, xs), (wq, ws) = _quant_plain(x, case["scale"]), _quant_plain(w, case["scale"])
    return dict(case=case, xq=_u8(xq), xs=xs, wq=_u8(wq), ws=ws, offsets=offsets, largest=int(sizes.max()), out=out)


def _values(q):
    return (q if q.dtype == torch.int8 else q.view(torch.float8_e4m3fn)).to(torch.float32)


def _over_rows(q, s):
    """Dequantized rows: codes [R, K] times scales [R, ceil(K/128)]."""
    return _values(q) * s.repeat_interleave(B, dim=-1)[..., :q.shape[-1]]


def _over_blocks(q, s):
    """Dequantized weights: codes [E, N, K] times block scales [E, ceil(N/128), ceil(K/128)]."""
    return _over_rows(q, s.repeat_interleave(B, dim=-2)[..., :q.shape[-2], :])


def _run_own(st):
    import w8a8_post_quantization_channel_b200 as sq
    case = st["case"]
    op = case["op"]
    if op == "quant_act":
        q, s = sq.sq_quant_act_e4m3_block(st["x"], st["inv"])
        return [q.view(torch.float8_e4m3fn), s]
    if op == "quant_weight":
        q, s, smooth, inv = sq.sq_smooth_quant_weight_e4m3_block(st["w"], st["amax"], case["alpha"])
        q = q.view(torch.float8_e4m3fn)
        return [q, s] if smooth is None else [q, s, smooth, inv]
    if op == "linear_block":
        return sq.sq_w8a8_linear_e4m3_block(st["xq"], st["xs"], st["wq"], st["ws"], st["out"])
    call = {"i8": sq.sq_w8a8_linear_grouped, "e4m3": sq.sq_w8a8_linear_grouped_e4m3,
            "block": sq.sq_w8a8_linear_grouped_e4m3_block}[case["scale"]]
    return call(st["xq"], st["xs"], st["wq"], st["ws"], st["offsets"], st["out"])


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    op = case["op"]
    if op == "quant_act":
        x = st["x"].to(torch.float32)
        return list(_quant_rows(x if st["inv"] is None else x * st["inv"]))
    if op == "quant_weight":
        w = st["w"].to(torch.float32)
        if st["amax"] is None:
            return list(_quant_weight(w))
        a = st["amax"].clamp_min(1e-5)
        s = a ** case["alpha"] / w.abs().amax((0, 1)).clamp_min(1e-5) ** (1.0 - case["alpha"])
        return [*_quant_weight(w * s), s, 1.0 / s]
    if op == "linear_block":
        x = _over_rows(st["xq"], st["xs"])
        return torch.matmul(x, _over_blocks(st["wq"][None], st["ws"][None])[0].t()).to(st["out"])
    # every expert's rows side by side, padded to the largest group, one
    # product per expert, and the rows back in their order
    row = torch.arange(case["T"], device=_DEV)
    e = torch.searchsorted(st["offsets"][1:].long(), row, right=True)
    at = row - st["offsets"].long()[e]
    if case["scale"] == "block":
        x, w = _over_rows(st["xq"], st["xs"]), _over_blocks(st["wq"], st["ws"])
    else:
        x, w = _values(st["xq"]) * st["xs"][:, None], _values(st["wq"]) * st["ws"][..., None]
    side = torch.zeros(case["E"], st["largest"], case["K"], device=_DEV)
    side[e, at] = x
    return torch.bmm(side, w.transpose(1, 2))[e, at].to(st["out"])


def work(case):
    op, K = case["op"], case["K"]
    kb = -(-K // B)
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if op == "quant_act":
        M = case["M"]
        return dict(bytes=M * K * (size[case["dt"]] + 1) + 4 * M * kb + (4 * K if case["smooth"] else 0),
                    flops=3 * M * K)
    if op == "quant_weight":
        n = case["E"] * case["N"]
        return dict(bytes=n * K * (size[case["dt"]] + 1) + 4 * case["E"] * -(-case["N"] // B) * kb
                    + (12 * K if case["alpha"] > 0 else 0), flops=3 * n * K)
    N = case["N"]
    if op == "linear_block":
        M = case["M"]
        return dict(bytes=M * K + 4 * M * kb + N * K + 4 * -(-N // B) * kb + M * N * size[case["out"]],
                    flops=2 * M * N * K)
    T, E = case["T"], case["E"]
    used = float(np.sum(1.0 - (1.0 - _shares(E, case["skew"])) ** T))  # experts with at least one row, on average
    block = case["scale"] == "block"
    rows = T * K + 4 * T * (kb if block else 1) + T * N * size[case["out"]] + 4 * (E + 1)
    return dict(bytes=rows + used * (N * K + 4 * (-(-N // B) * kb if block else N)), flops=2 * T * N * K)


def _e4m3_64(u):
    """The E4M3 value nearest to each u (ties to the even mantissa), |u| <= 448, in 64 bits."""
    e = torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(u / step) * step


def _block_exact(v):
    """Codes' values and scales of v [G, R, K] per block of R x 128."""
    G, R, K = v.shape
    kb = -(-K // B)
    s = torch.zeros(G, kb, dtype=torch.float64, device=v.device)
    q = torch.zeros_like(v)
    for b in range(kb):
        part = v[:, :, b * B:(b + 1) * B]
        s[:, b] = part.abs().amax((1, 2)) / 448.0
        d = s[:, b, None, None]
        q[:, :, b * B:(b + 1) * B] = _e4m3_64(part / torch.where(d > 0, d, torch.ones_like(d)))
    return q.to(torch.float32).to(torch.float8_e4m3fn), s


def exact(case, seed):
    st = prepare(case, seed)
    op, K = case["op"], case["K"]
    if op == "quant_act":
        v = st["x"].double()
        if st["inv"] is not None:
            v = v * st["inv"].double()
        q, s = _block_exact(v[:, None, :])
        return [q[:, 0, :], s]
    if op == "quant_weight":
        E, N = case["E"], case["N"]
        more = []
        smooth = torch.ones(K, dtype=torch.float64, device=_DEV)
        if st["amax"] is not None:
            top = st["w"].reshape(-1, K).abs().amax(0).double().clamp_min(1e-5)
            smooth = st["amax"].double().clamp_min(1e-5) ** case["alpha"] * top ** (case["alpha"] - 1.0)
            more = [smooth, smooth.reciprocal()]
        q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=_DEV)
        s = torch.empty(E, -(-N // B), -(-K // B), dtype=torch.float64, device=_DEV)
        for nb in range(s.shape[1]):
            rows = slice(nb * B, min(N, nb * B + B))
            q[:, rows], s[:, nb] = _block_exact(st["w"][:, rows].double() * smooth)
        return [q, s, *more]
    code = (lambda q: q.double()) if case.get("scale") == "i8" else (lambda q: q.view(torch.float8_e4m3fn).double())
    block = op == "linear_block" or case["scale"] == "block"

    def product(xq, xs, wq, ws):
        x, w = code(xq), code(wq)
        if not block:
            return (x @ w.t()) * xs.double()[:, None] * ws.double()
        y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=_DEV)
        for b in range(ws.shape[1]):
            part = x[:, b * B:(b + 1) * B] @ w[:, b * B:(b + 1) * B].t()
            wide = ws[:, b].double().repeat_interleave(B)[:w.shape[0]]
            y += part * xs[:, b].double()[:, None] * wide
        return y

    if op == "linear_block":
        return product(st["xq"], st["xs"], st["wq"], st["ws"])
    y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device=_DEV)
    bounds = st["offsets"].tolist()
    for e in range(case["E"]):
        rows = slice(bounds[e], bounds[e + 1])
        if bounds[e + 1] > bounds[e]:
            y[rows] = product(st["xq"][rows], st["xs"][rows], st["wq"][e], st["ws"][e])
    return y
