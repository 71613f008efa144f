"""Refusals of the block-scaled and the grouped calls, on the host: each call
below returns before its first CUDA call, or is refused by the binding."""
import ctypes

import pytest
import torch

import w8a8_post_quantization_channel_b200 as sq

INV, UNS = sq.SQ_ERR_INVALID_ARG, sq.SQ_ERR_UNSUPPORTED
A16 = 1 << 20          # a fake, 16-byte aligned address (never dereferenced)
MIS = (1 << 20) + 4    # misaligned


def _caller(f, base):
    def call(**kw):
        a = dict(base)
        assert set(kw) <= set(a)
        a.update(kw)
        return f(*a.values())
    return call


def test_quant_act_block():
    call = _caller(sq.lib().sq_quant_act_e4m3_block,
                   dict(x=A16, xt=sq.SQ_BF16, M=8, K=256, ldx=256, inv=A16, xq=A16, xs=A16, st=None))
    assert call(M=0) == sq.SQ_OK
    assert call(M=0, x=None, xq=None, xs=None) == sq.SQ_OK
    for bad in (dict(x=None), dict(x=MIS), dict(xt=7), dict(M=-1), dict(M=1 << 31), dict(K=0), dict(K=24),
                dict(K=1 << 31), dict(ldx=128), dict(ldx=260), dict(inv=MIS), dict(xq=None), dict(xq=MIS),
                dict(xs=None), dict(xs=MIS)):
        assert call(**bad) == INV, bad


def test_smooth_quant_weight_block():
    base = dict(w=A16, wt=sq.SQ_F16, E=4, N=512, K=256, ldw=256, amax=A16, alpha=ctypes.c_float(0.5), wq=A16, ws=A16,
                s=A16, inv=A16, st=None)
    call = _caller(sq.lib().sq_smooth_quant_weight_e4m3_block, base)
    for bad in (dict(w=None), dict(w=MIS), dict(wt=3), dict(E=0), dict(E=-1), dict(E=1 << 23), dict(N=500), dict(N=0),
                dict(K=248), dict(ldw=128), dict(ldw=258), dict(amax=MIS), dict(alpha=ctypes.c_float(-0.1)),
                dict(alpha=ctypes.c_float(1.5)), dict(alpha=ctypes.c_float(float("nan"))), dict(wq=None), dict(wq=MIS),
                dict(ws=None), dict(ws=MIS), dict(s=None), dict(s=MIS), dict(inv=None), dict(inv=MIS)):
        assert call(**bad) == INV, bad


def test_linear_block():
    call = _caller(sq.lib().sq_w8a8_linear_e4m3_block,
                   dict(xq=A16, xs=A16, wq=A16, ws=A16, M=64, N=256, K=256, y=A16, yt=sq.SQ_BF16, ldy=256, st=None))
    assert call(M=0) == sq.SQ_OK
    assert call(M=0, xq=None, xs=None, y=None) == sq.SQ_OK
    for bad in (dict(xq=None), dict(xq=MIS), dict(xs=None), dict(xs=MIS), dict(wq=None), dict(wq=MIS), dict(ws=None),
                dict(ws=MIS), dict(M=-1), dict(M=1 << 31), dict(N=40), dict(N=0), dict(K=40), dict(K=0), dict(y=None),
                dict(y=MIS), dict(yt=9), dict(ldy=128), dict(ldy=257)):
        assert call(**bad) == INV, bad
    assert call(M=(1 << 31) - 1023) == UNS


@pytest.mark.parametrize("name", ["sq_w8a8_linear_grouped", "sq_w8a8_linear_grouped_e4m3",
                                  "sq_w8a8_linear_grouped_e4m3_block"])
def test_grouped(name):
    call = _caller(getattr(sq.lib(), name),
                   dict(xq=A16, xs=A16, wq=A16, ws=A16, off=A16, T=64, E=4, N=256, K=256, y=A16, yt=sq.SQ_BF16,
                        ldy=256, st=None))
    assert call(T=0) == sq.SQ_OK
    assert call(T=0, xq=None, xs=None, y=None) == sq.SQ_OK
    for bad in (dict(xq=None), dict(xq=MIS), dict(xs=None), dict(xs=MIS), dict(wq=None), dict(wq=MIS), dict(ws=None),
                dict(ws=MIS), dict(off=None), dict(off=A16 + 2), dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=-3),
                dict(E=1 << 23), dict(N=40), dict(K=40), dict(K=0), dict(y=None), dict(y=MIS), dict(yt=9),
                dict(ldy=128), dict(ldy=257)):
        assert call(**bad) == INV, bad
    assert call(E=1025) == UNS
    assert call(T=(1 << 31) - 2048, N=1 << 20, ldy=1 << 20) == UNS    # more tiles than are numbered in 32 bits
    assert call(T=(1 << 31) - 1023) == UNS                            # a tile's last rows pass 2^31


def test_binding_refuses_what_it_cannot_pass_on():
    # host tensors, and (checked before the device) types and shapes
    u8 = torch.zeros(4, 256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        sq.sq_quant_act_e4m3_block(torch.zeros(4, 16))
    with pytest.raises(ValueError):
        sq.sq_smooth_quant_weight_e4m3_block(torch.zeros(4, 16))
    with pytest.raises(ValueError):
        sq.sq_smooth_quant_weight_e4m3_block(torch.zeros(16))
    with pytest.raises(ValueError):
        sq.sq_w8a8_linear_e4m3_block(u8, torch.zeros(4, 2), u8, torch.zeros(1, 2))
    with pytest.raises(ValueError):
        sq.sq_w8a8_linear_grouped(u8.to(torch.int8), torch.zeros(4), u8, torch.zeros(1, 4),
                                  torch.zeros(2, dtype=torch.int32))


def test_widths_whose_last_tile_passes_2_31():
    # counted in 32 bits on the device, a tile's last column or channel would wrap
    big = 1 << 31
    call = _caller(sq.lib().sq_w8a8_linear_e4m3_block,
                   dict(xq=A16, xs=A16, wq=A16, ws=A16, M=1, N=16, K=16, y=A16, yt=sq.SQ_BF16, ldy=big, st=None))
    for wide in (dict(N=big - 16), dict(N=big - 1008), dict(K=big - 16), dict(K=big - 1008)):
        assert call(**wide) == UNS, wide
    for name in ("sq_w8a8_linear_grouped", "sq_w8a8_linear_grouped_e4m3", "sq_w8a8_linear_grouped_e4m3_block"):
        call = _caller(getattr(sq.lib(), name), dict(xq=A16, xs=A16, wq=A16, ws=A16, off=A16, T=1, E=1, N=16, K=16,
                                                     y=A16, yt=sq.SQ_F32, ldy=big, st=None))
        for wide in (dict(N=big - 16), dict(K=big - 16), dict(E=23, N=(big // 23) // 16 * 16)):
            assert call(**wide) == UNS, (name, wide)
