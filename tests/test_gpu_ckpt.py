"""8-bit activation checkpoints: codes and scales bit for bit against the
oracle's block quantisers, values read back, non-finite blocks, and the
backward calls that take x from them."""

import numpy as np
import pytest
import torch

from sparse_moe_block_amd import fwmoe as fw
from . import dense_ref as ref
from .dense_ref import BF16, F32
from .test_gpu_dense import Case, out

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": BF16, "f32": F32}


def buffers(R, K, fmt):
    if fmt == "mxfp8":
        return (torch.full((R, K), 0x5A, dtype=torch.uint8, device=DEV),
                torch.full((R, K // 32), 0x5A, dtype=torch.uint8, device=DEV))
    return (torch.full((R, K), 0x5A, dtype=torch.int8, device=DEV),
            torch.full((R, K // 32), 77.0, dtype=F32, device=DEV))


def header():
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    fw.fw_moe_clear_status(ws)
    return ws


def pack(x, fmt, ws=None):
    R, K = x.shape
    d = fw.make_ckpt_desc(K, fmt, src_dtype="f32" if x.dtype == F32 else "bf16")
    codes, scales = buffers(R, K, fmt)
    fw.fw_moe_ckpt_pack(d, R, x.to(DEV), codes, scales, header() if ws is None else ws)
    return codes, scales


def inputs(R, K, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + R + K)
    x = torch.randn(R, K, generator=g) * torch.exp(3 * torch.randn(R, K // 32, generator=g)
                                                   ).repeat_interleave(32, 1)
    x[0, :32] = 0                               # an all-zero block
    if R > 1:
        x[1, :32] = 0
        x[1, 5] = -2.0 ** -120                  # a tiny block
        x[-1, -32:] = torch.linspace(-1, 1, 32) * 448   # codes on grid points and halves
    return x.to(dtype)


def oracle_pack(ref_lib, x, fmt):
    from oracle import fwref
    quant = fwref.mxfp8_quantize if fmt == "mxfp8" else fwref.q8a_quantize
    codes, scales = quant(x.float().numpy().reshape(-1))
    return np.asarray(codes).reshape(x.shape), np.asarray(scales).reshape(x.shape[0], -1)


def decoded(codes, scales, fmt):
    """The bf16 values of host codes and scales, in float64."""
    c, s = codes.cpu(), scales.cpu()
    if fmt == "mxfp8":
        v = c.view(torch.float8_e4m3fn).float().double()
        sc = torch.exp2(s.double() - 127)
    else:
        v, sc = c.double(), s.double()
    v = (v.reshape(*s.shape, 32) * sc[..., None]).reshape(c.shape)
    return v.float().bfloat16().double()


@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["mxfp8", "int8"])
@pytest.mark.parametrize("R,K", [(1, 32), (1, 96), (3, 64), (17, 2048), (130, 416), (1000, 32)])
def test_pack_matches_the_oracle(ref, R, K, fmt, src):
    x = inputs(R, K, DT[src])
    ws = header()
    codes, scales = pack(x, fmt, ws)
    want_c, want_s = oracle_pack(ref, x, fmt)
    assert np.array_equal(codes.cpu().numpy().view(np.uint8), want_c.view(np.uint8))
    assert np.array_equal(scales.cpu().numpy(), want_s.astype(scales.cpu().numpy().dtype))
    assert fw.fw_moe_read_status(ws) == 0
    for dst in ("bf16", "f32"):
        d = fw.make_ckpt_desc(K, fmt, src_dtype=src, dst_dtype=dst)
        y = out(R, K, dtype=DT[dst])
        fw.fw_moe_ckpt_unpack(d, R, codes, scales, y)
        assert torch.equal(y.double().cpu(), decoded(codes, scales, fmt))
    # how near the values are: half a code step, then the bf16 rounding of the
    # decoded int8 values (MXFP8's are exact in bf16)
    v, y = x.double().reshape(R, -1, 32), decoded(codes, scales, fmt).reshape(R, -1, 32)
    amax = v.abs().amax(-1, keepdim=True)
    if fmt == "int8":
        bound = amax / 127 * (0.5 + 1e-6) + 2.0 ** -8 * amax
    else:
        # E4M3 (half a step is 2^-4 relative, 2^-10 scales below its normal
        # range), saturated by at most 1/8 at the top of a block
        scale = torch.exp2(scales.cpu().double() - 127)[..., None]
        bound = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * scale)
        bound = torch.where(v.abs() > 448 * scale, v.abs() - 448 * scale, bound)
    assert ((v - y).abs() <= bound).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "int8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_non_finite_blocks(fmt, bad, src):
    """A non-finite value makes its block NaN, sets FW_STATUS_RANGE, and leaves
    every other block as it is without it."""
    x = inputs(5, 128, DT[src])
    clean = pack(x, fmt)
    x2 = x.clone()
    x2[2, 33] = bad
    ws = header()
    codes, scales = pack(x2, fmt, ws)
    assert fw.fw_moe_read_status(ws) == fw.FW_STATUS_RANGE
    y = out(5, 128)
    fw.fw_moe_ckpt_unpack(fw.make_ckpt_desc(128, fmt), 5, codes, scales, y)
    hit = torch.zeros(5, 128, dtype=torch.bool, device=DEV)
    hit[2, 32:64] = True
    assert torch.isnan(y[hit]).all() and torch.isfinite(y[~hit]).all()
    assert torch.equal(codes[~hit], clean[0][~hit])


@pytest.mark.parametrize("fmt", ["mxfp8", "int8"])
@pytest.mark.parametrize("shape", [(1, 32, 8, None), (33, 96, 136, None), (300, 160, 72, None),
                                   (70, 96, 88, [0, 0, 64, 64, 65, 69])])
def test_backward_from_checkpoints(shape, fmt):
    """The backward calls on a checkpoint are the backward calls on the values
    it reads back as, bit for bit, and match the float64 evaluation there."""
    c = Case(shape, seed=11)
    codes, scales = pack(c.x, fmt)
    xq = out(c.R, c.K)
    fw.fw_moe_ckpt_unpack(fw.make_ckpt_desc(c.K, fmt), c.R, codes, scales, xq)
    (wg, wu), dy, b = [w.to(DEV) for w in c.w], c.dy.to(DEV), c.bias.to(DEV)
    got = {}
    for kind, x, s in (("none", xq, None), (fmt, codes, scales)):
        d = c.desc(fn="silu", ckpt=kind)
        ws = c.ws(d)
        dx, h, dwg, dwu = out(c.R, c.K), out(c.R, c.N), out(c.E, c.N, c.K), out(c.E, c.N, c.K)
        fw.fw_moe_glu_backward(d, c.R, x, s, wg, wu, c.offsets, dy, dx, dwg, dwu, h, ws)
        lx, lw, lb = out(c.R, c.K), out(c.E, c.N, c.K), out(c.E, c.N, dtype=F32)
        fw.fw_moe_linear_backward(d, c.R, x, s, wg, b, c.offsets, dy, lx, lw, lb, ws)
        d0 = c.desc(fn="none", ckpt=kind, grad_dtype="f32")
        lw0 = out(c.E, c.N, c.K, dtype=F32)
        fw.fw_moe_linear_backward(d0, c.R, x, s, None, None, c.offsets, dy, None, lw0, None, ws)
        got[kind] = (dx, dwg, dwu, h, lx, lw, lb, lw0)
    for p, q in zip(got["none"], got[fmt]):
        assert torch.equal(p, q)
    dx, dwg, dwu, h = got[fmt][:4]
    x64 = decoded(codes, scales, fmt)
    for e, a, z in c.segs():
        r = ref.glu_backward(x64[a:z], c.w[0][e].double(), c.w[1][e].double(),
                             c.dy[a:z].double(), "silu", BF16)
        for name, t, (want, bound) in zip(("dx", "dwg", "dwu", "h"),
                                          (dx[a:z], dwg[e], dwu[e], h[a:z]), r):
            ref.check(f"{name} expert {e}", t, want, bound)
