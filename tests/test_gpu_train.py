"""The training products as they are used together: a routed MoE layer and a
dense feed-forward block, forward and backward, with 8-bit checkpoints in
between; and the calls' behaviour in graphs, on streams, from threads, on bad
offsets, beyond 32-bit offsets, and where the tile shapes change."""

import threading

import numpy as np
import pytest
import torch

from sparse_moe_block_amd import fwmoe as fw
from . import dense_ref as ref
from .dense_ref import BF16, F32
from .test_gpu_ckpt import decoded, header, pack
from .test_gpu_dense import DEV, Case, out

pytestmark = pytest.mark.gpu


def rel(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


@pytest.mark.parametrize("ckpt", ["none", "mxfp8", "int8"])
@pytest.mark.parametrize("T", [1, 37, 300])
def test_routed_layer_step(T, ckpt):
    """Route, permute, gather, gated and down products, weighted combine; then
    the way back: both products' gradients, x and h kept as checkpoints.  Every
    result against a float64 evaluation of the same layer (at the values the
    checkpoints and the bf16 rounding of h hold).

    Tolerances (relative 2-norm).  Each bf16 rounding on a value's way is at
    most 2^-8 relative: h two (its own; g, u carry none), y one more on top of
    h's, the gradients at most dh, dg / du and their own, and in dx the sum over
    a token's experts in fp32.  A norm of such errors is below the sum of the
    bounds: 3 * 2^-8 for every output here."""
    H, F, E, k = 96, 136, 7, 3
    P = T * k
    tol = 3 * 2.0 ** -8
    g = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g)
    x = r(T, H).bfloat16()
    wg, wu = [(r(E, F, H) * H ** -0.5).bfloat16() for _ in range(2)]
    wd = (r(E, H, F) * F ** -0.5).bfloat16()
    logits = r(T, E)
    logits[:, 5] = -50.0                     # an expert nobody takes
    dout = (r(T, H) * 0.01).bfloat16()
    # routing through the layer's own entry points
    md = fw.make_desc(256, E, k, 256, act_dtype="bf16", score="softmax")
    ids, wt = out(T, k, dtype=torch.int32), out(T, k, dtype=F32)
    off, sp, inv = (out(E + 1, dtype=torch.int32), out(P, dtype=torch.int32),
                    out(P, dtype=torch.int32))
    mws = torch.empty(fw.fw_moe_workspace_size(md, T), dtype=torch.uint8, device=DEV)
    fw.fw_moe_clear_status(mws)
    fw.fw_moe_route(md, T, None, None, None, logits.to(DEV), None, ids, wt)
    fw.fw_moe_permute(md, T, ids, off, sp, inv, mws)
    token = (sp // k).long()
    xr = x.to(DEV)[token]                    # rows in expert order
    d1 = fw.make_dense_desc(H, F, n_experts=E, fn="silu", ckpt=ckpt, grad_dtype="f32")
    d2 = fw.make_dense_desc(F, H, n_experts=E, fn="none", out_dtype="f32", grad_dtype="f32")
    ws = torch.empty(max(fw.fw_moe_dense_workspace_size(d1, P),
                         fw.fw_moe_dense_workspace_size(d2, P)), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)
    fw.fw_moe_clear_status(ws)
    wg_, wu_, wd_ = wg.to(DEV), wu.to(DEV), wd.to(DEV)
    h, y = out(P, F), out(P, H, dtype=F32)
    fw.fw_moe_glu_forward(d1, P, xr, wg_, wu_, off, h, ws)
    fw.fw_moe_linear_forward(d2, P, h, wd_, None, None, off, y, ws)
    layer = (y[inv.long()].view(T, k, H) * wt[..., None]).sum(1)
    # float64
    tok, idsc, wtc = token.cpu(), ids.cpu(), wt.cpu().double()
    pair_e = idsc.reshape(-1)[sp.cpu().long()].long()
    X = x.double()[tok]
    G = torch.einsum("ph,pfh->pf", X, wg.double()[pair_e])
    U = torch.einsum("ph,pfh->pf", X, wu.double()[pair_e])
    A, _, _ = ref.act("silu", G)
    Hh = A * U
    assert rel(h, Hh) <= tol
    Y = torch.einsum("pf,phf->ph", Hh, wd.double()[pair_e])
    wp = wtc.reshape(-1)[sp.cpu().long()]
    L = torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, Y * wp[:, None])
    assert rel(layer, L) <= tol
    # backward: dy of each pair row, then both products
    dy = (dout.to(DEV)[token].float() * wt.reshape(-1)[sp.long()][:, None]).bfloat16()
    dh = out(P, F)
    d2b = fw.make_dense_desc(F, H, n_experts=E, fn="none")   # dh in bf16, as glu_backward takes it
    fw.fw_moe_linear_backward(d2b, P, None, None, wd_, None, off, dy, dh, None, None, ws)
    xs = None
    if ckpt == "none":
        xc, X2 = xr, X
    else:
        xc, xs = pack(xr.cpu(), ckpt)
        X2 = decoded(xc, xs, ckpt)
    dx, hb = out(P, H, dtype=F32), out(P, F)
    dwg, dwu, dwd = (out(E, F, H, dtype=F32), out(E, F, H, dtype=F32), out(E, H, F, dtype=F32))
    fw.fw_moe_glu_backward(d1, P, xc, xs, wg_, wu_, off, dh, dx, dwg, dwu, hb, ws)
    fw.fw_moe_linear_backward(d2, P, hb, None, None, None, off, dy, None, dwd, None, ws)
    if ckpt == "none":
        assert torch.equal(h, hb)            # h formed again has the forward's bits
    DY = dy.double().cpu()
    DH = torch.einsum("ph,phf->pf", DY, wd.double()[pair_e])
    assert rel(dh, DH) <= tol
    G = torch.einsum("ph,pfh->pf", X2, wg.double()[pair_e])
    U = torch.einsum("ph,pfh->pf", X2, wu.double()[pair_e])
    A, dA, _ = ref.act("silu", G)
    DG, DU = DH * U * dA, DH * A
    DX = (torch.einsum("pf,pfh->ph", DG, wg.double()[pair_e]) +
          torch.einsum("pf,pfh->ph", DU, wu.double()[pair_e]))
    assert rel(dx, DX) <= tol
    for got, per_row, rows in ((dwg, DG, X2), (dwu, DU, X2), (dwd, DY, A * U)):
        want = torch.zeros(got.shape, dtype=torch.float64)
        for p in range(P):
            want[pair_e[p]] += torch.outer(per_row[p], rows[p])
        assert rel(got, want) <= tol
        for e in set(range(E)) - set(pair_e.tolist()):
            assert (got[e] == 0).all()
    assert fw.fw_moe_read_status(ws) == 0 and fw.fw_moe_read_status(mws) == 0


@pytest.mark.parametrize("R", [1, 20, 200, 1000])
def test_dense_block_step(R):
    """y = x + W_d (f(x Wg^T) * (x Wu^T)) + b with the residual and bias in the
    epilogue, a gradient step through both products (the two-call chain of a
    dense feed-forward layer), against float64 autograd.  Tolerance as above,
    the residual's exact share aside."""
    H, F = 264, 200
    tol = 3 * 2.0 ** -8
    g = torch.Generator().manual_seed(R)
    r = lambda *s: torch.randn(*s, generator=g)
    x = r(R, H).bfloat16()
    wg, wu = [(r(F, H) * H ** -0.5).bfloat16() for _ in range(2)]
    wd, b = (r(H, F) * F ** -0.5).bfloat16(), r(H)
    dy = (r(R, H) * 0.01).bfloat16()
    dev = [t.to(DEV) for t in (x, wg, wu, wd, b, dy)]
    xd, wgd, wud, wdd, bd, dyd = dev
    d1 = fw.make_dense_desc(H, F, fn="gelu_tanh")
    d2 = fw.make_dense_desc(F, H, fn="none")
    ws = torch.empty(max(fw.fw_moe_dense_workspace_size(d1, R),
                         fw.fw_moe_dense_workspace_size(d2, R)), dtype=torch.uint8, device=DEV)
    fw.fw_moe_clear_status(ws)
    h, y = out(R, F), out(R, H)
    fw.fw_moe_glu_forward(d1, R, xd, wgd, wud, None, h, ws)
    fw.fw_moe_linear_forward(d2, R, h, wdd, bd, xd, None, y, ws)
    dh, dwd, db = out(R, F), out(H, F), out(H, dtype=F32)
    dx, dwg, dwu = out(R, H), out(F, H), out(F, H)
    fw.fw_moe_linear_backward(d2, R, h, None, wdd, None, None, dyd, dh, dwd, db, ws)
    fw.fw_moe_glu_backward(d1, R, xd, None, wgd, wud, None, dh, dx, dwg, dwu, None, ws)
    t = [v.double().requires_grad_() for v in (x, wg, wu, wd, b)]
    X, Wg, Wu, Wd, B = t
    Y = ref.act("gelu_tanh", X @ Wg.T)[0] * (X @ Wu.T) @ Wd.T + B
    assert rel(y, (Y + X).detach()) <= tol
    grads = torch.autograd.grad(Y, t, dy.double())
    for name, got, want in zip(("dx", "dwg", "dwu", "dwd", "db"), (dx, dwg, dwu, dwd, db), grads):
        assert rel(got, want) <= tol, name


def step_calls(c, fmt, stream=None):
    """One training step of both products on c's inputs: buffers, and a call that
    runs it into them."""
    codes, scales = pack(c.x, fmt)
    (wg, wu), dy, b = [w.to(DEV) for w in c.w], c.dy.to(DEV), c.bias.to(DEV)
    x = c.x.to(DEV)
    d = c.desc(fn="silu", ckpt=fmt)
    ws = c.ws(d)
    o = dict(h=out(c.R, c.N), y=out(c.R, c.N), dx=out(c.R, c.K), dwg=out(c.E, c.N, c.K),
             dwu=out(c.E, c.N, c.K), h2=out(c.R, c.N), lx=out(c.R, c.K), lw=out(c.E, c.N, c.K),
             lb=out(c.E, c.N, dtype=F32), xq=out(c.R, c.K))
    cd = fw.make_ckpt_desc(c.K, fmt)
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)

    def run(s=None):
        fw.fw_moe_glu_forward(d, c.R, x, wg, wu, c.offsets, o["h"], ws, stream=s)
        fw.fw_moe_linear_forward(d, c.R, x, wg, b, None, c.offsets, o["y"], ws, stream=s)
        fw.fw_moe_ckpt_pack(cd, c.R, x, c2, s2, ws, stream=s)
        fw.fw_moe_ckpt_unpack(cd, c.R, c2, s2, o["xq"], stream=s)
        fw.fw_moe_glu_backward(d, c.R, c2, s2, wg, wu, c.offsets, dy, o["dx"], o["dwg"], o["dwu"],
                               o["h2"], ws, stream=s)
        fw.fw_moe_linear_backward(d, c.R, c2, s2, wg, b, c.offsets, dy, o["lx"], o["lw"], o["lb"],
                                  ws, stream=s)
    return o, ws, run, (x, dy)


SHAPES = [(1, 64, 136, None), (300, 160, 264, None), (777, 96, 136, None),
          (70, 96, 88, [0, 0, 64, 64, 65, 69]), (520, 160, 72, [0, 1, 259, 259, 400, 519])]


@pytest.mark.parametrize("shape", SHAPES)
def test_graph_replays_equal_eager(shape):
    """A whole step captured once and replayed on new inputs in the same buffers,
    with eager steps of another workspace and synchronisations in between."""
    c, other = Case(shape, seed=21), Case(shape, seed=22)
    o, ws, run, (x, dy) = step_calls(c, "int8")
    eo, _, erun, (ex, edy) = step_calls(other, "int8")
    run(), erun()
    torch.cuda.synchronize()
    first, second = {k: v.clone() for k, v in o.items()}, {k: v.clone() for k, v in eo.items()}
    # the graph's weights are c's: the second set of expectations needs them too
    x0, dy0 = x.clone(), dy.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(torch.cuda.current_stream())
    x.copy_(ex), dy.copy_(edy)
    run()
    torch.cuda.synchronize()
    swapped = {k: v.clone() for k, v in o.items()}
    for rep in range(3):
        for src, want in (((x0, dy0), first), ((ex, edy), swapped)):
            x.copy_(src[0]), dy.copy_(src[1])
            for v in o.values():
                v[:c.end if v.shape[0] == c.R else None].fill_(7.0)
            erun()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for k, v in o.items():
                n = c.end if v.shape[0] == c.R and k != "xq" else v.shape[0]
                assert torch.equal(v[:n], want[k][:n]), f"replay {rep}: {k}"
            for k, v in eo.items():
                assert torch.equal(v, second[k])
    assert fw.fw_moe_read_status(ws) == 0


def test_two_threads_on_their_own_streams():
    """Two host threads, each with its stream, workspace and buffers, at the same
    time: the serial results bit for bit."""
    cases = [Case((300, 160, 264, None), seed=31), Case((520, 160, 72, [0, 1, 259, 259, 400, 519]),
                                                         seed=32)]
    steps = [step_calls(c, f) for c, f in zip(cases, ("mxfp8", "int8"))]
    want = []
    for o, _, run, _ in steps:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in o.items()})
    streams = [torch.cuda.Stream() for _ in steps]
    got, errors, start = [[], []], [], threading.Barrier(2)

    def worker(i):
        try:
            start.wait()
            for _ in range(10):
                steps[i][2](streams[i])
                with torch.cuda.stream(streams[i]):
                    got[i].append({k: v.clone() for k, v in steps[i][0].items()})
        except Exception as e:   # reported below, in the main thread
            errors.append(e)
    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i in range(2):
        for r in got[i]:
            for k, v in r.items():
                assert torch.equal(v, want[i][k]), k


@pytest.mark.parametrize("offsets", [[0, 40, 20, 64], [5, 20, 40, 64], [0, 30, 90, 64],
                                     [0, -3, 20, 64], [0, 64, 0, 64], [2 ** 31 - 1, -2 ** 31, 7, 1]])
@pytest.mark.parametrize("R,K", [(64, 96), (1000, 96)])
def test_bad_offsets_are_reported(offsets, R, K):
    """Offsets that do not ascend from 0 within the rows: FW_STATUS_BAD_OFFSETS
    (sticky) from every product, nothing written outside the buffers (guards on
    both sides of each).  Every segment the kernels use is clamped to [0, R], the
    tile list to the workspace's room."""
    E, N, G = 3, 72, 4096
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    d = fw.make_dense_desc(K, N, n_experts=E, fn="silu")

    def guarded(n, dtype=BF16):
        buf = torch.full((n + 2 * G,), 3.0, dtype=dtype, device=DEV)
        return buf, buf[G:G + n]
    x = torch.ones(R, K, dtype=BF16, device=DEV)
    dy = torch.ones(R, N, dtype=BF16, device=DEV)
    w = torch.full((E, N, K), 0.01, dtype=BF16, device=DEV)
    need = fw.fw_moe_dense_workspace_size(d, R)
    wbuf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    ws = wbuf[256:256 + need]
    bufs = [guarded(n) for n in (R * N, R * N, R * K, E * N * K, E * N * K, R * N, R * K, E * N * K)]
    bufs.append(guarded(E * N, F32))
    h, y, dx, dwg, dwu, h2, lx, lw, lb = [b[1] for b in bufs]
    for call in (lambda: fw.fw_moe_glu_forward(d, R, x, w, w, off, h, ws),
                 lambda: fw.fw_moe_linear_forward(d, R, x, w, None, None, off, y, ws),
                 lambda: fw.fw_moe_glu_backward(d, R, x, None, w, w, off, dy, dx, dwg, dwu, h2, ws),
                 lambda: fw.fw_moe_linear_backward(d, R, x, None, w, None, off, dy, lx, lw, lb, ws)):
        fw.fw_moe_clear_status(ws)
        call()
        assert fw.fw_moe_read_status(ws) == fw.FW_STATUS_BAD_OFFSETS
    for buf, _ in bufs:
        assert (buf[:G] == 3).all() and (buf[-G:] == 3).all()
    assert (wbuf[:256] == 0x5A).all() and (wbuf[-256:] == 0x5A).all()


def test_rows_beyond_32_bit_offsets():
    """x and y of more than 2^32 bytes (and 2^31 elements): rows at both ends and
    in the middle, and the weight gradient over all of the rows."""
    R, K, N = 1 << 20, 2304, 2304
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(R, K, dtype=BF16, device=DEV)
    for i in range(0, R, 1 << 17):
        x[i:i + (1 << 17)] = torch.randn(1 << 17, K, generator=g, device=DEV)
    w = (torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).bfloat16()
    assert R * K > 2 ** 31
    d = fw.make_dense_desc(K, N, fn="none", grad_dtype="f32")
    ws = torch.empty(fw.fw_moe_dense_workspace_size(d, R), dtype=torch.uint8, device=DEV)
    fw.fw_moe_clear_status(ws)
    y = out(R, N)
    fw.fw_moe_linear_forward(d, R, x, w, None, None, None, y, ws)
    rows = torch.tensor([0, 1, 931_000, 932_067, 932_068, R // 2, R - 257, R - 1], device=DEV)
    want, bound = ref.linear_forward(x[rows].double().cpu(), w.double().cpu(), None, None, "none",
                                     BF16)
    ref.check("y", y[rows], want, bound)
    # dx as large, and dw with only far rows' gradients set: their sum alone
    dy = y
    dy.zero_()
    dy[rows] = torch.randn(8, N, generator=g, device=DEV).bfloat16()
    dx, dw = torch.empty(R, K, device=DEV), torch.empty(N, K, device=DEV)
    fw.fw_moe_linear_backward(d, R, x, None, w, None, None, dy, dx, dw, None, ws)
    (want, bound), (wantw, boundw), _ = ref.linear_backward(
        x[rows].double().cpu(), w.double().cpu(), None, dy[rows].double().cpu(), "none", F32)
    ref.check("dx", dx[rows], want, bound)
    ref.check("dw", dw, wantw, boundw)
    assert torch.equal(dx[rows[-1] - 3], torch.zeros(K, device=DEV))
    # a checkpoint of them
    c = torch.empty(R, K, dtype=torch.int8, device=DEV)
    s = torch.empty(R, K // 32, device=DEV)
    cd = fw.make_ckpt_desc(K, "int8")
    fw.fw_moe_ckpt_pack(cd, R, x, c, s, header())
    fw.fw_moe_ckpt_unpack(cd, R, c, s, y)
    c1, s1 = pack(x[rows].cpu(), "int8")
    assert torch.equal(c[rows], c1) and torch.equal(s[rows], s1)
    assert torch.equal(y[rows].double().cpu(), decoded(c1, s1, "int8"))


def test_experts_beyond_32_bit_offsets():
    """Weights and weight gradients of more than 2^31 elements: the last expert's
    rows, forward (few rows, and tiles) and backward."""
    E, N, K = 300, 2048, 4096
    g = torch.Generator(device=DEV).manual_seed(2)
    w = torch.zeros(E, N, K, dtype=BF16, device=DEV)
    assert w.numel() > 2 ** 31
    for e in (0, 150, E - 1):
        w[e] = (torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).bfloat16()
    for rows in ({0: 3, 150: 2, E - 1: 4}, {0: 3, 150: 300, E - 1: 2400}):
        ends = np.cumsum([0] + [rows.get(e, 0) for e in range(E)]).astype(np.int32)
        R = int(ends[-1])
        off = torch.from_numpy(ends).to(DEV)
        x = torch.randn(R, K, generator=g, device=DEV).bfloat16()
        dy = (torch.randn(R, N, generator=g, device=DEV) * 0.01).bfloat16()
        d = fw.make_dense_desc(K, N, n_experts=E, fn="none")
        ws = torch.empty(fw.fw_moe_dense_workspace_size(d, R), dtype=torch.uint8, device=DEV)
        fw.fw_moe_clear_status(ws)
        y, dx = out(R, N), out(R, K)
        dw = torch.empty(E, N, K, dtype=BF16, device=DEV)
        fw.fw_moe_linear_forward(d, R, x, w, None, None, off, y, ws)
        fw.fw_moe_linear_backward(d, R, x, None, w, None, off, dy, dx, dw, None, ws)
        for e, n in rows.items():
            a = int(ends[e])
            pick = slice(a, a + min(n, 5))
            W = w[e].double().cpu()
            want, bound = ref.linear_forward(x[pick].double().cpu(), W, None, None, "none", BF16)
            ref.check(f"y expert {e}", y[pick], want, bound)
            want, err = ref.dot(dy[pick].double().cpu(), W)
            ref.check(f"dx expert {e}", dx[pick], want, ref.rounded(want, err, BF16))
            cols = slice(0, 16)
            want, err = ref.dot(dy[a:a + n, cols].double().cpu().T, x[a:a + n].double().cpu())
            ref.check(f"dw expert {e}", dw[e, cols], want, ref.rounded(want, err, BF16))
        for e in (1, 149, 151, E - 2):
            assert not dw[e].any()
        assert fw.fw_moe_read_status(ws) == 0
        del dw


# One size on either side of every choice of a kernel or tile shape: few rows and
# tiles, each row-product shape, each shape of the joint backward launch, weight
# gradients by expert in each shape, gradients stored past the caches (> 256 MB).
CHOICES = [(16, 512, 264, 1), (17, 512, 264, 1), (32, 4096, 72, 1), (33, 4096, 72, 1),
           (64, 264, 136, 8), (65, 264, 136, 8), (512, 264, 136, 8), (511, 264, 136, 8),
           (2048, 264, 136, 8), (2050, 264, 520, 8), (2047, 72, 520, 8), (300, 264, 4104, 1),
           (1500, 264, 4104, 1), (4100, 72, 4104, 1), (2100, 1032, 8200, 1), (5000, 520, 520, 1),
           (100, 1032, 1032, 64), (40, 2056, 4104, 16), (777, 1536, 4096, 1), (1100, 2048, 264, 1),
           (1300, 264, 4104, 1), (6000, 2048, 2056, 8), (2000, 2048, 2056, 12),
           (1100, 2048, 1032, 4), (4100, 2056, 2048, 1), (2048, 4104, 4096, 1)]


@pytest.mark.parametrize("R,K,N,E", CHOICES)
def test_tile_choices(R, K, N, E):
    g = torch.Generator().manual_seed(R + K + N)
    cuts = sorted(torch.randint(0, R + 1, (E - 1,), generator=g).tolist())
    off = None if E == 1 else [0] + cuts + [R]
    c = Case((R, K, N, off), seed=41)
    d = c.desc(fn="silu", grad_dtype="bf16")
    ws = c.ws(d)
    x, (wg, wu), dy, b = c.x.to(DEV), [w.to(DEV) for w in c.w], c.dy.to(DEV), c.bias.to(DEV)
    h, y, dx, h2 = out(R, N), out(R, N), out(R, K), out(R, N)
    dwg, dwu, lx, lw = (out(E, N, K), out(E, N, K), out(R, K), out(E, N, K))
    lb = out(E, N, dtype=F32)
    fw.fw_moe_glu_forward(d, R, x, wg, wu, c.offsets, h, ws)
    fw.fw_moe_linear_forward(d, R, x, wg, b, None, c.offsets, y, ws)
    fw.fw_moe_glu_backward(d, R, x, None, wg, wu, c.offsets, dy, dx, dwg, dwu, h2, ws)
    fw.fw_moe_linear_backward(d, R, x, None, wg, b, c.offsets, dy, lx, lw, lb, ws)
    for e, a, z in c.segs():
        X, D = c.x[a:z].to(DEV).double(), c.dy[a:z].to(DEV).double()
        Wg, Wu, B = wg[e].double(), wu[e].double(), b[e].double()
        checks = [("h", h[a:z]) + ref.glu_forward(X, Wg, Wu, "silu", BF16),
                  ("y", y[a:z]) + ref.linear_forward(X, Wg, B, None, "silu", BF16)]
        checks += [(n, t) + wb for n, t, wb in zip(
            ("dx", "dwg", "dwu", "h2"), (dx[a:z], dwg[e], dwu[e], h2[a:z]),
            ref.glu_backward(X, Wg, Wu, D, "silu", BF16))]
        checks += [(n, t) + wb for n, t, wb in zip(
            ("lx", "lw", "lb"), (lx[a:z], lw[e], lb[e]),
            ref.linear_backward(X, Wg, B, D, "silu", BF16))]
        for name, got, want, bound in checks:
            if got.numel():
                ref.check(f"{name} expert {e}", got, want.cpu(), bound.cpu())
    # dx and dw by launches of their own, in the tile shapes that those take: the
    # sums run over the reduction in the same order, so the same bits
    dx2, dwg2, dwu2, lx2, lw2 = (torch.full_like(t, 9.0) for t in (dx, dwg, dwu, lx, lw))
    fw.fw_moe_glu_backward(d, R, x, None, wg, wu, c.offsets, dy, dx2, None, None, None, ws)
    fw.fw_moe_glu_backward(d, R, x, None, wg, wu, c.offsets, dy, None, dwg2, dwu2, None, ws)
    fw.fw_moe_linear_backward(d, R, x, None, wg, b, c.offsets, dy, lx2, None, None, ws)
    fw.fw_moe_linear_backward(d, R, x, None, wg, b, c.offsets, dy, None, lw2, None, ws)
    for p, q in ((dx, dx2), (dwg, dwg2), (dwu, dwu2), (lx, lx2), (lw, lw2)):
        assert torch.equal(p, q)
    assert fw.fw_moe_read_status(ws) == 0


# The last tile of dw has columns in one half of a lane's values only (8 to 32 of
# 64) or in both; each tile shape, and gradients stored past the caches.
@pytest.mark.parametrize("R,K,N,E", [(5, 8, 8, 1), (70, 40, 72, 3), (130, 104, 136, 1),
                                     (300, 232, 264, 2), (600, 1000, 1096, 1),
                                     (900, 2024, 2088, 1), (1024, 4128, 4104, 1),
                                     (200, 1064, 1032, 70), (100, 4104, 2088, 8)])
def test_weight_gradient_types(R, K, N, E):
    """fp32 weight gradients against the formula, the bf16 ones as their rounding,
    and accumulation as the sum of both."""
    g = torch.Generator().manual_seed(R + K + N)
    cuts = sorted(torch.randint(0, R + 1, (E - 1,), generator=g).tolist())
    c = Case((R, K, N, None if E == 1 else [0] + cuts + [R]), seed=43)
    d32, d16 = c.desc(fn="none", grad_dtype="f32"), c.desc(fn="none", grad_dtype="bf16")
    acc = c.desc(fn="none", grad_dtype="f32", accumulate=True)
    ws = c.ws(d32)
    x, w, dy = c.x.to(DEV), c.w[0].to(DEV), c.dy.to(DEV)
    for dx in (None, out(R, K, dtype=F32)):   # by itself, and joint with dx
        dx16 = None if dx is None else out(R, K)
        dw, low = out(E, N, K, dtype=F32), out(E, N, K)
        start = torch.randn(E, N, K, device=DEV)
        total = start.clone()
        for d, a, b in ((d32, dx, dw), (d16, dx16, low), (acc, dx, total)):
            fw.fw_moe_linear_backward(d, R, x, None, w, None, c.offsets, dy, a, b, None, ws)
        for e, a, z in c.segs():
            want, bound = ref.linear_backward(x[a:z].double(), w[e].double(), None,
                                              dy[a:z].double(), "none", F32)[1]
            ref.check(f"dw expert {e}", dw[e], want.cpu(), bound.cpu())
        assert torch.equal(dw.to(BF16), low)
        assert torch.equal(total, start + dw)
    assert fw.fw_moe_read_status(ws) == 0
