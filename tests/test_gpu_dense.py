"""The training products (fw_moe_glu_*, fw_moe_linear_*) against a float64
evaluation, element by element within bounds derived from the kernels' own
roundings (dense_ref)."""

import pytest
import torch

from sparse_moe_block_amd import fwmoe as fw
from . import dense_ref as ref
from .dense_ref import BF16, F32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": BF16, "f32": F32}
SENTINEL = 123.0

# (rows, in, out, offsets or None): odd row counts, feature counts that end
# inside a tile, a 64-step stage, a 16-byte chunk; experts without rows, one
# expert with all of them, rows behind the last expert's
SHAPES = [
    (1, 8, 8, None), (1, 264, 136, None), (3, 72, 24, None), (16, 64, 128, None),
    (17, 200, 264, None), (33, 520, 40, None), (64, 1032, 72, None), (127, 96, 392, None),
    (128, 128, 128, None), (129, 64, 520, None), (257, 328, 200, None), (300, 136, 1032, None),
    (5, 64, 136, [0, 3]), (200, 96, 136, [0, 131, 200]), (70, 72, 88, [0, 0, 64, 64, 65, 69]),
    (20, 4104, 40, None), (31, 4128, 24, [0, 29]), (777, 72, 1032, None), (1400, 40, 136, [0, 700, 700, 1390]), (9, 264, 40, [0, 1, 2, 3, 4, 5, 6, 7, 8, 9]), (40, 40, 64, [0, 0, 0, 0]),
    (520, 136, 72, [0, 1, 259, 259, 400, 519]), (300, 64, 24, [0, 0, 300, 300]),
    (60, 296, 40, [0, 33, 33, 34, 34, 34, 34, 34, 51, 59]),
]
IDS = [f"{r}x{k}x{n}" + ("" if o is None else f"e{len(o) - 1}") for r, k, n, o in SHAPES]


class Case:
    def __init__(self, shape, seed=0, std=1.0):
        self.R, self.K, self.N, off = shape
        self.E = 1 if off is None else len(off) - 1
        self.off = off
        g = torch.Generator().manual_seed(1000 * seed + 7 * self.R + self.K + 3 * self.N)
        r = lambda *s: torch.randn(*s, generator=g)
        self.x = (r(self.R, self.K) * std).bfloat16()
        self.w = [(r(self.E, self.N, self.K) * self.K ** -0.5).bfloat16() for _ in range(2)]
        self.bias = r(self.E, self.N)
        self.dy = (r(self.R, self.N) * 0.01).bfloat16()
        self.res = r(self.R, self.N)
        self.offsets = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
        self.end = self.R if off is None else off[-1]

    def desc(self, **kw):
        return fw.make_dense_desc(self.K, self.N, n_experts=self.E, **kw)

    def ws(self, desc):
        ws = torch.empty(fw.fw_moe_dense_workspace_size(desc, self.R), dtype=torch.uint8,
                         device=DEV)
        ws.fill_(0xFF)   # whatever a workspace held before must not matter (all NaN)
        fw.fw_moe_clear_status(ws)
        return ws

    def segs(self):
        return ref.segments(self.off, self.R, self.E)


def out(*shape, dtype=BF16):
    return torch.full(shape, SENTINEL, dtype=dtype, device=DEV)


def behind(c, *tensors):
    """Rows behind the last expert's are left as they were."""
    for t in tensors:
        assert (t[c.end:] == SENTINEL).all()


def check_rows(c, name, got, per_segment):
    for e, a, b in c.segs():
        if b > a:
            want, bound = per_segment(e, a, b)
            ref.check(f"{name} expert {e}", got[a:b], want, bound)


@pytest.mark.parametrize("fn,out_dtype", [("silu", "bf16"), ("gelu_tanh", "f32")])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_glu_forward(shape, fn, out_dtype):
    c = Case(shape)
    d = c.desc(fn=fn, out_dtype=out_dtype)
    ws, h = c.ws(d), out(c.R, c.N, dtype=DT[out_dtype])
    x, (wg, wu) = c.x.to(DEV), [w.to(DEV) for w in c.w]
    fw.fw_moe_glu_forward(d, c.R, x, wg, wu, c.offsets, h, ws)
    check_rows(c, "h", h, lambda e, a, b: ref.glu_forward(
        c.x[a:b].double(), c.w[0][e].double(), c.w[1][e].double(), fn, DT[out_dtype]))
    behind(c, h)
    assert fw.fw_moe_read_status(ws) == 0


@pytest.mark.parametrize("fn,grad", [("silu", "bf16"), ("gelu_tanh", "f32"), ("relu", "bf16")])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_glu_backward(shape, fn, grad):
    c = Case(shape, seed=1)
    d = c.desc(fn=fn, grad_dtype=grad)
    ws, gd = c.ws(d), DT[grad]
    x, (wg, wu), dh = c.x.to(DEV), [w.to(DEV) for w in c.w], c.dy.to(DEV)
    dx, h = out(c.R, c.K, dtype=gd), out(c.R, c.N)
    dwg, dwu = out(c.E, c.N, c.K, dtype=gd), out(c.E, c.N, c.K, dtype=gd)
    fw.fw_moe_glu_backward(d, c.R, x, None, wg, wu, c.offsets, dh, dx, dwg, dwu, h, ws)
    for e, a, b in c.segs():
        r = ref.glu_backward(c.x[a:b].double(), c.w[0][e].double(), c.w[1][e].double(),
                             c.dy[a:b].double(), fn, gd)
        for name, got, (want, bound) in zip(("dx", "dwg", "dwu", "h"),
                                            (dx[a:b], dwg[e], dwu[e], h[a:b]), r):
            ref.check(f"{name} expert {e}", got, want, bound)
    behind(c, dx, h)
    assert fw.fw_moe_read_status(ws) == 0
    # the same call again, and each output by itself: the same bits
    dx2, h2, dg2, du2 = (torch.full_like(t, SENTINEL) for t in (dx, h, dwg, dwu))
    call = lambda *o: fw.fw_moe_glu_backward(d, c.R, x, None, wg, wu, c.offsets, dh, *o, ws)
    call(dx2, None, None, None)
    call(None, dg2, du2, None)
    call(None, None, None, h2)
    for p, q in ((dx, dx2), (h, h2), (dwg, dg2), (dwu, du2)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("fn,out_dtype,bias,residual", [
    ("none", "bf16", True, True), ("gelu_tanh", "f32", True, True), ("silu", "bf16", False, True),
    ("relu", "f32", True, False), ("none", "f32", False, False)])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear_forward(shape, fn, out_dtype, bias, residual):
    c = Case(shape, seed=2)
    dt = DT[out_dtype]
    d = c.desc(fn=fn, out_dtype=out_dtype)
    ws, y = c.ws(d), out(c.R, c.N, dtype=dt)
    res = c.res.to(dt) if residual else None
    x, w = c.x.to(DEV), c.w[0].to(DEV)
    b, r = c.bias.to(DEV) if bias else None, res.to(DEV) if residual else None
    fw.fw_moe_linear_forward(d, c.R, x, w, b, r, c.offsets, y, ws)
    check_rows(c, "y", y, lambda e, a, z: ref.linear_forward(
        c.x[a:z].double(), c.w[0][e].double(), c.bias[e].double() if bias else None,
        res[a:z].double() if residual else None, fn, dt))
    behind(c, y)
    if residual:   # y may be the residual itself
        fw.fw_moe_linear_forward(d, c.R, x, w, b, r, c.offsets, r, ws)
        assert torch.equal(r[:c.end], y[:c.end])
    assert fw.fw_moe_read_status(ws) == 0


@pytest.mark.parametrize("fn,grad,bias", [("none", "f32", True), ("none", "bf16", False),
                                          ("silu", "bf16", True), ("gelu_tanh", "f32", True),
                                          ("relu", "bf16", False)])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear_backward(shape, fn, grad, bias):
    c = Case(shape, seed=3)
    gd = DT[grad]
    d = c.desc(fn=fn, grad_dtype=grad)
    ws = c.ws(d)
    x, w, dy = c.x.to(DEV), c.w[0].to(DEV), c.dy.to(DEV)
    b = c.bias.to(DEV) if bias else None
    dx, dw = out(c.R, c.K, dtype=gd), out(c.E, c.N, c.K, dtype=gd)
    db = out(c.E, c.N, dtype=F32) if bias else None
    fw.fw_moe_linear_backward(d, c.R, x, None, w, b, c.offsets, dy, dx, dw, db, ws)
    for e, a, z in c.segs():
        r = ref.linear_backward(c.x[a:z].double(), c.w[0][e].double(),
                                c.bias[e].double() if bias else None, c.dy[a:z].double(), fn, gd)
        got = [dx[a:z], dw[e]] + ([db[e]] if bias else [])
        for name, t, (want, bound) in zip(("dx", "dw", "db"), got, r):
            ref.check(f"{name} expert {e}", t, want, bound)
    behind(c, dx)
    assert fw.fw_moe_read_status(ws) == 0
    # each output by itself: the same bits; without an activation dx needs no x and
    # dw no w
    call = lambda *o: fw.fw_moe_linear_backward(d, c.R, *o, ws)
    dx2, dw2 = torch.full_like(dx, SENTINEL), torch.full_like(dw, SENTINEL)
    need = fn != "none"
    call(x if need else None, None, w, b, c.offsets, dy, dx2, None, None)
    call(x, None, w if need else None, b, c.offsets, dy, None, dw2, None)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    if bias:
        db2 = torch.full_like(db, SENTINEL)
        call(x if need else None, None, w if need else None, b, c.offsets, dy, None, None, db2)
        assert torch.equal(db, db2)


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(40, 72, 136, None), (70, 72, 88, [0, 0, 64, 64, 65, 69])])
def test_accumulate(shape, grad):
    """accumulate adds to the weight and bias gradients (not to dx): one more
    rounding of the sum in the gradients' type."""
    c = Case(shape, seed=4)
    gd = DT[grad]
    d, d1 = c.desc(fn="silu", grad_dtype=grad), c.desc(fn="silu", grad_dtype=grad, accumulate=True)
    ws = c.ws(d)
    x, (w, wu), dy, b = c.x.to(DEV), [t.to(DEV) for t in c.w], c.dy.to(DEV), c.bias.to(DEV)
    g = torch.Generator().manual_seed(5)
    start = (torch.randn(c.E, c.N, c.K, generator=g) * 0.05).to(gd)
    bstart = torch.randn(c.E, c.N, generator=g) * 0.05
    dx, dx1 = out(c.R, c.K, dtype=gd), out(c.R, c.K, dtype=gd)
    # f32 gradients show the sum before a bf16 rounding
    exact = out(c.E, c.N, c.K, dtype=F32)
    db, db1 = out(c.E, c.N, dtype=F32), bstart.to(DEV)
    dw1 = start.to(DEV)
    fw.fw_moe_linear_backward(c.desc(fn="silu", grad_dtype="f32"), c.R, x, None, w, b, c.offsets,
                              dy, None, exact, db, ws)
    fw.fw_moe_linear_backward(d1, c.R, x, None, w, b, c.offsets, dy, dx1, dw1, db1, ws)
    fw.fw_moe_linear_backward(d, c.R, x, None, w, b, c.offsets, dy, dx, None, None, ws)
    assert torch.equal(dx[:c.end], dx1[:c.end])
    want = exact.double().cpu() + start.double()
    slack = 2.0 ** -22 * (exact.double().cpu().abs() + start.double().abs())
    ref.check("dw", dw1, want, ref.rounded(want, slack, gd))
    wb = db.double().cpu() + bstart.double()
    ref.check("db", db1, wb, 2.0 ** -22 * (db.double().cpu().abs() + bstart.double().abs()))
    dwg, dwu = start.to(DEV), start.to(DEV)
    eg, eu = out(c.E, c.N, c.K, dtype=F32), out(c.E, c.N, c.K, dtype=F32)
    fw.fw_moe_glu_backward(c.desc(fn="silu", grad_dtype="f32"), c.R, x, None, w, wu, c.offsets,
                           dy, None, eg, eu, None, ws)
    fw.fw_moe_glu_backward(d1, c.R, x, None, w, wu, c.offsets, dy, None, dwg, dwu, None, ws)
    for got, ex in ((dwg, eg), (dwu, eu)):
        want = ex.double().cpu() + start.double()
        slack = 2.0 ** -22 * (ex.double().cpu().abs() + start.double().abs())
        ref.check("dw", got, want, ref.rounded(want, slack, gd))


@pytest.mark.parametrize("offsets", [None, [0, 0, 0, 0]])
def test_no_rows(offsets):
    """R = 0: weight and bias gradients are zeros, or unchanged with accumulate;
    nothing else is written."""
    K, N, E = 72, 136, 1 if offsets is None else len(offsets) - 1
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    w = torch.ones(E, N, K, dtype=BF16, device=DEV)
    for acc in (False, True):
        d = fw.make_dense_desc(K, N, n_experts=E, fn="silu", accumulate=acc)
        ws = torch.empty(fw.fw_moe_dense_workspace_size(d, 0), dtype=torch.uint8, device=DEV)
        fw.fw_moe_clear_status(ws)
        none = torch.empty(0, K, dtype=BF16, device=DEV)
        empty = torch.empty(0, N, dtype=BF16, device=DEV)
        a, b, e, db = (out(E, N, K), out(E, N, K), out(E, N, K), out(E, N, dtype=F32))
        fw.fw_moe_glu_forward(d, 0, none, w, w, off, empty, ws)
        fw.fw_moe_linear_forward(d, 0, none, w, None, None, off, empty, ws)
        fw.fw_moe_glu_backward(d, 0, none, None, w, w, off, empty, none, a, b, empty, ws)
        fw.fw_moe_linear_backward(d, 0, none, None, w, None, off, empty, none, e, db, ws)
        want = SENTINEL if acc else 0.0
        for t in (a, b, e, db):
            assert (t == want).all()
        assert fw.fw_moe_read_status(ws) == 0


def test_non_finite_values_stay_in_their_rows():
    """A NaN or infinite row of x, or a non-finite arriving gradient, reaches
    its own rows of h, y and dx and the weight gradients of its own expert, and
    nothing else -- also where the row shares a tile or a stage with others."""
    R, K, N, off = 200, 72, 136, [0, 70, 130, 200]
    c = Case((R, K, N, off), seed=6)
    c.x[75, 3], c.x[100, 71] = float("nan"), float("inf")
    d = c.desc(fn="silu")
    ws = c.ws(d)
    x, (wg, wu), dy = c.x.to(DEV), [w.to(DEV) for w in c.w], c.dy.to(DEV)
    h, y, dx = out(R, N), out(R, N), out(R, K)
    dwg, dwu, dw = out(3, N, K), out(3, N, K), out(3, N, K)
    fw.fw_moe_glu_forward(d, R, x, wg, wu, c.offsets, h, ws)
    fw.fw_moe_linear_forward(d, R, x, wg, None, None, c.offsets, y, ws)
    bad = torch.zeros(R, dtype=torch.bool, device=DEV)
    bad[[75, 100]] = True
    for t in (h, y):
        assert torch.isfinite(t[~bad]).all() and not torch.isfinite(t[75]).any()
        assert not torch.isfinite(t[100]).all()
    fw.fw_moe_glu_backward(d, R, x, None, wg, wu, c.offsets, dy, dx, dwg, dwu, None, ws)
    fw.fw_moe_linear_backward(d, R, x, None, wg, None, c.offsets, dy, None, dw, None, ws)
    assert torch.isfinite(dx[~bad]).all() and not torch.isfinite(dx[bad]).any()
    for t in (dwg, dwu, dw):
        assert torch.isfinite(t[0]).all() and torch.isfinite(t[2]).all()
        assert not torch.isfinite(t[1]).any()
    # an infinite gradient of one row
    dy2 = c.dy.clone()
    dy2[131, 5] = float("inf")
    x2 = Case((R, K, N, off), seed=6).x.to(DEV)
    fw.fw_moe_glu_backward(d, R, x2, None, wg, wu, c.offsets, dy2.to(DEV), dx, dwg, dwu, None, ws)
    row = torch.arange(R, device=DEV) == 131
    assert torch.isfinite(dx[~row]).all() and not torch.isfinite(dx[row]).any()
    for t in (dwg, dwu):
        assert torch.isfinite(t[:2]).all() and not torch.isfinite(t[2, 5]).any()
        assert torch.isfinite(t[2, :5]).all() and torch.isfinite(t[2, 6:]).all()


@pytest.mark.parametrize("fn", ["silu", "gelu_tanh", "relu", "none"])
def test_large_pre_activations(fn):
    """f and f' at arguments from -3e4 to 3e4: the limits, no NaN from inf * 0."""
    K = N = 64
    vals = torch.tensor([0.0, 1e-3, -1e-3, 1.0, -1.0, 10.0, -10.0, 30.0, -30.0, 89.0, -89.0, 104.0,
                         -104.0, 3e4, -3e4, -0.0])
    x = torch.zeros(16, K)
    x[:, 0] = vals
    x = x.bfloat16()
    w = torch.zeros(N, K)
    w[:, 0] = 1.0
    w = w.bfloat16()
    dy = torch.ones(16, N).bfloat16()
    d = fw.make_dense_desc(K, N, fn=fn, out_dtype="f32", grad_dtype="f32")
    ws = torch.empty(fw.fw_moe_dense_workspace_size(d, 16), dtype=torch.uint8, device=DEV)
    fw.fw_moe_clear_status(ws)
    y, db = out(16, N, dtype=F32), out(1, N, dtype=F32)
    fw.fw_moe_linear_forward(d, 16, x.to(DEV), w.to(DEV), None, None, None, y, ws)
    want, bound = ref.linear_forward(x.double(), w.double(), None, None, fn, F32)
    ref.check("y", y, want, bound)
    dx = out(16, K, dtype=F32)
    fw.fw_moe_linear_backward(d, 16, x.to(DEV), None, w.to(DEV), None, None, dy.to(DEV), dx, None,
                              db, ws)
    (want, bound), _, (wb, bb) = ref.linear_backward(x.double(), w.double(), None, dy.double(), fn,
                                                     F32)
    ref.check("dx", dx, want, bound)
    ref.check("db", db[0], wb, bb)


def test_gradients_match_differences():
    """Central differences of the forward calls' sums (f32 outputs) against the
    backward calls.  The difference quotient of L = sum(dy * out) along a
    direction v is off by its third-derivative term and by the forward's
    rounding over the step; both are bounded by the comparison with a float64
    quotient of the same step, so only the calls' own errors remain."""
    c = Case((24, 72, 40, None), seed=8)
    d = c.desc(fn="silu", out_dtype="f32", grad_dtype="f32")
    ws = c.ws(d)
    x, (wg, wu), dy = c.x.to(DEV), [w.to(DEV) for w in c.w], c.dy.to(DEV)
    dx, dwg, dwu = (out(c.R, c.K, dtype=F32), out(c.E, c.N, c.K, dtype=F32),
                    out(c.E, c.N, c.K, dtype=F32))
    fw.fw_moe_glu_backward(d, c.R, x, None, wg, wu, None, dy, dx, dwg, dwu, None, ws)
    g = torch.Generator().manual_seed(9)

    def loss(x_, wg_, wu_):
        h = out(c.R, c.N, dtype=F32)
        fw.fw_moe_glu_forward(d, c.R, x_, wg_, wu_, None, h, ws)
        return (h.double() * dy.double()).sum().item()

    for which, grad in ((0, dx), (1, dwg), (2, dwu)):
        args = [x, wg, wu]
        v = torch.randn(args[which].shape, generator=g).to(DEV) * 2.0 ** -5 * args[which].abs().max()
        lo, hi = list(args), list(args)
        lo[which], hi[which] = (args[which] - v).bfloat16(), (args[which] + v).bfloat16()
        step = hi[which].double() - lo[which].double()   # exact step between bf16 points
        diff = loss(*hi) - loss(*lo)
        along = (grad.double() * step).sum().item()

        def f64(a):
            xx, g_, u_ = a[0].double().cpu(), a[1][0].double().cpu(), a[2][0].double().cpu()
            h = ref.act("silu", xx @ g_.T)[0] * (xx @ u_.T)
            return (h * dy.double().cpu()).sum().item()
        diff64 = f64(hi) - f64(lo)
        r = ref.glu_backward(c.x.double(), c.w[0][0].double(), c.w[1][0].double(),
                             c.dy.double(), "silu", F32)[which]
        st = step.cpu().reshape(r[0].shape)
        along64 = (r[0] * st).sum().item()
        _, hb = ref.glu_forward(c.x.double(), c.w[0][0].double(), c.w[1][0].double(), "silu", F32)
        fwd = 4 * (hb * c.dy.double().abs()).sum().item()     # both sides, perturbed inputs
        assert abs(diff - diff64) <= fwd
        assert abs(along - along64) <= (r[1] * st.abs()).sum().item()
