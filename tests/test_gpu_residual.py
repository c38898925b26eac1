"""Gated residual, its backward and the RMSNorm backward on the GPU against fp64, within the bounds of tests/_residual.py."""
import pytest
import torch

from depth_wise_attention_attnres_gb300 import binding as ar
from depth_wise_attention_attnres_gb300 import inputs
from tests import _residual as ref
from tests._gpu import dev, dtype_of

pytestmark = pytest.mark.gpu
EPS_POST, EPS_PRE = 1e-6, 1e-5
# Odd and unaligned widths (general kernels), multiples of 8 that fill a team of warps, part of one, or several
# passes of it; past the fast kernels' width.
SHAPES = [(1, 1), (3, 3), (5, 100), (1, 8), (7, 64), (129, 256), (1, 2048), (300, 640), (1000, 896), (33, 1000),
          (2, 4096), (17, 4104), (150, 6400), (40, 8192), (5, 8200)]
TYPES = [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"),
         ("f32", "f32", "f32")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Case:
    def __init__(self, T, d, types=("bf16", "f32", "f32"), gate="sigmoid", gate_rows=1, gate_type="bf16", post=True,
                 pre=True, with_x=True, with_dxo=True, scale=0.7, seed=0, shift=0):
        g = inputs.generator(seed, dev())

        def make(shape, dt, std=1.0, mean=0.0):
            n = 1
            for k in shape:
                n *= k
            t = torch.empty(n + shift, device=dev(), dtype=dtype_of(dt))[shift:].view(shape)
            return t.copy_(inputs.randn(shape, "f32", g, dev()) * std + mean)
        self.make = make
        self.T, self.d, self.types = T, d, types
        dt, xt, gt = types
        self.f, self.x = make((T, d), dt, 1.5), make((T, d), xt, 2.0) if with_x else None
        self.gpost = make((d,), "f32", 0.3, 1.0) if post else None
        self.gpre = make((d,), "f32", 0.3, 1.0) if pre else None
        self.gate_rows = gate_rows
        self.gate = make((-(-T // gate_rows), d), gate_type, 2.0) if gate != "none" else None
        self.sigmoid, self.scale = gate == "sigmoid", scale
        self.xo = make((T, d), xt)
        self.normed = make((T, d), dt) if pre else None
        self.dxo = make((T, d), gt, 0.5) if with_dxo else None
        self.dn = make((T, d), dt, 0.8) if pre else None

    def forward(self, x_out=None, stream=None):
        return ar.attnres_gated_residual(self.f, self.x, self.gpost, EPS_POST, self.gate, self.gate_rows,
                                         int(self.sigmoid), self.scale, self.xo if x_out is None else x_out, self.gpre,
                                         EPS_PRE, self.normed, stream=stream)

    def reference(self):
        return ref.forward(self.f, self.x, self.gpost, EPS_POST, self.gate, self.gate_rows, self.sigmoid, self.scale,
                           self.gpre, EPS_PRE)

    def outputs(self):
        dt, xt, gt = self.types
        out = {"df": self.make((self.T, self.d), dt), "dx": self.make((self.T, self.d), gt)}
        if self.gate is not None:
            out["dgate"] = torch.full_like(self.gate, float("nan"))
        if self.gpost is not None:
            out["dgamma_post"] = self.make((self.d,), "f32")
        if self.gpre is not None:
            out["dgamma_pre"] = self.make((self.d,), "f32")
        return out

    def backward(self, out, accumulate=False, **kw):
        ar.attnres_gated_residual_bwd(
            self.f, self.gpost, EPS_POST, self.gate, self.gate_rows, int(self.sigmoid), self.scale, self.xo, self.gpre,
            EPS_PRE, self.dxo, self.dn, out.get("df"), out.get("dx"), out.get("dgate"), out.get("dgamma_post"),
            out.get("dgamma_pre"), accumulate=accumulate, **kw)

    def bwd_reference(self):
        return ref.backward(self.f, self.gpost, EPS_POST, self.gate, self.gate_rows, self.sigmoid, self.scale, self.xo,
                            self.gpre, EPS_PRE, self.dxo, self.dn)


def check_forward(c):
    c.forward()
    vals, bounds = c.reference()
    ref.check(c.xo, vals["x_out"], bounds["x_out"], "x_out")
    if c.normed is not None:
        ref.check(c.normed, vals["normed"], bounds["normed"], "normed")


def check_backward(c):
    out = c.outputs()
    c.backward(out)
    vals, bounds = c.bwd_reference()
    for name, t in out.items():
        ref.check(t, vals[name], bounds[name], name)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_shapes(T, d, types):
    check_forward(Case(T, d, types, seed=T + d))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_backward_shapes(T, d, types):
    check_backward(Case(T, d, types, seed=T + d))


# One row for all tokens, more rows than tokens, runs that end inside a CTA's share, runs of 2, a short last run, and
# token counts that leave some team of the grid without a row (153, 305, 457).
@pytest.mark.parametrize("gate,gate_type", [("sigmoid", "bf16"), ("identity", "f32"), ("identity", "bf16")])
@pytest.mark.parametrize("T,d,gate_rows", [(50, 256, 50), (50, 256, 1000), (333, 640, 2), (1000, 320, 17), (700, 1024, 699),
                                           (1, 512, 1), (2, 512, 1), (1700, 264, 800), (40, 100, 7), (90, 8192, 31),
                                           (153, 256, 4), (153, 256, 100), (305, 264, 7), (457, 512, 150), (3000, 136, 40)])
def test_gate_rows(T, d, gate_rows, gate, gate_type):
    c = Case(T, d, gate=gate, gate_rows=gate_rows, gate_type=gate_type, seed=gate_rows)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("T,d", [(37, 640), (20, 100), (9, 8192)])
@pytest.mark.parametrize("gate", ["none", "identity"])
@pytest.mark.parametrize("post,pre,with_x,with_dxo", [
    (True, True, False, True), (True, False, True, True), (False, True, True, True), (False, False, False, True),
    (True, True, True, False), (False, True, True, False)])
def test_parts_left_out(T, d, gate, post, pre, with_x, with_dxo):
    c = Case(T, d, gate=gate, post=post, pre=pre, with_x=with_x, with_dxo=with_dxo)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("scale", [-1.5, 0.0])
@pytest.mark.parametrize("T,d,gate_rows", [(30, 640, 1), (30, 640, 7), (30, 640, 30), (30, 100, 7)])
def test_scales(T, d, gate_rows, scale):
    c = Case(T, d, gate_rows=gate_rows, scale=scale)
    check_forward(c)
    check_backward(c)


# Rows on both sides of where the kernels change: teams of one warp and several, 8 and 16 features a thread, the last
# widths of each, and fp32 rows that leave room for one row or none in shared memory.
@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("d", [248, 264, 504, 512, 520, 704, 712, 768, 776, 4096, 4104, 5120, 5128, 7168, 7176, 8184])
def test_widths(d, types):
    for gate, rows in (("none", 1), ("sigmoid", 1), ("sigmoid", 9)):
        c = Case(23, d, types, gate=gate, gate_rows=rows, gate_type="f32", seed=d)
        check_forward(c)
        check_backward(c)


@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("shift", [1, 4])
def test_unaligned_storage(types, shift):
    # 4 elements: fp32 rows on 16 bytes, bf16 rows on 8.
    c = Case(21, 512, types, shift=shift)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("T,d,join", [(1, 1, True), (5, 3, False), (64, 256, True), (1000, 640, True), (33, 1000, False),
                                      (150, 2048, True), (11, 4104, True), (31, 8192, False), (3, 8208, True)])
@pytest.mark.parametrize("dt,gt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_rmsnorm_bwd(T, d, join, dt, gt):
    c = Case(T, d, (dt, dt, gt), gate="none", with_dxo=join, seed=d)
    dx, dgamma = torch.empty(T, d, device=dev(), dtype=dtype_of(gt)), c.make((d,), "f32")
    start = dgamma.clone()
    ar.attnres_rmsnorm_bwd(c.xo, c.gpre, EPS_PRE, c.dn, c.dxo, dx, dgamma)
    vals, bounds = ref.backward(None, None, 0.0, None, 1, False, 1.0, c.xo, c.gpre, EPS_PRE, c.dxo, c.dn)
    ref.check(dx, vals["dx"], bounds["dx"], "dx")
    total = start.double() + vals["dgamma_pre"]
    ref.check(dgamma, total, bounds["dgamma_pre"], "dgamma")
    if join:  # in place
        ar.attnres_rmsnorm_bwd(c.xo, c.gpre, EPS_PRE, c.dn, c.dxo, c.dxo, None)
        assert torch.equal(c.dxo, dx)


def test_rmsnorm_bwd_matches_the_forward_by_differences():
    # Central differences of the library's own forward in fp32: h = 2^-6 of a loss of O(1) terms. Rounding of the
    # two losses (each a sum of 512 terms, each within 2^-22 of its magnitude) over 2h, plus h^2 / 6 of the third
    # derivative, which along a unit-size direction stays under 10 times the terms' magnitude.
    T, d = 2, 256
    c = Case(T, d, ("f32", "f32", "f32"), gate="none", with_dxo=False)
    dx = torch.empty(T, d, device=dev())
    ar.attnres_rmsnorm_bwd(c.xo, c.gpre, EPS_PRE, c.dn, None, dx)
    v = inputs.randn((T, d), "f32", inputs.generator(5, dev()), dev())
    h = 2.0 ** -6
    ends = []
    for sign in (1, -1):
        y = torch.empty(T, d, device=dev())
        ar.attnres_rmsnorm(c.xo + sign * h * v, c.gpre, EPS_PRE, y)
        ends.append(float((y.double() * c.dn.double()).sum()))
    size = float((y.double() * c.dn.double()).abs().sum())
    slope = float((dx.double() * v.double()).sum())
    assert abs((ends[0] - ends[1]) / (2 * h) - slope) <= size * (2 * 2.0 ** -22 / (2 * h) + 10 * h * h / 6)


@pytest.mark.parametrize("T,d", [(40, 640), (9, 101)])
def test_in_place(T, d):
    c = Case(T, d)
    c.forward()
    want, normed = c.xo.clone(), c.normed.clone()
    c.forward(x_out=c.x)
    assert torch.equal(c.x, want) and torch.equal(c.normed, normed)
    out, again = c.outputs(), c.outputs()
    c.backward(out)
    again["dx"] = c.dxo
    c.backward(again)
    assert all(torch.equal(out[k], again[k]) for k in out)


# (The last ones: a few rows, with a gate row for each, for runs of them, and for all.)
@pytest.mark.parametrize("T,d,gate_rows", [(700, 896, 1), (700, 896, 700), (500, 640, 37), (60, 100, 60), (30, 8192, 30),
                                           (3, 896, 1), (10, 896, 10), (11, 896, 11), (40, 256, 3), (41, 256, 3),
                                           (40, 256, 40), (2, 8192, 2), (2, 8192, 1), (16, 640, 1), (9, 896, 4)])
def test_same_bits_and_accumulate(T, d, gate_rows):
    c = Case(T, d, gate_rows=gate_rows, gate_type="f32")
    a, b = c.outputs(), c.outputs()
    c.backward(a)
    scratch = torch.full((ar.attnres_gated_residual_bwd_scratch_floats(T, d, gate_rows),), float("nan"), device=dev())
    c.backward(b, scratch=scratch)
    assert all(torch.equal(a[k], b[k]) for k in a)
    start = {k: c.make((d,), "f32") for k in ("dgamma_post", "dgamma_pre")}
    acc = {k: v.clone() for k, v in start.items()}
    c.backward(acc, accumulate=True)
    assert all(torch.equal(acc[k], start[k] + a[k]) for k in acc)


# Rings of one row and of two, several runs of a gate row to a team, scratch that is not on 16 bytes.
@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("T,gate_rows", [(500, 1), (500, 2), (500, 3), (500, 200), (1, 2), (7, 2)])
def test_widest_rows(T, gate_rows, types):
    c = Case(T, 8192, types, gate_rows=gate_rows, gate_type="f32")
    check_backward(c)
    need = ar.attnres_gated_residual_bwd_scratch_floats(T, 8192, gate_rows)
    a, b = c.outputs(), c.outputs()
    c.backward(a, scratch=torch.empty(need, device=dev()))
    c.backward(b, scratch=torch.full((need + 1,), float("nan"), device=dev())[1:])
    assert all(torch.equal(a[k], b[k]) for k in a)
    assert ar.attnres_device_status() == 0


# Rows of which an SM holds two when gamma_pre is not kept there, and the widths on both sides.
@pytest.mark.parametrize("types,gate,gate_rows,gate_type,d", [
    (types, gate, rows, gate_type, d) for types, gate, rows, gate_type, edges in [
        (("bf16", "f32", "f32"), "none", 1, "bf16", (7184, 8192)), (("bf16", "f32", "f32"), "sigmoid", 3, "f32", (7184, 8192)),
        (("bf16", "f32", "f32"), "sigmoid", 1, "bf16", (6384, 7184)), (("f32", "f32", "f32"), "none", 1, "bf16", (5744, 6384)),
        (("f32", "f32", "f32"), "sigmoid", 3, "f32", (5744, 6384)), (("f32", "f32", "f32"), "sigmoid", 1, "bf16", (5224, 5744)),
        (("bf16", "bf16", "bf16"), "sigmoid", 1, "f32", (7184, 8192))]
    for d in (edges[0] - 8, edges[0], edges[0] + 8, edges[1] - 8, edges[1], min(edges[1] + 8, 8192))])
def test_two_rows_in_an_sm(types, gate, gate_rows, gate_type, d):
    check_backward(Case(400, d, types, gate=gate, gate_rows=gate_rows, gate_type=gate_type, seed=d))


@pytest.mark.parametrize("T,d", [(50, 640), (50, 100), (12, 8192)])
def test_outputs_not_wanted(T, d):
    c = Case(T, d, gate_rows=50, gate_type="f32")
    full = c.outputs()
    c.backward(full)
    for name in full:
        only = {name: torch.full_like(full[name], 3.0)}
        c.backward(only)
        assert torch.equal(only[name], full[name]), name


@pytest.mark.parametrize("T,d", [(41, 640), (41, 100), (5, 8192)])
def test_nothing_else_is_written(T, d):
    c = Case(T, d, gate_rows=7, gate_type="f32")
    pad = 4096
    bufs, views = {}, {}
    shapes = {"x_out": c.xo, "normed": c.normed, **c.outputs()}
    for k, t in shapes.items():
        bufs[k] = torch.full((t.numel() + 2 * pad,), 12345.0, device=dev(), dtype=t.dtype)
        views[k] = bufs[k][pad:pad + t.numel()].view(t.shape)
    need = ar.attnres_gated_residual_bwd_scratch_floats(T, d, 7)
    sbuf = torch.full((need + 2 * pad,), 12345.0, device=dev())
    keep = [t.clone() for t in (c.f, c.x, c.gate, c.gpost, c.gpre, c.dxo, c.dn)]
    c.normed = views["normed"]
    c.forward(x_out=views["x_out"])
    c.xo = views["x_out"]
    c.backward(views, scratch=sbuf[pad:pad + need])
    torch.cuda.synchronize()
    for k, b in list(bufs.items()) + [("scratch", sbuf)]:
        edge = torch.full((pad,), 12345.0, device=dev(), dtype=b.dtype)
        assert torch.equal(b[:pad], edge) and torch.equal(b[-pad:], edge), k
    assert all(torch.equal(a, b) for a, b in zip(keep, (c.f, c.x, c.gate, c.gpost, c.gpre, c.dxo, c.dn)))
    assert ar.attnres_device_status() == 0


@pytest.mark.parametrize("d", [640, 100])
def test_a_bad_row_stays_in_its_row(d):
    c, good = Case(30, d), Case(30, d)
    for k in ("f", "x"):
        getattr(c, k)[11, 5] = float("nan")
        getattr(c, k)[13, 7] = float("inf")
    c.forward()
    good.forward()
    rest = [i for i in range(30) if i not in (11, 13)]
    assert torch.isnan(c.normed[11].float()).all()
    assert torch.equal(c.xo[rest], good.xo[rest]) and torch.equal(c.normed[rest], good.normed[rest])
    a, b = c.outputs(), good.outputs()
    c.backward(a)
    good.backward(b)
    for k in ("df", "dx", "dgate"):
        assert torch.equal(a[k][rest], b[k][rest]), k
    assert torch.isnan(a["dx"][11].float()).all()


def test_zero_rows_and_extreme_gates():
    # A row of zeros has a finite norm by eps; a gate of +-100 saturates without overflow, one of +-inf too.
    c = Case(20, 640, gate_type="f32")
    c.f[3].zero_()
    c.x[3].zero_()
    c.gate[:, :8] = torch.tensor([100.0, -100.0, 80.0, -80.0, 90.0, -90.0, 0.0, 15.0], device=dev())
    check_forward(c)
    check_backward(c)
    c.gate[:, 0], c.gate[:, 1] = float("inf"), float("-inf")
    c.forward()
    out = c.outputs()
    c.backward(out)
    assert torch.equal(c.xo[:, 1], c.x[:, 1]) and torch.isfinite(c.xo).all()
    assert (out["dgate"][:, :2] == 0).all() and torch.isfinite(out["df"].float()).all()


@pytest.mark.parametrize("d", [640, 100])
def test_no_tokens(d):
    c = Case(0, d, gate="none")
    c.forward()
    out = c.outputs()
    kept = {k: v.clone() for k, v in out.items()}
    c.backward(out, accumulate=True)
    assert torch.equal(out["dgamma_post"], kept["dgamma_post"])
    c.backward(out)
    assert (out["dgamma_post"] == 0).all() and (out["dgamma_pre"] == 0).all()
    c, dgamma = Case(0, d, ("bf16", "bf16", "bf16"), gate="none"), c.make((d,), "f32")
    ar.attnres_rmsnorm_bwd(c.xo, c.gpre, EPS_PRE, c.dn, None, torch.empty_like(c.xo), dgamma, accumulate=False)
    assert (dgamma == 0).all()


@pytest.mark.parametrize("d", [256, 100, 8192])
def test_one_gate_row_whatever_the_run(d):
    # Any gate_rows from T on means the one row, up to the largest number the call takes.
    want = None
    for rows in (20, 21, 2**31, 2**62):
        c = Case(20, d, gate_rows=rows, gate_type="f32", seed=7)
        out = c.outputs()
        c.forward()
        c.backward(out)
        got = [c.xo, c.normed] + [out[k] for k in sorted(out)]
        assert want is None or all(torch.equal(a, b) for a, b in zip(want, got))
        want = got


@pytest.mark.parametrize("gate_rows", [1, 130, 400])
def test_graph_and_streams(gate_rows):
    # Two captured graphs that share a scratch, replayed in turn on new values, on a stream that is not the current one.
    c, e = Case(400, 640, gate_rows=gate_rows, seed=1), Case(400, 640, gate_rows=gate_rows, seed=2)
    scratch = torch.empty(ar.attnres_gated_residual_bwd_scratch_floats(400, 640, gate_rows), device=dev())
    s = torch.cuda.Stream()
    outs, graphs = [c.outputs(), e.outputs()], []
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for case, out in zip((c, e), outs):
            case.forward()
            case.backward(out, scratch=scratch)
        torch.cuda.synchronize()
        for case, out in zip((c, e), outs):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                case.forward()
                case.backward(out, scratch=scratch)
            graphs.append(graph)
        fresh = Case(400, 640, gate_rows=gate_rows, seed=3)
        for k in ("f", "x", "gate", "dxo", "dn"):
            getattr(c, k).copy_(getattr(fresh, k))
        for _ in range(3):
            for graph in graphs:
                graph.replay()
    s.synchronize()
    for case, out in zip((c, e), outs):
        vals, bounds = case.reference()
        ref.check(case.xo, vals["x_out"], bounds["x_out"], "x_out")
        vals, bounds = case.bwd_reference()
        for name, t in out.items():
            ref.check(t, vals[name], bounds[name], name)
    # An explicit stream, the scratch allocated by the call.
    again = c.outputs()
    torch.cuda.synchronize()
    c.backward(again, stream=s)
    s.synchronize()
    assert all(torch.equal(again[k], outs[0][k]) for k in again)


def test_two_streams_at_once():
    cases = [Case(3000, 640, seed=4), Case(2500, 896, seed=5)]
    want = []
    for c in cases:
        out = c.outputs()
        c.forward()
        c.backward(out)
        want.append(out)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                out = c.outputs()
                c.forward()
                c.backward(out)
                got.append(out)
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert all(torch.equal(out[k], want[i % 2][k]) for k in out)


def test_rows_past_32_bit_offsets():
    # 2^31 + elements of bf16 (4.3 GB a tensor): the last rows against the reference of those rows alone.
    d = 8192
    T = (1 << 31) // d + 5
    g = inputs.generator(9, dev())
    tail = 8
    f = torch.zeros(T, d, device=dev(), dtype=torch.bfloat16)
    f[-tail:] = inputs.randn((tail, d), "bf16", g, dev())
    dn = torch.zeros_like(f)
    dn[-tail:] = inputs.randn((tail, d), "bf16", g, dev())
    gamma = torch.ones(d, device=dev())
    xo, normed = torch.empty_like(f), torch.empty_like(f)
    ar.attnres_gated_residual(f, None, gamma, EPS_POST, None, 1, 0, 1.0, xo, gamma, EPS_PRE, normed)
    vals, bounds = ref.forward(f[-tail:], None, gamma, EPS_POST, None, 1, False, 1.0, gamma, EPS_PRE)
    ref.check(xo[-tail:], vals["x_out"], bounds["x_out"], "x_out")
    ref.check(normed[-tail:], vals["normed"], bounds["normed"], "normed")
    df, dx, dgamma = f.new_empty(T, d), f.new_empty(T, d), torch.empty(d, device=dev())
    ar.attnres_gated_residual_bwd(f, gamma, EPS_POST, None, 1, 0, 1.0, xo, gamma, EPS_PRE, None, dn, df, dx,
                                  dgamma_pre=dgamma, accumulate=False)
    vals, bounds = ref.backward(f[-tail:], gamma, EPS_POST, None, 1, False, 1.0, xo[-tail:], gamma, EPS_PRE, None, dn[-tail:])
    ref.check(dx[-tail:], vals["dx"], bounds["dx"], "dx")
    ref.check(dgamma, vals["dgamma_pre"], bounds["dgamma_pre"], "dgamma_pre")
    assert (dx[:-tail] == 0).all()


def test_withheld_row_times_out_and_recovers():
    # 900 rows of 640 over at most 760 teams: every team has one row or two, each withholds its first.
    c = Case(900, 640, gate_rows=100, gate_type="f32")
    good = c.outputs()
    c.forward()
    c.backward(good)
    want = c.xo.clone()
    assert ar.attnres_device_status() == 0
    for run in (c.forward, lambda: c.backward(c.outputs())):
        ar.attnres_test_withhold_stage(ar.WITHHOLD_RESIDUAL, 0)
        try:
            run()
        finally:
            ar.attnres_test_withhold_stage(ar.WITHHOLD_NONE)
        assert ar.attnres_device_status() == 4          # ATTNRES_ERR_TIMEOUT
        assert ar.attnres_device_status() == 0
        c.xo.copy_(want)
    again = c.outputs()
    c.forward()
    c.backward(again)
    assert torch.equal(c.xo, want) and all(torch.equal(again[k], good[k]) for k in good)


@pytest.mark.parametrize("d", [512, 100])
def test_sigmoid_alone(d):
    # f = 1, x = 0, no norms, scale 1: x_out is the sigmoid itself and with dx_out = 1 dgate is its slope; over the
    # whole range of fp32's results, subnormal ones too (half a step of 2^-149 more).
    g = torch.cat([torch.linspace(-106, 106, 400 * d - 4 * d, device=dev()),
                   torch.logspace(-30, 2, 2 * d, device=dev()), -torch.logspace(-30, 2, 2 * d, device=dev())]).view(400, d)
    f, out, dgate = torch.ones(400, d, device=dev()), torch.empty(400, d, device=dev()), torch.empty(400, d, device=dev())
    ar.attnres_gated_residual(f, None, None, 0.0, g, 1, ar.GATE_SIGMOID, 1.0, out)
    ar.attnres_gated_residual_bwd(f, None, 0.0, g, 1, ar.GATE_SIGMOID, 1.0, None, None, 0.0, f, None, None, None, dgate)
    want, slope = ref.act(g.double(), True)
    for got, value in ((out, want), (dgate, slope)):
        assert ((got.double() - value).abs() <= 20 * ref.U * value + 2.0 ** -149).all()
