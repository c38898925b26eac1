"""8-bit rows on the GPU: writing, reading back, the Full read over them, weights and the query projection, each
against its fp64 definition (tests/_q8.py, whose bounds are those of fp32 evaluation)."""
import copy

import pytest
import torch

import depth_wise_attention_attnres_gb300 as ar
from depth_wise_attention_attnres_gb300 import binding
from tests import _q8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def filled(n, T, d, value=0xA5):
    rows = ar.Q8Rows(n, T, d, device=DEV)
    rows.buffer.fill_(value)
    return rows


def values_of(rows):
    """What rows stand for, in fp64 [n, T, d]."""
    return rows.codes.double() * _q8.power(rows.exponents.long() - 127)[..., torch.arange(rows.d, device=DEV) // 128]


def made(n, T, d, g, loud=True):
    """Rows written by the library, and the values they stand for in fp64."""
    rows = ar.Q8Rows(n, T, d, device=DEV)
    ar.attnres_q8_write(_q8.history(n, T, d, g, DEV, loud), rows)
    return rows, values_of(rows)


def check_rows(rows, x, n, T, d):
    G = _q8.groups(d)
    for i in range(n):
        codes, e = _q8.quantise(x[i], 1)
        assert torch.equal(rows.exponents[i, :T].int(), e + 127)
        got = rows.codes[i, :T].double()
        assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(codes, nan=1e9))
        v = _q8.values(codes, e)
        ms = v.square().mean(1)
        room = ms * ((d + 4) * _q8.U) + 2.0 ** -120
        ok = ((rows.mean_square[i, :T].double() - ms).abs() <= room) | (ms.isnan() & rows.mean_square[i, :T].isnan())
        ok |= ms > 2.0 ** 127  # past fp32
        assert ok.all()
    # what pads codes and tails is zero
    at = -(-G // 4) * 4
    tails = rows.tails[:n, :T]
    assert not padded_codes(rows)[:n, :T, d:].any() and not tails[..., G:at].any() and not tails[..., at + 4:].any()


def padded_codes(rows):
    width = 128 * _q8.groups(rows.d)
    return rows.buffer[:, :rows.T * width].view(rows.n, rows.T, width)


def source(rows, i):
    """Source i of `rows` as rows of their own (a copy)."""
    one = ar.Q8Rows(1, rows.T, rows.d, device=DEV)
    one.buffer.copy_(rows.buffer[i:i + 1])
    return one


WIDTHS = [1, 7, 16, 100, 127, 128, 129, 200, 256, 384, 520, 640, 896, 1000, 1016, 1024, 1025, 1160, 2048, 2050, 4099]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_write(d, dtype):
    for n, T in ((1, 1), (1, 8), (2, 5), (3, 67)):
        x = _q8.history(n, T, d, gen(d * 7 + T), DEV).to(TYPES[dtype])
        rows = filled(n + 1, T + 2, d)
        ar.attnres_q8_write(x, rows, src=1)
        assert (rows.buffer[0] == 0xA5).all()
        used = (T + 2) * (128 * _q8.groups(d) + rows.tails.shape[-1])
        for rest in (padded_codes(rows)[1:, T:], rows.tails[1:, T:], rows.buffer[1:, used:]):
            assert (rest == 0xA5).all()
        for i in range(n):
            check_rows(source(rows, 1 + i), x[i:i + 1], 1, T, d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_write_special_values(dtype):
    d, t = 300, TYPES[dtype]
    x = torch.randn(12, d, generator=gen(3), device=DEV)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 130] = float("nan")
    x[3, 131:] = float("-inf")
    x[4] *= 1e-38
    x[5] *= 1e-43
    x[6] = torch.finfo(t).max
    x[7, ::3] = -3.3e38
    x[8, 200] = 448.0 * 2 ** 7
    x[9] = 0
    x[9, 299] = -torch.finfo(torch.float32).smallest_normal
    x[10, :128] = 1.75 * 2.0 ** 10
    x[11, 0] = 1.7500001 * 2.0 ** 10
    x = x.to(t)
    rows = filled(1, 12, d)
    ar.attnres_q8_write(x, rows)
    check_rows(rows, x[None], 1, 12, d)
    assert rows.mean_square[0, [1, 2, 3]].isnan().all() and rows.mean_square[0, 0] == 0
    back = torch.empty(12, d, device=DEV)
    ar.attnres_q8_read(rows, back)
    assert torch.equal(back.isfinite(), x.isfinite())


def test_every_code_and_ties():
    """Every e4m3 number, and the middles between neighbours (which go to the even one), come out as the definition's."""
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).float()
    codes = codes[codes.isfinite()].sort().values
    mid = (codes[1:].double() + codes[:-1].double()) / 2
    x = torch.cat([codes.double(), mid, mid * (1 + 2 ** -20), mid * (1 - 2 ** -20)]).float()
    x = torch.cat([x, torch.zeros(-x.numel() % 127, device=DEV)]).view(-1, 127)
    x = torch.cat([torch.full((x.shape[0], 1), 448.0, device=DEV), x], 1)  # the scale is 1
    for scale in (1.0, 2.0 ** -100, 2.0 ** 90):
        rows = filled(1, x.shape[0], 128)
        ar.attnres_q8_write(x * scale, rows)
        assert (rows.exponents[0] == 127 + round(torch.tensor(scale).log2().item())).all()
        assert torch.equal(rows.codes[0].double(), _q8.round_e4m3(x.double()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_read_back(d, dtype):
    for n, T in ((1, 1), (2, 9), (3, 70)):
        rows, v = made(n + 1, T + 1, d, gen(d + T))
        store = torch.full((n + 1, T + 1, d), 7.0, device=DEV, dtype=TYPES[dtype])
        out = store.view(-1)[:n * (T + 1) * d].view(n, T + 1, d)[:, :T]
        ar.attnres_q8_read(rows, out, src=1)
        assert torch.equal(out, v[1:, :T].float().to(TYPES[dtype]))
        store.view(-1)[:n * (T + 1) * d].view(n, T + 1, d)[:, :T] = 7.0
        assert (store == 7.0).all()
        # writing what was read back gives the same values
        again = ar.Q8Rows(1, T, d, device=DEV)
        first = torch.empty(T, d, device=DEV)
        ar.attnres_q8_write(ar.attnres_q8_read(rows, first), again)
        assert torch.equal(ar.attnres_q8_read(again, torch.empty_like(first)), first)


def read_case(n, T, d, dtype, query, pre, seed, eps=1e-6, keep=True):
    g = gen(seed)
    rows, v = made(n, T, d, g)
    gamma = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    q = torch.randn((T, d) if query == "token" else (d,), generator=g, device=DEV) * (2 / d ** 0.5)
    gp = 1 + 0.2 * torch.randn(d, generator=g, device=DEV) if pre else None
    store = torch.full((T + 2, d), 9.0, device=DEV, dtype=TYPES[dtype])
    store2 = torch.full((T + 2, d), 9.0, device=DEV, dtype=TYPES[dtype]) if pre else None
    out = store[1:T + 1] if keep else None
    normed = store2[1:T + 1] if pre else None
    w, Q = (None, q) if query == "token" else (q, None)
    ar.attnres_full_fwd_q8(rows, n, w, gamma, eps, out, Q=Q, gamma_pre=gp, eps_pre=1e-5, out_normed=normed)
    assert ar.attnres_device_status() == 0
    z, dz, zn, dn = _q8.read(v, q, gamma, eps, gp, 1e-5)
    if keep:
        _q8.assert_within(out, z, dz, "z")
    if pre:
        _q8.assert_within(normed, zn, dn, "normed")
    for s in (store, store2):
        assert s is None or (s[0] == 9.0).all() and (s[T + 1] == 9.0).all()


@pytest.mark.parametrize("d", WIDTHS)
def test_full_read_widths(d):
    read_case(5, 13, d, "f32", "fixed", False, d)
    read_case(9, 70, d, "bf16", "token", True, d + 1)
    read_case(2, 3, d, "f32", "token", True, d + 2, keep=False)


@pytest.mark.parametrize("n,T", [(1, 1), (1, 9), (2, 1), (3, 2), (7, 1), (8, 5), (9, 33), (64, 1), (141, 1), (141, 3),
                                 (33, 700), (4, 3001), (300, 2)])
@pytest.mark.parametrize("d", [128, 256, 384, 640, 896, 1152, 2048, 2304])
def test_full_read_sources_and_tokens(n, T, d):
    read_case(n, T, d, "f32", "fixed", T % 2 == 1, n * 1000 + T)


@pytest.mark.parametrize("T", [150, 608, 1215, 1216, 1217, 2431, 2433, 4865, 4900])
def test_full_read_around_the_sharing_of_sources(T):
    """Token counts at which the warps a token's sources are shared by change, and the last groups of tokens."""
    for d in (128, 512, 896, 2048):
        read_case(9, T, d, "bf16", "fixed", False, T)


@pytest.mark.parametrize("d", [100, 256, 384, 512, 640, 896, 1000, 1152, 2048])
def test_full_read_stages(d):
    """Source counts around the number a stage holds, with sources shared between warps and without."""
    for n in (1, 2, 3, 4, 5, 6, 7, 8, 9, 13):
        read_case(n, 350 + n, d, "f32", "fixed", False, n)
        read_case(n, 5003, d, "bf16", "fixed", n % 2 == 1, n + 50)


@pytest.mark.parametrize("n,T", [(12, 227), (12, 228), (12, 229), (40, 19), (40, 38), (17, 39), (33, 76), (33, 77), (9, 152),
                                 (9, 153), (200, 11)])
def test_full_read_clusters(n, T):
    """Token counts around those at which CTAs begin to share a token's sources, and at which this ends."""
    for d in (128, 512, 640, 1024, 1152, 1600, 2048):
        read_case(n, T, d, "f32", "token" if T % 2 else "fixed", T % 3 == 0, n + T)


@pytest.mark.parametrize("d", [2176, 3000, 4096, 5120, 8200, 16384])
def test_full_read_wide(d):
    """Rows past the streaming kernel: fewer and more sources than warps, more tokens than CTAs at once, each query and output."""
    read_case(3, 700, d, "bf16", "fixed", False, d)
    read_case(17, 21, d, "f32", "token", True, d + 1)
    read_case(64, 2, d, "bf16", "fixed", True, d + 2, keep=False)
    read_case(9, 650, d, "f32", "fixed", True, d + 3)


def test_broken_rows_in_clusters():
    """NaN in one of many sources, and a token whose other sources have weight 0."""
    n, T, d = 141, 3, 640
    x = _q8.history(n, T, d, gen(4), DEV, loud=False)
    w, gamma = torch.randn(d, generator=gen(5), device=DEV) / d ** 0.5, torch.ones(d, device=DEV)
    for i in (0, 70, 140):
        y = x.clone()
        y[i, 1, 639] = float("inf")
        rows = ar.Q8Rows(n, T, d, device=DEV)
        ar.attnres_q8_write(y, rows)
        out = ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, torch.empty(T, d, device=DEV))
        assert out[1].isnan().all() and out[[0, 2]].isfinite().all()
    y = x.clone()
    y[100, 2] = 50 * w  # the score of one source is above all others
    rows = ar.Q8Rows(n, T, d, device=DEV)
    ar.attnres_q8_write(y, rows)
    out = ar.attnres_full_fwd_q8(rows, n, 90 * w, gamma, 1e-6, torch.empty(T, d, device=DEV))
    z, dz, _, _ = _q8.read(values_of(rows), 90 * w, gamma, 1e-6)
    _q8.assert_within(out, z, dz)


def test_two_graphs_at_once():
    """Two captured chains replayed on two streams at the same time: no memory is shared between calls."""
    n, T, d = 9, 2500, 640
    w, gamma = torch.randn(d, generator=gen(2), device=DEV) * 0.1, torch.ones(d, device=DEV)
    W8 = ar.attnres_q8_weight(torch.randn(d, d, generator=gen(3), device=DEV) / d ** 0.5, ar.Q8Weight(d, d, device=DEV))
    runs = []
    for k in range(2):
        x = _q8.history(n, T, d, gen(10 + k), DEV)
        rows, out, Q = ar.Q8Rows(n, T, d, device=DEV), torch.empty(T, d, device=DEV), torch.empty(T, d, device=DEV)
        few = torch.empty(2, d, device=DEV)

        def chain(x=x, rows=rows, out=out, Q=Q, few=few):
            ar.attnres_q8_write(x, rows)
            ar.attnres_query_projection_q8(rows, n - 1, W8, Q)
            ar.attnres_full_fwd_q8(rows, n, None, gamma, 1e-6, out, Q=Q)
            ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, few)

        chain()
        torch.cuda.synchronize()
        want = [t.clone() for t in (rows.buffer, out, Q, few)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain()
        runs.append((graph, [rows.buffer, out, Q, few], want, torch.cuda.Stream(), chain))  # the chain keeps its input
    for _, got, *_ in runs:
        for t in got:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, _, _, stream, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert ar.attnres_device_status() == 0
    for _, got, want, *_ in runs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("shift", [16, 112])
def test_rows_off_128_bytes(shift):
    """Sources and weights on 16-byte boundaries that are not 128-byte ones: the same bits."""

    def moved(holder):
        store = torch.full((holder.buffer.numel() + 256,), 0x5A, dtype=torch.uint8, device=DEV)
        other = copy.copy(holder)
        other.__dict__.pop("codes", None)
        other.buffer = store[shift:shift + holder.buffer.numel()].view(holder.buffer.shape)
        assert other.pointer % 128 == shift
        return other, store

    for n, T, d, m in ((5, 700, 640, 640), (9, 40, 1000, 77), (3, 2, 2048, 300), (4, 60, 2304, 130)):
        g = gen(n)
        x = _q8.history(n, T, d, g, DEV)
        W = torch.randn(m, d, generator=g, device=DEV) / d ** 0.5
        w, gamma = torch.randn(d, generator=g, device=DEV) * 0.05, torch.ones(d, device=DEV)
        results = []
        for off in (False, True):
            rows, W8 = filled(n, T, d, 0), ar.Q8Weight(m, d, device=DEV)
            stores = []
            if off:
                (rows, a), (W8, b) = moved(rows), moved(W8)
                rows.buffer.zero_()
                stores = [(a, rows), (b, W8)]
            ar.attnres_q8_write(x, rows)
            ar.attnres_q8_weight(W, W8)
            out, Q, back = torch.empty(T, d, device=DEV), torch.empty(T, m, device=DEV), torch.empty(n, T, d, device=DEV)
            ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, out)
            ar.attnres_query_projection_q8(rows, n - 1, W8, Q)
            ar.attnres_q8_read(rows, back)
            for store, holder in stores:
                assert (store[:shift] == 0x5A).all() and (store[shift + holder.buffer.numel():] == 0x5A).all()
            results.append((rows.buffer.clone(), W8.buffer.clone(), out, Q, back))
        assert ar.attnres_device_status() == 0
        for a, b in zip(*results):
            assert torch.equal(a, b)


def test_copies_of_rows():
    """A copied Q8Rows or Q8Weight has storage of its own."""
    T, d = 20, 256
    rows, v = made(2, T, d, gen(1))
    other = copy.deepcopy(rows)
    ar.attnres_q8_write(torch.ones(T, d, device=DEV), other, 1)
    assert torch.equal(values_of(rows), v) and (values_of(other)[1] == 1).all() and torch.equal(values_of(other)[0], v[0])
    W8 = ar.attnres_q8_weight(torch.ones(d, d, device=DEV), ar.Q8Weight(d, d, device=DEV))
    zero = ar.attnres_q8_weight(torch.zeros(d, d, device=DEV), copy.deepcopy(W8))
    Q = torch.empty(T, d, device=DEV)
    assert (ar.attnres_query_projection_q8(other, 1, W8, Q) == d).all()
    assert not ar.attnres_query_projection_q8(other, 1, zero, Q).any()


def test_single_source_is_returned():
    rows, v = made(1, 50, 700, gen(1))
    out = torch.empty(50, 700, device=DEV)
    ar.attnres_full_fwd_q8(rows, 1, torch.randn(700, device=DEV), torch.ones(700, device=DEV), 1e-6, out)
    assert torch.equal(out.double(), v[0])


def test_scores_apart():
    """Queries so long that one source takes all weight, and zero ones (the plain mean)."""
    for scale, n, T, d in ((0.0, 6, 40, 640), (80.0, 6, 40, 640), (80.0, 141, 2, 2048), (300.0, 17, 9, 256)):
        g = gen(5)
        rows, v = made(n, T, d, g, loud=False)
        q = torch.randn(d, generator=g, device=DEV) * (scale / d ** 0.5)
        gamma = torch.ones(d, device=DEV)
        out = torch.empty(T, d, device=DEV)
        ar.attnres_full_fwd_q8(rows, n, q, gamma, 1e-6, out)
        z, dz, _, _ = _q8.read(v, q, gamma, 1e-6)
        _q8.assert_within(out, z, dz, f"scale {scale}")


def test_broken_rows_stay_to_themselves():
    """A token with a NaN in one source is NaN; its neighbours, in the same warp or not, are what they were. A score of
    -inf has weight 0, zero rows have score 0."""
    for n, T, d in ((5, 37, 512), (9, 37, 1024), (5, 2, 2048), (3, 5000, 256), (20, 1, 384), (9, 7, 2600)):
        x = _q8.history(n, T, d, gen(2), DEV, loud=False)
        w, gamma = torch.randn(d, generator=gen(3), device=DEV) / d ** 0.5, torch.ones(d, device=DEV)
        rows = ar.Q8Rows(n, T, d, device=DEV)
        ar.attnres_q8_write(x, rows)
        want = torch.empty(T, d, device=DEV)
        ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, want)
        x[n - 1, T // 2, 3] = float("nan")
        ar.attnres_q8_write(x, rows)
        got = torch.empty(T, d, device=DEV)
        ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, got)
        assert got[T // 2].isnan().all()
        others = torch.arange(T, device=DEV) != T // 2
        assert torch.equal(got[others], want[others])
        x[n - 1, T // 2] = 0
        x[0, T // 2] = 0
        ar.attnres_q8_write(x, rows)
        ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, got)
        v = values_of(rows)
        z, dz, _, _ = _q8.read(v, w, gamma, 1e-6)
        _q8.assert_within(got, z, dz)
    # -inf: a query whose product with the first source passes fp32's range downwards
    n, T, d = 4, 3, 256
    x = torch.ones(n, T, d, device=DEV)
    x[0] = -1
    x[1:] *= 1e-3
    rows = ar.Q8Rows(n, T, d, device=DEV)
    ar.attnres_q8_write(x, rows)
    out = torch.empty(T, d, device=DEV)
    ar.attnres_full_fwd_q8(rows, n, torch.full((d,), 2.0e36, device=DEV), torch.ones(d, device=DEV), 1.0, out)
    assert out.isfinite().all() and (out > 0).all()


def test_unaligned_outputs_and_queries():
    for d in (256, 896, 1000):
        n, T = 4, 21
        rows, v = made(n, T, d, gen(d))
        flat = torch.randn(T * d + 2 * d + 16, generator=gen(d + 1), device=DEV) * 0.05
        w, gamma = flat[1:1 + d], 1 + flat[d + 3:2 * d + 3]
        Q = flat[2 * d + 7:2 * d + 7 + T * d].view(T, d)
        for dtype in TYPES.values():
            store = torch.zeros(T * d + 8, device=DEV, dtype=dtype)
            out = store[3:3 + T * d].view(T, d)
            for q in (w, Q):
                ar.attnres_full_fwd_q8(rows, n, w if q is w else None, gamma, 1e-6, out, Q=Q if q is Q else None)
                z, dz, _, _ = _q8.read(v, q, gamma, 1e-6)
                _q8.assert_within(out, z, dz)
            assert not store[:3].any() and not store[3 + T * d:].any()
            ar.attnres_q8_read(rows, out, src=2)
            assert torch.equal(out, v[2].float().to(dtype))
            assert not store[:3].any() and not store[3 + T * d:].any()
            again = filled(1, T, d)
            ar.attnres_q8_write(out, again)
            check_rows(again, out[None], 1, T, d)


def test_offsets_past_32_bits():
    """A history of over 4 GiB: its last source and last tokens."""
    n, T, d = 3, 700_000, 2048
    rows = ar.Q8Rows(n, T, d, device=DEV)
    assert rows.buffer.numel() > 1 << 32
    tail = T - 50
    x = _q8.history(1, T, d, gen(1), DEV)[0]
    for i in range(n):
        ar.attnres_q8_write(x * (i + 1), rows, src=i)
    v = torch.stack([_q8.values(rows.codes[i, tail:], rows.exponents[i, tail:].int() - 127) for i in range(n)])
    codes, e = _q8.quantise(3 * x[tail:])
    assert torch.equal(v[2], _q8.values(codes, e))
    w, gamma = torch.randn(d, generator=gen(2), device=DEV) * 0.03, torch.ones(d, device=DEV)
    out = torch.empty(T, d, device=DEV, dtype=torch.bfloat16)
    ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, out)
    z, dz, _, _ = _q8.read(v, w, gamma, 1e-6)
    _q8.assert_within(out[tail:], z, dz)
    ar.attnres_q8_read(rows, out, src=2)
    assert torch.equal(out[tail:], v[2].float().to(torch.bfloat16))
    W8 = ar.Q8Weight(128, d, device=DEV)
    W = torch.randn(128, d, generator=gen(3), device=DEV)
    ar.attnres_q8_weight(W, W8)
    Q = torch.empty(T, 128, device=DEV)
    ar.attnres_query_projection_q8(rows, 2, W8, Q)
    assert ar.attnres_device_status() == 0
    wv = _q8.values(W8.codes, W8.exponents.int() - 127, 128)
    _q8.assert_within(Q[tail:], v[2] @ wv.t(), (v[2].abs() @ wv.abs().t()) * ((d + 8) * _q8.U))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,d", [(1, 1), (3, 200), (128, 128), (129, 127), (300, 640), (640, 300), (130, 2200)])
def test_weight(m, d, dtype):
    W = torch.randn(m, d, generator=gen(m), device=DEV).to(TYPES[dtype]) * 0.1
    W[0, 0] = 3.0
    if m > 2:
        W[2, d - 1] = float("inf")
    W8 = ar.Q8Weight(m, d, device=DEV)
    W8.buffer.fill_(0xA5)
    ar.attnres_q8_weight(W, W8)
    codes, e = _q8.quantise(W, 128)
    assert torch.equal(W8.exponents.int(), e + 127)
    assert torch.equal(torch.nan_to_num(W8.codes.double(), nan=1e9), torch.nan_to_num(codes, nan=1e9))
    G = _q8.groups(d)
    assert not W8.buffer[:m * G * 128].view(m, G * 128)[:, d:].any()
    assert not W8.buffer[m * G * 128:].view(-1, -(-G // 16) * 16)[:, G:].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weight_off_16_bytes(dtype):
    """Weights that start between 16-byte boundaries: the same bits."""
    W = torch.randn(200 * 256 + 8, generator=gen(1), device=DEV).to(TYPES[dtype])
    want, got = ar.Q8Weight(200, 256, device=DEV), ar.Q8Weight(200, 256, device=DEV)
    for off in (1, 3):
        part = W[off:off + 200 * 256].view(200, 256)
        ar.attnres_q8_weight(part, got)
        ar.attnres_q8_weight(part.clone(), want)
        assert torch.equal(got.buffer, want.buffer)


def projection_case(T, d, m, seed, spread=0.0, src=0):
    g = gen(seed)
    rows, v = made(src + 1, T, d, g)
    W = torch.randn(m, d, generator=g, device=DEV) / d ** 0.5
    if spread:
        W *= torch.exp2(torch.randint(-int(spread), int(spread) + 1, (1, d), generator=g, device=DEV).float())
    W8 = ar.Q8Weight(m, d, device=DEV)
    ar.attnres_q8_weight(W, W8)
    store = torch.full((T + 2, m), 5.0, device=DEV)
    ar.attnres_query_projection_q8(rows, src, W8, store[1:T + 1])
    assert ar.attnres_device_status() == 0
    wv = _q8.values(W8.codes, W8.exponents.int() - 127, 128)
    ref = v[src] @ wv.t()
    # any order of d products and G scaled sums
    bound = (v[src].abs() @ wv.abs().t()) * ((d + 2 * _q8.groups(d) + 4) * _q8.U)
    _q8.assert_within(store[1:T + 1], ref, bound, f"{T} {d} {m}")
    assert (store[0] == 5.0).all() and (store[T + 1] == 5.0).all()


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 100, 128, 129, 300])
@pytest.mark.parametrize("d,m", [(1, 1), (128, 128), (200, 77), (640, 640), (896, 900), (1000, 130), (2048, 256), (2200, 2052)])
def test_projection(T, d, m):
    projection_case(T, d, m, T + d)


@pytest.mark.parametrize("T", [1, 3, 5, 8, 12, 16])
@pytest.mark.parametrize("d,m", [(640, 5120), (1024, 4000), (2048, 2050), (2176, 1025), (4096, 300)])
def test_projection_few_tokens(T, d, m):
    """Sizes on both sides of the choice between the kernels for few tokens and the tensor cores."""
    projection_case(T, d, m, T)


def test_projection_larger():
    projection_case(4999, 896, 896, 1)
    projection_case(20000, 1024, 1024, 2, src=1)
    projection_case(2500, 2048, 6144, 3, spread=6)


@pytest.mark.parametrize("T", [3, 40])
def test_projection_far_scales(T):
    """Products of scales that are no fp32 number by themselves: 2^120 times 2^-126, and sums below 2^-126."""
    d, m = 384, 130
    x = torch.randn(T, d, generator=gen(1), device=DEV)
    W = torch.randn(m, d, generator=gen(2), device=DEV)
    # groups of features: 1e37 by 1e-37, 1e-30 by 1e-15, 1 by 1e-30
    x[:, :128] *= 1e37
    W[:, :128] *= 1e-37
    x[:, 128:256] *= 1e-30
    W[:, 128:256] *= 1e-15
    W[:, 256:] *= 1e-30
    for cut in (0, 128):  # with the ordinary group, and without
        rows, W8 = ar.Q8Rows(1, T, d - cut, device=DEV), ar.Q8Weight(m, d - cut, device=DEV)
        ar.attnres_q8_write(x[:, cut:].contiguous(), rows)
        ar.attnres_q8_weight(W[:, cut:].contiguous(), W8)
        Q = torch.empty(T, m, device=DEV)
        ar.attnres_query_projection_q8(rows, 0, W8, Q)
        v = _q8.values(rows.codes[0], rows.exponents[0].int() - 127)
        wv = _q8.values(W8.codes, W8.exponents.int() - 127, 128)
        _q8.assert_within(Q, v @ wv.t(), (v.abs() @ wv.abs().t()) * ((d + 8) * _q8.U) + 2.0 ** -148)


def test_projection_nan():
    T, d, m = 40, 256, 200
    x, W = torch.randn(T, d, generator=gen(1), device=DEV), torch.randn(m, d, generator=gen(2), device=DEV)
    x[7, 200] = float("nan")
    W[11, 3] = float("inf")
    for t in (T, 9):
        rows, W8 = ar.Q8Rows(1, t, d, device=DEV), ar.Q8Weight(m, d, device=DEV)
        ar.attnres_q8_write(x[:t].contiguous(), rows)
        ar.attnres_q8_weight(W, W8)
        Q = torch.empty(t, m, device=DEV)
        ar.attnres_query_projection_q8(rows, 0, W8, Q)
        broken = torch.zeros(t, m, dtype=torch.bool, device=DEV)
        broken[7], broken[:, 11] = True, True
        assert torch.equal(Q.isnan(), broken)


def test_same_bits_and_batch_independence():
    """The same call gives the same bits, and a token's results do not depend on which others are in the batch."""
    n, T, d = 12, 4000, 640
    rows, _ = made(n, T, d, gen(1))
    w, gamma = torch.randn(d, generator=gen(2), device=DEV) * 0.1, torch.ones(d, device=DEV)
    a, b = torch.empty(T, d, device=DEV), torch.empty(T, d, device=DEV)
    for out in (a, b):
        ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, out)
    assert torch.equal(a, b)
    few = ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, torch.empty(2001, d, device=DEV))
    assert torch.allclose(few, a[:2001], rtol=1e-4, atol=1e-4)
    W8 = ar.attnres_q8_weight(torch.randn(640, d, generator=gen(3), device=DEV), ar.Q8Weight(640, d, device=DEV))
    qa, qb = torch.empty(T, 640, device=DEV), torch.empty(T, 640, device=DEV)
    for q in (qa, qb):
        ar.attnres_query_projection_q8(rows, 3, W8, q)
    assert torch.equal(qa, qb)


def model(x, W, Gamma, Pre, mats, W8s, rows, reads, normed, Q, stream=None):
    """A Full AttnRes model over an 8-bit history, sublayers being a product with a matrix: odd reads with the fixed
    query, even ones with a query projected from the last source."""
    ar.attnres_q8_write(x, rows, 0, stream=stream)
    for r in range(len(reads)):
        if r % 2:
            ar.attnres_query_projection_q8(rows, r, W8s[r], Q, stream=stream)
            ar.attnres_full_fwd_q8(rows, r + 1, None, Gamma[r], 1e-6, reads[r], Q=Q, gamma_pre=Pre[r], eps_pre=1e-5,
                                   out_normed=normed, stream=stream)
        else:
            ar.attnres_full_fwd_q8(rows, r + 1, W[r], Gamma[r], 1e-6, reads[r], gamma_pre=Pre[r], eps_pre=1e-5,
                                   out_normed=normed, stream=stream)
        if r + 1 < len(reads):
            ar.attnres_q8_write(torch.mm(normed, mats[r]), rows, r + 1, stream=stream)


@pytest.mark.parametrize("T", [1, 33, 600])
def test_model_run(T):
    """The operators in turn, as a model runs them: each read against the definition on the rows as they were written;
    the same captured into a graph and replayed on new inputs; and the backward through the rows read back."""
    R, d, g = 6, 256, gen(T)
    x = torch.randn(T, d, generator=g, device=DEV).bfloat16()
    W = torch.randn(R, d, generator=g, device=DEV) * 0.1
    Gamma, Pre = 1 + 0.1 * torch.randn(R, d, generator=g, device=DEV), 1 + 0.1 * torch.randn(R, d, generator=g, device=DEV)
    mats = (torch.randn(R, d, d, generator=g, device=DEV) / d ** 0.5).bfloat16()
    wq = torch.randn(R, d, d, generator=g, device=DEV) / d ** 0.5
    W8s = [ar.attnres_q8_weight(wq[r], ar.Q8Weight(d, d, device=DEV)) for r in range(R)]
    rows = ar.Q8Rows(R, T, d, device=DEV)
    reads, normed = torch.empty(R, T, d, device=DEV, dtype=torch.bfloat16), torch.empty(T, d, device=DEV, dtype=torch.bfloat16)
    Q = torch.empty(T, d, device=DEV)
    args = (W, Gamma, Pre, mats, W8s, rows, reads, normed, Q)
    model(x, *args)

    def check():
        assert ar.attnres_device_status() == 0
        v = values_of(rows)
        for r in range(R):
            q, extra = W[r], 0.0
            if r % 2:
                wv = _q8.values(W8s[r].codes, W8s[r].exponents.int() - 127, 128)
                q = v[r] @ wv.t()
                # the query's own error moves every score by at most |dq| |gamma v| / rms, each weight by twice that
                dq = (v[r].abs() @ wv.abs().t()) * ((d + 12) * _q8.U) + q.abs() * _q8.U
                size = (v[:r + 1].square().mean(-1) + 1e-6).sqrt()
                extra = 2 * ((v[:r + 1] * Gamma[r].double()).abs() * dq).sum(-1).div(size).amax(0).unsqueeze(-1)
                extra = extra * v[:r + 1].abs().amax(0)
            z, dz, _, _ = _q8.read(v[:r + 1], q, Gamma[r], 1e-6)
            _q8.assert_within(reads[r], z, dz + extra, f"read {r}")

    check()
    first = reads.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model(x, *args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model(x, *args)
    rows.buffer.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(reads, first)
    x.copy_(torch.randn(T, d, generator=g, device=DEV))
    graph.replay()
    check()
    # the backward: the history's exact values in bf16, then the Full read's backward
    V = torch.empty(R, T, d, device=DEV, dtype=torch.bfloat16)
    ar.attnres_q8_read(rows, V)
    dz = torch.randn(T, d, generator=g, device=DEV)
    dV, dw, dg = torch.zeros(R, T, d, device=DEV), torch.zeros(d, device=DEV), torch.zeros(d, device=DEV)
    ar.attnres_full_bwd(V, R, W[4], Gamma[4], 1e-6, dz, dV, dw, dg)
    v = values_of(rows)
    leaves = [t.double().clone().requires_grad_() for t in (v, W[4], Gamma[4])]
    e = (leaves[0] * (leaves[1] * leaves[2])).sum(-1) / (leaves[0].square().mean(-1) + 1e-6).sqrt()
    ((torch.softmax(e, 0).unsqueeze(-1) * leaves[0]).sum(0) * dz.double()).sum().backward()
    for got, leaf in ((dV, leaves[0]), (dw, leaves[1]), (dg, leaves[2])):
        assert float((got.double() - leaf.grad).abs().max()) <= 1e-5 * float(leaf.grad.abs().max())


def test_streams():
    """Calls on a stream of their own while another stream is busy, ordered by that stream alone."""
    n, T, d = 5, 3000, 896
    x = _q8.history(n, T, d, gen(1), DEV)
    w, gamma = torch.randn(d, generator=gen(2), device=DEV) * 0.1, torch.ones(d, device=DEV)
    rows, want = ar.Q8Rows(n, T, d, device=DEV), torch.empty(T, d, device=DEV)
    ar.attnres_q8_write(x, rows)
    ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, want)
    other, got = ar.Q8Rows(n, T, d, device=DEV), torch.empty(T, d, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ar.attnres_q8_write(x, other, stream=s)
    ar.attnres_full_fwd_q8(other, n, w, gamma, 1e-6, got, stream=s)
    ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, torch.empty(T, d, device=DEV))
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(other.buffer, rows.buffer)


def test_binding_refusals():
    rows = ar.Q8Rows(3, 8, 256, device=DEV)
    x, w = torch.zeros(8, 256, device=DEV), torch.zeros(256, device=DEV)
    W8 = ar.Q8Weight(64, 256, device=DEV)
    bad = [lambda: ar.attnres_q8_write(torch.zeros(9, 256, device=DEV), rows),
           lambda: ar.attnres_q8_write(x, rows, src=3),
           lambda: ar.attnres_q8_write(x, rows, src=-1),
           lambda: ar.attnres_q8_write(torch.zeros(8, 255, device=DEV), rows),
           lambda: ar.attnres_q8_write(torch.zeros(4, 8, 256, device=DEV), rows),
           lambda: ar.attnres_q8_write(torch.zeros(8, 512, device=DEV)[:, ::2], rows),
           lambda: ar.attnres_q8_write(torch.zeros(8, 256), rows),
           lambda: ar.attnres_q8_read(rows, torch.zeros(2, 8, 256, device=DEV), src=2),
           lambda: ar.attnres_full_fwd_q8(rows, 4, w, w, 1e-6, x),
           lambda: ar.attnres_full_fwd_q8(rows, 0, w, w, 1e-6, x),
           lambda: ar.attnres_full_fwd_q8(rows, 3, w, w, 1e-6, None),
           lambda: ar.attnres_full_fwd_q8(rows, 3, w[:8], w, 1e-6, x),
           lambda: ar.attnres_full_fwd_q8(rows, 3, None, w, 1e-6, x, Q=torch.zeros(7, 256, device=DEV)),
           lambda: ar.attnres_full_fwd_q8(rows, 3, w, w, 1e-6, x, gamma_pre=w, out_normed=x.bfloat16()),
           lambda: ar.attnres_full_fwd_q8(rows, 3, w, w, 1e-6, x.t().contiguous().t()),
           lambda: ar.attnres_query_projection_q8(rows, 3, W8, torch.zeros(8, 64, device=DEV)),
           lambda: ar.attnres_query_projection_q8(rows, 0, W8, torch.zeros(8, 63, device=DEV)),
           lambda: ar.attnres_query_projection_q8(rows, 0, W8, torch.zeros(9, 64, device=DEV)),
           lambda: ar.attnres_query_projection_q8(rows, 0, ar.Q8Weight(64, 128, device=DEV), torch.zeros(8, 64, device=DEV)),
           lambda: ar.attnres_q8_weight(torch.zeros(64, 255, device=DEV), W8),
           lambda: ar.Q8Rows(0, 8, 256, device=DEV)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(TypeError):
        ar.attnres_q8_write(x.half(), rows)
    for call in (lambda: ar.attnres_full_fwd_q8(rows, 3, w, w, 1e-6, x, Q=x + 1),     # both queries
                 lambda: ar.attnres_full_fwd_q8(rows, 3, None, w, 1e-6, x),           # none
                 lambda: ar.attnres_full_fwd_q8(rows, 3, w, w, 1e-6, x, gamma_pre=w)):  # a pre-norm without its output
        with pytest.raises(ar.AttnResError):
            call()
    empty = ar.Q8Rows(3, 0, 256, device=DEV)
    ar.attnres_q8_write(x[:0], empty)
    ar.attnres_full_fwd_q8(empty, 3, w, w, 1e-6, x[:0])
    ar.attnres_query_projection_q8(empty, 0, W8, torch.zeros(0, 64, device=DEV))


# The stages of a CTA: 2 where the warps (and CTAs) that share a token take 16 sources (and 128) at once.
@pytest.mark.parametrize("index", [0, 1, 3])
@pytest.mark.parametrize("n,T,d,stages", [(9, 80000, 256, 4), (20, 1, 640, 2), (13, 6000, 2048, 4), (141, 2, 640, 2)])
def test_a_copy_that_never_arrives(n, T, d, stages, index):
    """A withheld copy ends the kernel with a timeout on record, and the next call is right again."""
    rows, v = made(n, T, d, gen(1))
    w, gamma = torch.randn(d, generator=gen(2), device=DEV) * 0.1, torch.ones(d, device=DEV)
    want, out = torch.empty(T, d, device=DEV), torch.empty(T, d, device=DEV)
    ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, want)
    assert ar.attnres_device_status() == 0
    binding.attnres_test_withhold_stage(binding.WITHHOLD_Q8_READ, index)
    try:
        ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, out)
        status = ar.attnres_device_status()
    finally:
        binding.attnres_test_withhold_stage(binding.WITHHOLD_NONE)
    assert status == (4 if index < stages else 0)
    ar.attnres_full_fwd_q8(rows, n, w, gamma, 1e-6, out)
    assert ar.attnres_device_status() == 0 and torch.equal(out, want)
