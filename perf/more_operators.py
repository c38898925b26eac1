"""Cases of the 8-bit depth history, for timing and comparison.

Four operators. Rows of features are held in e4m3 with one power-of-two scale for each group of 128 features:
writing them (sources of an AttnRes history, or hidden states), reading them back, the Full read over a history of
such rows, and the projection of the input-dependent query, rows times a weight matrix in e4m3 with one scale for
each block of 128 x 128. `run` computes them in plain torch operations in fp32, or, with `own` set, by the
library's entry points.
"""
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
GROUP = 128
EPS, EPS_PRE = 1e-6, 1e-5


def listed():
    return [
        # One decoding step of 8 requests: a sublayer's output enters the history. Latency counts.
        {"name": "write_decode", "op": "write", "n": 1, "T": 8, "d": 2048, "dtype": "bf16"},
        # Sources kept in fp32 until now, moved over: an odd batch, a width that is no multiple of the group.
        {"name": "write_odd", "op": "write", "n": 3, "T": 8191, "d": 1000, "dtype": "f32"},
        # A sublayer's output of a 128K-token prefill.
        {"name": "write_prefill", "op": "write", "n": 1, "T": 131072, "d": 2048, "dtype": "bf16"},
        # A few sources back in fp32, for a look at them or for another program; odd sizes.
        {"name": "back_odd", "op": "back", "n": 5, "T": 1021, "d": 648, "dtype": "f32"},
        # The whole history of a 64-read model as bf16 (which holds its values exactly), as the backward takes it.
        {"name": "back_batch", "op": "back", "n": 64, "T": 8192, "d": 896, "dtype": "bf16"},
        # The last read of a 141-read model for a single token. Latency counts.
        {"name": "read_token", "op": "read", "n": 141, "T": 1, "d": 640, "dtype": "bf16", "query": "fixed", "pre": False},
        # An odd batch with a query for each token, fp32 results.
        {"name": "read_odd", "op": "read", "n": 17, "T": 4999, "d": 1000, "dtype": "f32", "query": "token", "pre": False},
        # The last read of a 64-read model over a training batch, with the consumer's pre-norm.
        {"name": "read_batch", "op": "read", "n": 64, "T": 8192, "d": 896, "dtype": "bf16", "query": "fixed", "pre": True},
        # The embedding and 8 block summaries of a 128K-token prefill.
        {"name": "read_prefill", "op": "read", "n": 9, "T": 131072, "d": 2048, "dtype": "bf16", "query": "fixed", "pre": False},
        # The queries of one decoding step of 8 requests. Latency counts.
        {"name": "projection_decode", "op": "projection", "T": 8, "d": 2048, "out": 2048},
        # The queries of a training batch.
        {"name": "projection_batch", "op": "projection", "T": 8192, "d": 896, "out": 896},
        # The queries of a ragged prefill of a wide model.
        {"name": "projection_prefill", "op": "projection", "T": 32749, "d": 2048, "out": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _width(rng):
    """A model width: a multiple of the group, of 8, or any."""
    d = _log(rng, 64, 2048)
    return rng.choice([max(GROUP, d // GROUP * GROUP), d // 8 * 8, d])


def draw(rng):
    op = rng.choice(["write", "back", "read", "read", "projection"])
    d = _width(rng)
    if op == "projection":
        return {"op": op, "T": _log(rng, 1, 32768), "d": d, "out": rng.choice([d, d, _width(rng)])}
    n = _log(rng, 1, 141) if op == "read" else _log(rng, 1, 16)
    T = _log(rng, 1, min(131072, 500_000_000 // (n * d)))
    case = {"op": op, "n": n, "T": T, "d": d, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "read":
        case |= {"query": rng.choice(["fixed", "fixed", "token"]), "pre": rng.random() < 0.4}
    return case


# ----------------------------------------------------------------- inputs ----

def _rows(g, n, T, d):
    """Sublayer outputs: their size differs by source, and a few features are far larger than the others."""
    x = torch.randn(n, T, d, generator=g, device="cuda")
    loud = 1 + 15 * (torch.rand(d, generator=g, device="cuda") < 0.01)
    size = torch.exp(0.5 * torch.randn(n, 1, 1, generator=g, device="cuda"))
    return x.mul_(size).mul_(loud)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T, d = case["op"], case["T"], case["d"]
    s = {"case": case}
    if op == "write":
        s["x"] = _rows(g, case["n"], T, d).to(TYPES[case["dtype"]])
    else:
        s["codes"], s["exponents"] = _quantise_rows(_rows(g, case.get("n", 1), T, d))
    if op == "back":
        s["out"] = torch.empty(case["n"], T, d, device="cuda", dtype=TYPES[case["dtype"]])
    if op == "read":
        s["gamma"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        shape = (T, d) if case["query"] == "token" else (d,)
        s["query"] = torch.randn(shape, generator=g, device="cuda") * (1.5 / d ** 0.5)
        s["out"] = torch.empty(T, d, device="cuda", dtype=TYPES[case["dtype"]])
        if case["pre"]:
            s["gamma_pre"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
            s["normed"] = torch.empty_like(s["out"])
    if op == "projection":
        s["W"] = _quantise_blocks(torch.randn(case["out"], d, generator=g, device="cuda") / d ** 0.5)
        s["Q"] = torch.empty(T, case["out"], device="cuda")
    if own:
        import depth_wise_attention_attnres_gb300 as ar
        s["rows"] = ar.Q8Rows(case.get("n", 1), T, d, device="cuda")
        if op != "write":
            s["rows"].codes.view(torch.uint8).copy_(s["codes"].view(torch.uint8))
            s["rows"].exponents.copy_(s["exponents"])
            s["rows"].mean_square.copy_(_dequantise_rows(s["codes"], s["exponents"]).square().mean(-1))
        if op == "projection":
            s["weight"] = ar.Q8Weight(case["out"], d, device="cuda")
            s["weight"].codes.view(torch.uint8).copy_(s["W"][0].view(torch.uint8))
            s["weight"].exponents.copy_(s["W"][1])
    return s


# ------------------------------------------------------------ plain forms ----

def _exponent(amax):
    """The biased exponent of the smallest power of two by which `amax` (fp32) divided is at most 448."""
    bits = amax.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=1)


def _power(e):
    """2^(e - 127) as fp32, for a biased exponent e from 1 to 254."""
    return (e.int() << 23).view(torch.float32)


def _encode(y, e):
    """y 2^(127 - e) as e4m3; the largest code of the largest exponent is 240, so that its value stays finite."""
    top = torch.where(e == 247, 240.0, 448.0)
    return (y * _power(254 - e)).clamp(-top, top).to(torch.float8_e4m3fn)


def _quantise_rows(x):
    """x [n, T, d] as codes [n, T, d] and biased exponents [n, T, ceil(d / 128)]."""
    n, T, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -d % GROUP)).view(n, T, -1, GROUP)
    e = _exponent(x.abs().amax(-1))
    return _encode(x, e.unsqueeze(-1)).view(n, T, -1)[..., :d].contiguous(), e.to(torch.uint8)


def _dequantise_rows(codes, e):
    return codes.float() * _power(e).repeat_interleave(GROUP, -1)[..., :codes.shape[-1]]


def _quantise_blocks(W):
    """W [m, d] as codes [m, d] and biased exponents [ceil(m / 128), ceil(d / 128)]."""
    m, d = W.shape
    W = torch.nn.functional.pad(W, (0, -d % GROUP, 0, -m % GROUP)).view(-1, GROUP, -(-d // GROUP), GROUP)
    e = _exponent(W.abs().amax(3).amax(1))
    codes = _encode(W, e[:, None, :, None]).view(W.shape[0] * GROUP, -1)[:m, :d].contiguous()
    return codes, e.to(torch.uint8)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "write":
        codes, e = _quantise_rows(s["x"])
        return {"codes": codes, "exponents": e, "mean_square": _dequantise_rows(codes, e).square().mean(-1)}
    v = _dequantise_rows(s["codes"], s["exponents"])
    if op == "back":
        return {"out": v.to(s["out"].dtype)}
    if op == "projection":
        codes, e = s["W"]
        scale = _power(e).repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)[:codes.shape[0], :codes.shape[1]]
        return {"Q": v[0] @ (codes.float() * scale).t()}
    score = (v * (s["query"] * s["gamma"])).sum(-1) * torch.rsqrt(v.square().mean(-1) + EPS)
    a = torch.exp(score - score.amax(0))
    z = ((a / a.sum(0)).unsqueeze(-1) * v).sum(0)
    out = {"out": z.to(s["out"].dtype)}
    if case["pre"]:
        out["normed"] = (s["gamma_pre"] * z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS_PRE)).to(s["out"].dtype)
    return out


# ---------------------------------------------------- the library's calls ----

def _own(s):
    import depth_wise_attention_attnres_gb300 as ar
    case, rows = s["case"], s["rows"]
    op = case["op"]
    if op == "write":
        ar.attnres_q8_write(s["x"], rows)
        return {"codes": rows.codes, "exponents": rows.exponents, "mean_square": rows.mean_square}
    if op == "back":
        ar.attnres_q8_read(rows, s["out"])
        return {"out": s["out"]}
    if op == "projection":
        ar.attnres_query_projection_q8(rows, 0, s["weight"], s["Q"])
        return {"Q": s["Q"]}
    w, Q = (None, s["query"]) if case["query"] == "token" else (s["query"], None)
    if not case["pre"]:
        ar.attnres_full_fwd_q8(rows, case["n"], w, s["gamma"], EPS, s["out"], Q=Q)
        return {"out": s["out"]}
    ar.attnres_full_fwd_q8(rows, case["n"], w, s["gamma"], EPS, s["out"], Q=Q, gamma_pre=s["gamma_pre"], eps_pre=EPS_PRE,
                           out_normed=s["normed"])
    return {"out": s["out"], "normed": s["normed"]}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, T, d = case["op"], case["T"], case["d"]
    row = d + -(-d // GROUP)  # codes and exponents
    if op == "projection":
        m = case["out"]
        return {"bytes": T * row + m * d + -(-m // GROUP) * -(-d // GROUP) + 4 * T * m, "flops": 2 * T * d * m}
    n, es = case["n"], SIZE[case["dtype"]]
    if op == "write":
        return {"bytes": n * T * (d * es + row + 4), "flops": 5 * n * T * d}
    if op == "back":
        return {"bytes": n * T * (d * es + row), "flops": n * T * d}
    nbytes = n * T * row + T * d * es * (2 if case["pre"] else 1) + 4 * d * (2 if case["pre"] else 1)
    nbytes += 4 * T * d if case["query"] == "token" else 4 * d
    return {"bytes": nbytes, "flops": 6 * n * T * d}


# ------------------------------------------------------------- in 64 bits ----

def _round_e4m3(y):
    """The e4m3 number nearest to y (fp64), ties to the even one: three bits behind the leading one, no finer than 2^-9."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def _values(codes, e):
    """Codes times 2^(e - 127) of their group in the last axis, in fp64."""
    group = torch.arange(codes.shape[-1], device=codes.device) // GROUP
    return codes.double() * torch.exp2(e.double() - 127)[..., group]


def exact(case, seed):
    """The definitions in fp64, a slab of tokens at a time."""
    s = prepare(case, seed)
    op, T, d = case["op"], case["T"], case["d"]
    n = case.get("n", 1)
    groups = -(-d // GROUP)
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    slab = max(1, (1 << 27) // (n * d))
    if op == "write":
        ans = {"codes": new(n, T, d), "exponents": torch.zeros(n, T, groups, dtype=torch.uint8, device="cuda"),
               "mean_square": new(n, T)}
    elif op == "projection":
        codes, e = s["W"]
        per_row = e[torch.arange(case["out"], device="cuda") // GROUP]
        Wt = _values(codes, per_row).t()
        ans = {"Q": new(T, case["out"])}
    else:
        ans = {"out": new(n, T, d) if op == "back" else new(T, d)}
        if case.get("pre"):
            ans["normed"] = new(T, d)
    for a in range(0, T, slab):
        b = min(T, a + slab)
        if op == "write":
            for k in range(groups):
                at = slice(k * GROUP, min(d, (k + 1) * GROUP))
                x = s["x"][:, a:b, at].double()
                top = x.abs().amax(-1)
                m, e = torch.frexp(top / 448)
                # top / 448 = m 2^e with 1/2 <= m < 1: the power is e, or e - 1 for a power of two itself
                e = torch.where(m == 0.5, e - 1, e)
                e = torch.where(top > 0, e, -126).clamp(min=-126)
                scale = torch.exp2(e.double()).unsqueeze(-1)
                q = torch.minimum(_round_e4m3(x / scale).abs(), torch.where(e == 120, 240.0, 448.0).unsqueeze(-1)) * torch.sign(x)
                ans["codes"][:, a:b, at] = q
                ans["exponents"][:, a:b, k] = (e + 127).to(torch.uint8)
                ans["mean_square"][:, a:b] += (q * scale).square().sum(-1) / d
            continue
        v = _values(s["codes"][:, a:b], s["exponents"][:, a:b])
        if op == "back":
            ans["out"][:, a:b] = v
        elif op == "projection":
            ans["Q"][a:b] = v[0] @ Wt
        else:
            q = s["query"][a:b] if case["query"] == "token" else s["query"]
            q = q.double() * s["gamma"].double()
            size = (v.square().sum(-1) / d + EPS).sqrt()
            weight = torch.softmax((v * q).sum(-1) / size, 0)
            z = (weight.unsqueeze(-1) * v).sum(0)
            ans["out"][a:b] = z
            if case["pre"]:
                ans["normed"][a:b] = s["gamma_pre"].double() * z / (z.square().sum(-1, keepdim=True) / d + EPS_PRE).sqrt()
    return ans
