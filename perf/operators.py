"""Cases of the training and residual-stream operators, for timing and comparison.

Five operators next to the AttnRes reads: the gated residual (a sublayer's post-norm, gate, residual scale and
add, with the next sublayer's pre-norm) and its backward, the backward of RMSNorm, the global norm of a list of
gradients, and clipping by it. `run` computes them in plain torch operations in fp32, or, with `own` set, by
the library's entry points.
"""
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS_POST, EPS_PRE = 1e-6, 1e-5


def _residual(name, T, d, dtype, x, gate, gate_rows, scale, **more):
    return {"name": name, "op": "gated_residual", "T": T, "d": d, "dtype": dtype, "x": x, "gate": gate,
            "gate_rows": gate_rows, "scale": scale, **more}


def _residual_bwd(name, T, d, dtype, x, dx, gate, gate_rows, scale, **more):
    return {**_residual(name, T, d, dtype, x, gate, gate_rows, scale, **more), "op": "gated_residual_bwd", "dx": dx}


def listed():
    return [
        # One decoding step of 8 requests: post-norm and residual scale, then the next pre-norm. Latency counts.
        _residual("residual_decode", 8, 2048, "bf16", "bf16", "none", 1, 0.5),
        # A training batch of 4 x 2048 tokens on the fp32 running sum of a block, with a sigmoid gate per element.
        _residual("residual_block_sum", 8192, 896, "bf16", "f32", "sigmoid", 1, 1.0),
        # A 128K-token prefill with a learned gain per feature in place of the gate.
        _residual("residual_prefill", 131072, 2048, "bf16", "bf16", "identity", 131072, 1.0),
        # A small fp32 model: the whole step is a few microseconds of work.
        _residual_bwd("residual_bwd_small", 256, 256, "f32", "f32", "f32", "identity", 256, 0.7),
        # The backward of the training batch above.
        _residual_bwd("residual_bwd_block_sum", 8192, 896, "bf16", "f32", "f32", "sigmoid", 1, 1.0),
        # A ragged batch whose sequences of 2048 tokens each have one gate row (conditioning), the last one short.
        _residual_bwd("residual_bwd_ragged", 32749, 640, "bf16", "bf16", "f32", "identity", 2048, 0.25),
        # The pre-norm's backward over a batch of the 8 x 8 Block model, joining the fp32 gradient of the stream.
        {"name": "rmsnorm_bwd_batch", "op": "rmsnorm_bwd", "T": 16384, "d": 1024, "dtype": "bf16", "dx": "f32",
         "join": True},
        # A wide model, a short odd batch, no gradient to join.
        {"name": "rmsnorm_bwd_wide", "op": "rmsnorm_bwd", "T": 1021, "d": 8192, "dtype": "bf16", "dx": "bf16",
         "join": False},
        # The pseudo-queries and key gains of 64 reads alone: 128 short fp32 vectors. Latency counts.
        {"name": "norm_queries", "op": "grad_norm", "tensors": 128, "elements": 128 * 896, "dtype": "f32"},
        # Every gradient of a 400M-parameter model, stored as bf16.
        {"name": "norm_model", "op": "grad_norm", "tensors": 291, "elements": 400_000_000, "dtype": "bf16"},
        # A shard's gradients, matrices in bf16 and gains in fp32, small enough to stay in the cache between the
        # two readings.
        {"name": "clip_shard", "op": "grad_clip", "tensors": 75, "elements": 24_000_001, "dtype": "mixed", "out": "same"},
        # fp32 gradient accumulators of an 800M-parameter model, clipped into the optimiser's bf16 gradients.
        {"name": "clip_model", "op": "grad_clip", "tensors": 339, "elements": 800_000_000, "dtype": "f32", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["gated_residual", "gated_residual_bwd", "gated_residual_bwd", "rmsnorm_bwd", "grad_norm", "grad_clip"])
    if op in ("grad_norm", "grad_clip"):
        dtype = rng.choice(["f32", "bf16", "mixed"])
        case = {"op": op, "tensors": _log(rng, 1, 600), "elements": _log(rng, 50_000, 300_000_000), "dtype": dtype}
        if op == "grad_clip":
            case["out"] = rng.choice(["same", "bf16"]) if dtype == "f32" else "same"
        return case
    d = 8 * _log(rng, 16, 1024)
    T = _log(rng, 1, min(65536, 60_000_000 // d))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    wide = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
    grad = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
    if op == "rmsnorm_bwd":
        return {"op": op, "T": T, "d": d, "dtype": dtype, "dx": grad, "join": rng.random() < 0.5}
    gate = rng.choice(["none", "sigmoid", "identity"])
    rows = rng.choice([1, 1, T, _log(rng, 1, T), 2048])
    case = {"op": op, "T": T, "d": d, "dtype": dtype, "x": wide, "gate": gate, "gate_rows": rows,
            "scale": round(rng.uniform(0.1, 1.0), 3)}
    if op == "gated_residual_bwd":
        case["dx"] = grad
    return case


def _gate_type(case):
    """A gate per token is an activation in the storage type; one that tokens share is a parameter in fp32."""
    return case["dtype"] if case["gate_rows"] == 1 else "f32"


def _sizes(case):
    """Elements of each gradient: matrices and gains in turn, as layers have them, the last taking what is left."""
    n, total = case["tensors"], case["elements"]
    if case["elements"] == n * 896:
        return [896] * n
    gains = [max(1, min(total // (4 * n), 2048) - i % 7) if i % 3 == 2 else 0 for i in range(n)]
    matrices = [i for i in range(n) if not gains[i]]
    left = total - sum(gains)
    each = left // len(matrices)
    sizes = list(gains)
    for i in matrices:
        sizes[i] = each
    sizes[matrices[-1]] += left - each * len(matrices)
    return sizes


def _kinds(case, sizes):
    if case["dtype"] != "mixed":
        return [case["dtype"]] * len(sizes)
    return ["f32" if i % 3 == 2 else "bf16" for i in range(len(sizes))]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _generator(seed)

    def normal(shape, dtype, std=1.0, mean=0.0):
        x = torch.randn(shape, generator=g, device="cuda")
        return x.mul_(std).add_(mean).to(TYPES[dtype])

    s = {"case": case}
    if case["op"] in ("grad_norm", "grad_clip"):
        sizes = _sizes(case)
        kinds = _kinds(case, sizes)
        # Buckets by type, each gradient on a boundary of 64 elements, as gradient buckets are laid out.
        ends = {k: 0 for k in sorted(set(kinds))}
        where = []
        for n, k in zip(sizes, kinds):
            where.append((k, ends[k], n))
            ends[k] += -(-n // 64) * 64
        out_kind = {k: k if case.get("out", "same") == "same" else case["out"] for k in ends}
        s["flat"] = {k: torch.zeros(n, device="cuda", dtype=TYPES[k]) for k, n in ends.items()}
        s["grads"] = [s["flat"][k][a:a + n] for k, a, n in where]
        for i, t in enumerate(s["grads"]):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").mul_(10.0 ** (-(i % 4))))
        s["max_norm"] = 1.0
        s["norm"] = torch.empty(1, device="cuda")
        if case["op"] == "grad_clip":
            s["out"] = {k: torch.zeros(n, device="cuda", dtype=TYPES[out_kind[k]]) for k, n in ends.items()}
            s["outs"] = [s["out"][k][a:a + n] for k, a, n in where]
        if own:
            import depth_wise_attention_attnres_gb300 as ar
            s["grad_list"] = ar.GradList(s["grads"], s.get("outs"))
            s["scratch"] = torch.empty(ar.attnres_grad_norm_scratch_floats(len(sizes)), device="cuda")
        return s

    T, d = case["T"], case["d"]
    if case["op"] == "rmsnorm_bwd":
        s["x"] = normal((T, d), case["dtype"], 2.0)
        s["gamma"] = normal((d,), "f32", 0.1, 1.0)
        s["dy"] = normal((T, d), case["dtype"], 0.01)
        s["dres"] = normal((T, d), case["dx"], 0.02) if case["join"] else None
        s["dx"] = torch.empty(T, d, device="cuda", dtype=TYPES[case["dx"]])
        s["dgamma"] = torch.empty(d, device="cuda")
    else:
        s["f"] = normal((T, d), case["dtype"], 1.5)
        s["gamma_post"] = normal((d,), "f32", 0.1, 1.0)
        s["gamma_pre"] = normal((d,), "f32", 0.1, 1.0)
        groups = -(-T // case["gate_rows"])
        kind = _gate_type(case)
        s["gate"] = (None if case["gate"] == "none" else normal((groups, d), kind) if case["gate"] == "sigmoid" else
                     normal((groups, d), kind, 0.2, 0.8))
        # The stream's values (backward: those the forward left) grow with depth; 3.0 is some ten sublayers' sum.
        s["x"] = normal((T, d), case["x"], 3.0)
        if case["op"] == "gated_residual":
            s["x_out"] = torch.empty_like(s["x"])
            s["normed"] = torch.empty_like(s["f"])
        else:
            s["dx_out"] = normal((T, d), case["dx"], 0.02)
            s["dnormed"] = normal((T, d), case["dtype"], 0.01)
            s["df"] = torch.empty_like(s["f"])
            s["dx"] = torch.empty_like(s["dx_out"])
            s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
            s["dgamma_post"] = torch.empty(d, device="cuda")
            s["dgamma_pre"] = torch.empty(d, device="cuda")
    if own and case["op"] != "gated_residual":
        import depth_wise_attention_attnres_gb300 as ar
        floats = (ar.attnres_rmsnorm_bwd_scratch_floats(T, d) if case["op"] == "rmsnorm_bwd" else
                  ar.attnres_gated_residual_bwd_scratch_floats(T, d, case["gate_rows"]))
        s["scratch"] = torch.empty(floats, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms ----

def _rms(x, eps):
    return torch.rsqrt(x.square().mean(1, keepdim=True) + eps)


def _per_token(rows, T, gate_rows):
    """Gate rows [groups, d] as one row per token."""
    if rows.shape[0] == 1 or gate_rows == 1:
        return rows
    return rows[torch.arange(T, device=rows.device) // gate_rows]


def _norm_bwd(x, gamma, eps, dy):
    """Gradient of gamma * x / rms(x) with respect to x, and each token's share of gamma's."""
    r = _rms(x, eps)
    xh = x * r
    h = gamma * dy
    return r * (h - xh * (h * xh).mean(1, keepdim=True)), dy * xh


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("grad_norm", "grad_clip"):
        wide = [t.float() for t in s["flat"].values()]
        norm = torch.stack([t.square().sum() for t in wide]).sum().sqrt()
        if op == "grad_norm":
            return {"norm": norm.reshape(1)}
        coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
        return {"norm": norm.reshape(1), "out": {k: (t * coef).to(s["out"][k].dtype) for k, t in zip(s["flat"], wide)}}
    T = case["T"]
    if op == "rmsnorm_bwd":
        dx, share = _norm_bwd(s["x"].float(), s["gamma"], EPS_PRE, s["dy"].float())
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(s["dx"].dtype), "dgamma": share.sum(0)}
    f, scale = s["f"].float(), case["scale"]
    fh = f * _rms(f, EPS_POST)
    y = s["gamma_post"] * fh
    gate = None if s["gate"] is None else s["gate"].float()
    act = gate.sigmoid() if case["gate"] == "sigmoid" else gate
    a = scale if act is None else scale * _per_token(act, T, case["gate_rows"])
    if op == "gated_residual":
        x = s["x"].float() + a * y
        return {"x_out": x.to(s["x"].dtype), "normed": (s["gamma_pre"] * x * _rms(x, EPS_PRE)).to(s["f"].dtype)}
    dx, pre = _norm_bwd(s["x"].float(), s["gamma_pre"], EPS_PRE, s["dnormed"].float())
    dx = dx + s["dx_out"].float()
    dy = a * dx
    df, post = _norm_bwd(f, s["gamma_post"], EPS_POST, dy)
    out = {"df": df.to(s["f"].dtype), "dx": dx.to(s["dx"].dtype), "dgamma_post": post.sum(0), "dgamma_pre": pre.sum(0)}
    if act is not None:
        share = scale * y * dx
        rows, groups = case["gate_rows"], gate.shape[0]
        if groups == 1:
            share = share.sum(0, keepdim=True)
        elif rows > 1:
            pad = groups * rows - T
            share = torch.nn.functional.pad(share, (0, 0, 0, pad)).view(groups, rows, -1).sum(1)
        out["dgate"] = (share * act * (1 - act) if case["gate"] == "sigmoid" else share).to(s["gate"].dtype)
    return out


# ---------------------------------------------------------- the library's calls ----

def _own(s):
    import depth_wise_attention_attnres_gb300 as ar
    case = s["case"]
    op = case["op"]
    if op == "grad_norm":
        ar.attnres_grad_norm(s["grad_list"], s["norm"], scratch=s["scratch"])
        return {"norm": s["norm"]}
    if op == "grad_clip":
        ar.attnres_grad_clip(s["grad_list"], s["max_norm"], s["norm"], scratch=s["scratch"])
        return {"norm": s["norm"], "out": s["out"]}
    if op == "rmsnorm_bwd":
        ar.attnres_rmsnorm_bwd(s["x"], s["gamma"], EPS_PRE, s["dy"], s["dres"], s["dx"], s["dgamma"], accumulate=False,
                               scratch=s["scratch"])
        return {"dx": s["dx"], "dgamma": s["dgamma"]}
    act = ar.GATE_SIGMOID if case["gate"] == "sigmoid" else ar.GATE_IDENTITY
    if op == "gated_residual":
        ar.attnres_gated_residual(s["f"], s["x"], s["gamma_post"], EPS_POST, s["gate"], case["gate_rows"], act, case["scale"],
                                  s["x_out"], s["gamma_pre"], EPS_PRE, s["normed"])
        return {"x_out": s["x_out"], "normed": s["normed"]}
    ar.attnres_gated_residual_bwd(s["f"], s["gamma_post"], EPS_POST, s["gate"], case["gate_rows"], act, case["scale"], s["x"],
                                  s["gamma_pre"], EPS_PRE, s["dx_out"], s["dnormed"], s["df"], s["dx"], s["dgate"],
                                  s["dgamma_post"], s["dgamma_pre"], accumulate=False, scratch=s["scratch"])
    out = {k: s[k] for k in ("df", "dx", "dgamma_post", "dgamma_pre")}
    if s["dgate"] is not None:
        out["dgate"] = s["dgate"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op in ("grad_norm", "grad_clip"):
        sizes = _sizes(case)
        kinds = _kinds(case, sizes)
        nbytes = sum(n * SIZE[k] for n, k in zip(sizes, kinds))
        if op == "grad_clip":
            nbytes += sum(n * SIZE[k if case["out"] == "same" else case["out"]] for n, k in zip(sizes, kinds))
        return {"bytes": nbytes + 4, "flops": (2 if op == "grad_norm" else 3) * sum(sizes)}
    E, d, es = case["T"] * case["d"], case["d"], SIZE[case["dtype"]]
    if op == "rmsnorm_bwd":
        per = 2 * es + SIZE[case["dx"]] * (2 if case["join"] else 1)
        return {"bytes": E * per + 8 * d, "flops": 14 * E}
    gate = 0
    if case["gate"] != "none":
        gate = -(-case["T"] // case["gate_rows"]) * d * SIZE[_gate_type(case)]
    if op == "gated_residual":
        return {"bytes": E * (2 * es + 2 * SIZE[case["x"]]) + gate + 8 * d, "flops": 12 * E}
    per = 3 * es + SIZE[case["x"]] + 2 * SIZE[case["dx"]]
    return {"bytes": E * per + 2 * gate + 16 * d, "flops": 34 * E}


# ------------------------------------------------------------------- in 64 bits ----

def exact(case, seed):
    """The definitions in fp64, a slab of tokens (or one gradient) at a time; gradients by the chain rule written
    through the normalised rows' projections."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op in ("grad_norm", "grad_clip"):
        total = sum((float(torch.dot(p, p)) for t in s["grads"] for p in (q.double() for q in t.split(1 << 26))))
        norm = total ** 0.5
        ans = {"norm": torch.tensor([norm], dtype=f64, device="cuda")}
        if op == "grad_clip":
            by = min(1.0, s["max_norm"] / norm) if norm > 0 else 1.0
            ans["out"] = {k: t.to(f64).mul_(by) for k, t in s["flat"].items()}
        return ans
    T, d = case["T"], case["d"]
    slab = max(1, (1 << 25) // d)
    new = lambda *shape: torch.zeros(shape, dtype=f64, device="cuda")  # noqa: E731

    def unit(v, eps):
        size = ((v * v).sum(1, keepdim=True) / d + eps).sqrt()
        return v / size, size

    if op == "rmsnorm_bwd":
        ans = {"dx": new(T, d), "dgamma": new(d)}
        for a in range(0, T, slab):
            b = min(T, a + slab)
            u, size = unit(s["x"][a:b].to(f64), EPS_PRE)
            dy = s["dy"][a:b].to(f64)
            w = dy * s["gamma"].to(f64)
            ans["dx"][a:b] = (w - u * ((w * u).sum(1, keepdim=True) / d)) / size
            if s["dres"] is not None:
                ans["dx"][a:b] += s["dres"][a:b].to(f64)
            ans["dgamma"] += (dy * u).sum(0)
        return ans
    scale, rows = case["scale"], case["gate_rows"]
    gp, gn = s["gamma_post"].to(f64), s["gamma_pre"].to(f64)
    ans = ({"x_out": new(T, d), "normed": new(T, d)} if op == "gated_residual" else
           {"df": new(T, d), "dx": new(T, d), "dgamma_post": new(d), "dgamma_pre": new(d)})
    if s["gate"] is not None and op == "gated_residual_bwd":
        ans["dgate"] = new(*s["gate"].shape)
    for a in range(0, T, slab):
        b = min(T, a + slab)
        u, size = unit(s["f"][a:b].to(f64), EPS_POST)
        at = torch.arange(a, b, device="cuda") // rows
        gain, slope = torch.ones(1, 1, dtype=f64, device="cuda"), torch.ones(1, 1, dtype=f64, device="cuda")
        if s["gate"] is not None:
            logits = s["gate"].to(f64)[at] if s["gate"].shape[0] > 1 else s["gate"].to(f64)
            if case["gate"] == "sigmoid":
                gain = 1 / (1 + torch.exp(-logits))
                slope = torch.exp(-logits) * gain * gain
            else:
                gain = logits
        if op == "gated_residual":
            x = s["x"][a:b].to(f64) + scale * gain * gp * u
            ans["x_out"][a:b] = x
            ans["normed"][a:b] = gn * unit(x, EPS_PRE)[0]
            continue
        v, big = unit(s["x"][a:b].to(f64), EPS_PRE)
        dn = s["dnormed"][a:b].to(f64)
        w = dn * gn
        D = s["dx_out"][a:b].to(f64) + (w - v * ((w * v).sum(1, keepdim=True) / d)) / big
        ans["dx"][a:b] = D
        ans["dgamma_pre"] += (dn * v).sum(0)
        dm = scale * D
        w = dm * gain * gp
        ans["df"][a:b] = (w - u * ((w * u).sum(1, keepdim=True) / d)) / size
        ans["dgamma_post"] += (dm * gain * u).sum(0)
        if s["gate"] is not None:
            share = (dm * gp * u * slope).expand(b - a, d)
            if s["gate"].shape[0] == 1:
                ans["dgate"][0] += share.sum(0)
            else:
                ans["dgate"].index_add_(0, at, share)
    return ans
