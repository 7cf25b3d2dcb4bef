"""Cases for the operators of a layer of experts between its products, and for its weights in 4 bits:

  layer_norm   layer norm in front of the projections: forward, backward with the gradients of
               weight and bias, or both
  route        the router's choice of k experts for each token with its gates, and its gradient
  dispatch     (token, choice) pairs sorted by expert, and the tokens' rows brought into that order
  combine      the experts' rows back, weighted by the gates (or summed: the gradient of dispatch),
               and the gradients of rows and gates
  round_trip   dispatch and combine of one decoding batch
  int4_*       quantisation of weights to 4 bits with a scale per group and back, and products of
               few rows with such weights, plain and grouped by expert

``run`` computes a case in plain torch operations in 32 bits (``own`` false) or through the
framework's entry points (``own`` true); ``exact`` gives the same from the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
INF = float("inf")


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # decoding, 16 sequences: the norm in front of a projection, latency
        dict(name="layer_norm_decode", op="layer_norm", what="fwd", T=16, C=4096, x32=False, g32=False, w32=True, out32=False),
        # a training step over an odd number of tokens, the residual stream in FP32
        dict(name="layer_norm_step", op="layer_norm", what="both", T=16173, C=1024, x32=True, g32=False, w32=True, out32=True),
        # training: the backward pass in BF16
        dict(name="layer_norm_bwd_train", op="layer_norm", what="bwd", T=16384, C=4096, x32=False, g32=False, w32=False, out32=False),
        # decoding: the choice of 8 of 64 experts for 8 sequences, latency
        dict(name="route_decode", op="route", what="fwd", T=8, E=64, k=8, renormalize=True, masked=0.0, padding=0.0, ties=False),
        # training: 8 of 256 experts with the softmax over all of them, some experts closed and some tokens padding
        dict(name="route_train", op="route", what="both", T=16384, E=256, k=8, renormalize=False, masked=0.05, padding=0.02, ties=True),
        # one decoding batch through sort, dispatch and combine: 8 sequences, 8 experts each
        dict(name="round_trip_decode", op="round_trip", T=8, k=8, E=64, C=4096, skew=0.3, dropped=0.0),
        # training: 16384 pairs over 64 experts, rows of the wide side
        dict(name="dispatch_train", op="dispatch", T=2048, k=8, E=64, C=4096, skew=0.5, dropped=0.01, f32=False),
        # training: the way back with its gradients, BF16 rows
        dict(name="combine_train", op="combine", what="both", T=2048, k=8, E=64, C=4096, skew=0.5, dropped=0.01, y32=False, out32=False,
             gates=True, add=True),
        # the wide projection's weights quantised, and expanded again for the many rows of a prefill
        dict(name="int4_quantize", op="int4_quantize", N=12288, K=4096, group=128, zeros=True, w32=False, s32=False),
        # decoding one sequence through the wide projection: bound by the 4-bit weights
        dict(name="int4_fwd_single", op="int4_fwd", T=1, N=12288, K=4096, group=128, zeros=False, s32=False, f32=False),
        # decoding 16 sequences through the square projection, small groups with zero points
        dict(name="int4_fwd_batch", op="int4_fwd", T=16, N=4096, K=4096, group=32, zeros=True, s32=False, f32=True),
        # one decoding batch over 64 experts: 64 rows, bound by the weights of the experts that have rows
        dict(name="int4_grouped_decode", op="int4_grouped", rows=64, pad=0, E=64, N=1024, K=4096, skew=0.3, group=128, zeros=True,
             s32=False, f32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _dim(rng, lo, hi, multiple):
    return max(multiple, _log(rng, lo, hi) // multiple * multiple)


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm", "route", "dispatch", "combine", "round_trip", "int4_quantize", "int4_fwd", "int4_fwd",
                     "int4_grouped"])
    if op == "layer_norm":
        C = _dim(rng, 64, 16384, 8)
        return dict(op=op, what=rng.choice(["fwd", "bwd", "both"]), T=_log(rng, 1, min(16384, (1 << 25) // C)), C=C, x32=rng.random() < 0.4,
                    g32=rng.random() < 0.3, w32=rng.random() < 0.5, out32=rng.random() < 0.3)
    if op == "route":
        E = _log(rng, 2, 512)
        return dict(op=op, what=rng.choice(["fwd", "both"]), T=_log(rng, 1, 16384), E=E, k=_log(rng, 1, min(E, 16)),
                    renormalize=rng.random() < 0.5, masked=rng.choice([0.0, 0.1, 0.6]), padding=rng.choice([0.0, 0.1]),
                    ties=rng.random() < 0.3)
    if op in ("dispatch", "combine", "round_trip"):
        C, k = _dim(rng, 64, 8192, 8), _log(rng, 1, 12)
        c = dict(op=op, T=_log(rng, 1, min(16384, (1 << 24) // (C * k)) if op == "round_trip" else min(65536, (1 << 25) // (C * k))), k=k,
                 E=_log(rng, max(2, k), 512), C=C, skew=round(rng.uniform(0.0, 1.0), 3), dropped=rng.choice([0.0, 0.0, 0.05, 0.5]))
        if op == "dispatch":
            c.update(f32=rng.random() < 0.3)
        if op == "combine":
            c.update(what=rng.choice(["fwd", "both"]), y32=rng.random() < 0.3, out32=rng.random() < 0.4, gates=rng.random() < 0.7,
                     add=rng.random() < 0.5)
        return c
    group = rng.choice([32, 64, 128])
    c = dict(op=op, K=_dim(rng, 128, 8192, group), group=group, zeros=rng.random() < 0.5, s32=rng.random() < 0.3)
    if op == "int4_quantize":
        return dict(c, N=_dim(rng, 8, min(12288, (1 << 25) // c["K"]), 8), w32=rng.random() < 0.3)
    if op == "int4_fwd":
        return dict(c, T=_log(rng, 1, 64), N=_dim(rng, 8, min(16384, (1 << 26) // c["K"]), 8), f32=rng.random() < 0.3)
    N = _dim(rng, 64, 4096, 8)
    return dict(c, rows=_log(rng, 1, 256), pad=rng.choice([0, 0, rng.randrange(1, 40)]), E=_log(rng, 1, max(1, min(256, (1 << 28) // (N * c["K"])))), N=N,
                skew=round(rng.uniform(0.0, 1.0), 3), f32=rng.random() < 0.3)


# ----------------------------------------------------------------------- inputs

def _gen(seed, role, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 64 + role)
    return g


def _normal(shape, seed, role, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, device="cuda", generator=_gen(seed, role)) * scale).to(dtype)


def _uniform(shape, seed, role):
    return torch.rand(shape, device="cuda", generator=_gen(seed, role))


def _activations(shape, seed, role, dtype=torch.bfloat16):
    """N(0.1, 1) with a few feature columns ten times larger, as activations have."""
    x = torch.randn(shape, device="cuda", generator=_gen(seed, role)) + 0.1
    hot = _uniform((shape[-1],), seed, role + 32) < 0.01
    return torch.where(hot, x * 10, x).to(dtype)


def _type(f32):
    return torch.float32 if f32 else torch.bfloat16


def _choices(case, seed):
    """k different experts for each token, from a skewed distribution; pairs that are dropped have -1."""
    T, E, k = case["T"], case["E"], case["k"]
    bias = torch.randn(E, device="cuda", generator=_gen(seed, 1)) * case["skew"]
    score = torch.randn((T, E), device="cuda", generator=_gen(seed, 2)) + bias
    choice = score.topk(k, dim=1).indices.int()
    return torch.where(_uniform((T, k), seed, 3) < case["dropped"], -1, choice)


def _groups(case, seed):
    """Rows per expert: tokens pick experts from a skewed distribution; some get none."""
    g = _gen(seed, 1, "cpu")
    p = torch.softmax(torch.randn(case["E"], generator=g) * case["skew"], 0)
    picks = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    return torch.bincount(picks, minlength=case["E"]).tolist()


def _weights(shape, seed):
    return _normal(shape, seed, 4, 1.0 / math.sqrt(shape[-1]), torch.float32)


def prepare(case, seed):
    op = case["op"]
    s = {"case": case}
    if op == "layer_norm":
        T, C = case["T"], case["C"]
        s["x"] = _activations((T, C), seed, 1, _type(case["x32"]))
        s["w"] = (1 + _normal((C,), seed, 2, 0.2, torch.float32)).to(_type(case["w32"]))
        s["b"] = _normal((C,), seed, 3, 0.1, _type(case["w32"]))
        if case["what"] != "fwd":
            s["dy"] = _normal((T, C), seed, 4, 1e-2, _type(case["g32"]))
        if case["what"] == "bwd":  # what the forward pass saved
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = ((x - s["mean"][:, None]).square().mean(1) + EPS).rsqrt()
        return s
    if op == "route":
        T, E = case["T"], case["E"]
        logits = torch.randn((T, E), device="cuda", generator=_gen(seed, 1)) * 1.5
        logits = logits.bfloat16().float() if case["ties"] else logits
        closed = _uniform((E,), seed, 2) < case["masked"]
        away = _uniform((T,), seed, 3) < case["padding"]
        s["logits"] = torch.where(closed[None, :] | away[:, None], -INF, logits)
        s["d_gates"] = _normal((T, case["k"]), seed, 4, 1e-2, torch.float32)
        return s
    if op in ("dispatch", "combine", "round_trip"):
        T, k, C = case["T"], case["k"], case["C"]
        s["choice"] = _choices(case, seed)
        if op != "combine":
            s["x"] = _activations((T, C), seed, 5, _type(case.get("f32", False)))
        if op != "dispatch":
            gates = _uniform((T, k), seed, 6) + 0.05
            s["gates"] = gates / gates.sum(1, keepdim=True)
            s["y"] = _normal((T * k, C), seed, 7, 1.0, _type(case.get("y32", False)))  # what the experts made of the rows
        if op == "combine":  # the forward pass has sorted the pairs
            s["row_of"] = _sort(s["choice"], case["E"])[1]
            s["d_out"] = _normal((T, C), seed, 8, 1e-2, _type(case["out32"]))
            s["add"] = _normal((T, C), seed, 9, 1.0, _type(case["out32"])) if case["add"] else None
            s["gates"] = s["gates"] if case["gates"] else None
        return s
    if op == "int4_quantize":
        s["W"] = _weights((case["N"], case["K"]), seed).to(_type(case["w32"]))
        return s
    if op == "int4_fwd":
        s["X"] = _activations((case["T"], case["K"]), seed, 2)
        s["q"], s["s"], s["z"] = _encode(_weights((case["N"], case["K"]), seed), case)
        return s
    counts = _groups(case, seed)
    edges = [case["pad"] // 3]  # part of the padding in front, the rest behind
    for c in counts:
        edges.append(edges[-1] + c)
    T, E = case["rows"] + case["pad"], case["E"]
    s.update(edges=edges, T=T, widest=max(counts), offsets=torch.tensor(edges, dtype=torch.int32, device="cuda"),
             X=_activations((T, case["K"]), seed, 2))
    s["q"], s["s"], s["z"] = _encode(_weights((E, case["N"], case["K"]), seed), case)
    return s


# ------------------------------------------------------------------ plain forms

def _norm(x):
    """(mean, 1 / standard deviation, normalised rows) in 32 bits."""
    x = x.float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = (d.square().mean(1) + EPS).rsqrt()
    return mean, rstd, d * rstd[:, None]


def _plain_layer_norm(s):
    case, out = s["case"], {}
    dtype = _type(case["out32"])
    w = s["w"].float()
    if case["what"] != "bwd":
        mean, rstd, xh = _norm(s["x"])
        out.update(y=(xh * w + s["b"].float()).to(dtype), mean=mean, rstd=rstd)
    if case["what"] != "fwd":
        if case["what"] == "bwd":
            rstd = s["rstd"]
            xh = (s["x"].float() - s["mean"][:, None]) * rstd[:, None]
        dy = s["dy"].float()
        g = dy * w
        dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * rstd[:, None]
        out.update(dx=dx.to(dtype), dw=(dy * xh).sum(0), db=dy.sum(0))
    return out


def _gates(logits, k, renormalize):
    """(gates, choice): the k largest, the lowest index first among equals; -1 and 0 where all are closed."""
    top, choice = logits.sort(dim=1, descending=True, stable=True)
    top, choice = top[:, :k], choice[:, :k].int()
    most = torch.where(top[:, :1] == -INF, 0.0, top[:, :1])
    e = (top - most).exp()
    total = (e if renormalize else (logits - most).exp()).sum(1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0), torch.where(top == -INF, -1, choice)


def _plain_route(s):
    case, logits = s["case"], s["logits"]
    gates, choice = _gates(logits, case["k"], case["renormalize"])
    out = {"gates": gates, "choice": choice}
    if case["what"] == "both":
        inner = (s["d_gates"] * gates).sum(1, keepdim=True)
        at = choice.long().clamp_min(0)
        if case["renormalize"]:
            d = torch.zeros_like(logits).scatter_add_(1, at, gates * (s["d_gates"] - inner))
        else:
            most = logits.amax(1, keepdim=True)
            e = (logits - torch.where(most == -INF, 0.0, most)).exp()
            total = e.sum(1, keepdim=True)
            p = torch.where(total > 0, e / total, 0.0)
            d = (-p * inner).scatter_add_(1, at, gates * s["d_gates"])
        out["d_logits"] = d
    return out


def _sort(choice, E):
    """(offsets, row of each pair, pair of each row); pairs without an expert follow the last group, their rows as ~row."""
    flat = choice.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = key.argsort(stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=order.device)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    return offsets, torch.where(key < E, row, ~row).int().view(choice.shape), order.int()


def _gather(x, row_of):
    T, k = row_of.shape
    at = row_of.flatten().long()
    rows = torch.empty((T * k, x.shape[1]), dtype=x.dtype, device=x.device)
    rows[torch.where(at < 0, ~at, at)] = torch.where((at >= 0)[:, None], x.repeat_interleave(k, 0), 0)
    return rows


def _combine(y, row_of, gates, add, dtype):
    T, k = row_of.shape
    at = row_of.long()
    w = torch.ones(T, k, device=y.device) if gates is None else gates
    w = torch.where(at >= 0, w, 0.0)
    out = (y[at.clamp_min(0).flatten()].float().view(T, k, -1) * w[:, :, None]).sum(1)
    return (out if add is None else out + add.float()).to(dtype)


def _combine_bwd(d_out, y, row_of, gates):
    T, k = row_of.shape
    at = row_of.flatten().long()
    have = (at >= 0)[:, None]
    place = torch.where(at < 0, ~at, at)
    d = d_out.float().repeat_interleave(k, 0)
    d_y = torch.empty_like(y)
    d_y[place] = torch.where(have, d * gates.flatten()[:, None], 0.0).to(y.dtype)
    d_gates = torch.where(have, d * y[place].float(), 0.0).sum(1)
    return d_y, d_gates.view(T, k)


def _encode(W, case):
    """4-bit codes (two to a byte, the even column in the low half), scales and zero points of groups along the rows:
    w is about (q - z) s, with z = 8 and s = max|w| / 7, or both from the range of w and 0."""
    kind = _type(case["s32"])
    g = W.float().unflatten(-1, (-1, case["group"]))
    if case["zeros"]:
        lo, hi = g.amin(-1).clamp_max(0.0), g.amax(-1).clamp_min(0.0)
        s = ((hi - lo) / torch.full_like(hi, 15.0)).clamp_min(1e-30).to(kind)
        z = (-lo / s.float()).round().clamp_(0, 15)
    else:
        s = (g.abs().amax(-1) / torch.full_like(g[..., 0], 7.0)).clamp_min(1e-30).to(kind)
        z = torch.full_like(s, 8.0, dtype=torch.float32)
    q = ((g / s.float()[..., None]).round() + z[..., None]).clamp_(0, 15).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), s, z.to(torch.uint8) if case["zeros"] else None


def _codes(q):
    return torch.stack((q & 15, q >> 4), -1).flatten(-2)


def _decode(q, s, z, group):
    q = _codes(q).float().unflatten(-1, (-1, group))
    return ((q - (8.0 if z is None else z.float()[..., None])) * s.float()[..., None]).flatten(-2)


def _places(s):
    start = s["offsets"][:-1].long()
    count = (s["offsets"][1:] - s["offsets"][:-1]).long()
    i = torch.arange(s["widest"], device="cuda")
    ok = i[None, :] < count[:, None]
    return torch.where(ok, start[:, None] + i[None, :], 0), ok


def _plain_grouped(s):
    case = s["case"]
    at, ok = _places(s)
    rows = torch.where(ok[:, :, None], s["X"][at.view(-1)].view(*at.shape, -1).float(), 0.0)
    y = rows @ _decode(s["q"], s["s"], s["z"], case["group"]).transpose(1, 2)
    out = torch.zeros(s["T"] + 1, y.shape[-1], device="cuda")
    out[torch.where(ok, at, s["T"]).view(-1)] = y.view(-1, y.shape[-1])
    return out[:-1].to(_type(case["f32"]))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "layer_norm":
        return _plain_layer_norm(s)
    if op == "route":
        return _plain_route(s)
    if op in ("dispatch", "round_trip"):
        offsets, row_of, order = _sort(s["choice"], case["E"])
        rows = _gather(s["x"], row_of)
        out = {"offsets": offsets, "row_of": row_of, "order": order, "rows": rows}
        if op == "round_trip":
            out["out"] = _combine(s["y"], row_of, s["gates"], None, torch.bfloat16)
        return out
    if op == "combine":
        out = {"out": _combine(s["y"], s["row_of"], s["gates"], s["add"], _type(case["out32"]))}
        if case["what"] == "both" and case["gates"]:
            out["d_y"], out["d_gates"] = _combine_bwd(s["d_out"], s["y"], s["row_of"], s["gates"])
        return out
    if op == "int4_quantize":
        q, scales, z = _encode(s["W"], case)
        return {"W": _decode(q, scales, z, case["group"]).to(s["W"].dtype), "s": scales, "z": z}
    if op == "int4_fwd":
        return (s["X"].float() @ _decode(s["q"], s["s"], s["z"], case["group"]).T).to(_type(case["f32"]))
    return _plain_grouped(s)


def run(s):
    if not own:
        return _plain(s)
    import fp32_dense_projection_gb300 as dp
    case = s["case"]
    op = case["op"]
    if op == "layer_norm":
        out, dtype = {}, _type(case["out32"])
        mean, rstd = s.get("mean"), s.get("rstd")
        if case["what"] != "bwd":
            y, mean, rstd = dp.layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS, out_dtype=dtype)
            out.update(y=y, mean=mean, rstd=rstd)
        if case["what"] != "fwd":
            out["dx"], out["dw"], out["db"] = dp.layer_norm_bwd(s["dy"], s["x"], mean, rstd, s["w"], dx_dtype=dtype)
        return out
    if op == "route":
        gates, choice = dp.route_topk(s["logits"], case["k"], renormalize=case["renormalize"])
        out = {"gates": gates, "choice": choice}
        if case["what"] == "both":
            out["d_logits"] = dp.route_topk_bwd(s["d_gates"], s["logits"], gates, choice, renormalize=case["renormalize"])
        return out
    if op in ("dispatch", "round_trip"):
        offsets, row_of, order = dp.expert_sort(s["choice"], case["E"])
        rows = dp.expert_gather(s["x"], row_of)
        out = {"offsets": offsets, "row_of": row_of, "order": order, "rows": rows}
        if op == "round_trip":
            out["out"] = dp.expert_combine(s["y"], row_of, s["gates"])
        return out
    if op == "combine":
        out = {"out": dp.expert_combine(s["y"], s["row_of"], s["gates"], add=s["add"], out_dtype=_type(case["out32"]))}
        if case["what"] == "both" and case["gates"]:
            out["d_y"], out["d_gates"] = dp.expert_combine_bwd(s["d_out"], s["y"], s["row_of"], s["gates"], dy_dtype=_type(case["y32"]))
        return out
    if op == "int4_quantize":
        q, scales, z = dp.int4_quantize(s["W"], case["group"], zeros=case["zeros"], scale_dtype=_type(case["s32"]))
        return {"W": dp.int4_dequantize(q, scales, zeros=z, out_dtype=s["W"].dtype), "s": scales, "z": z}
    dtype = _type(case["f32"])
    if op == "int4_fwd":
        return dp.dp_gemm_fwd_int4(s["X"], s["q"], s["s"], zeros=s["z"], out_dtype=dtype)
    return dp.dp_gemm_fwd_int4_grouped(s["X"], s["q"], s["s"], s["offsets"], zeros=s["z"], out_dtype=dtype)


# ------------------------------------------------------------------------- work

def _size(f32):
    return 4 if f32 else 2


def work(case):
    op = case["op"]
    if op == "layer_norm":
        n, o, what = case["T"] * case["C"], _size(case["out32"]), case["what"]
        each = _size(case["x32"]) + (o if what != "bwd" else 0) + (_size(case["g32"]) + o if what != "fwd" else 0)
        params = case["C"] * (_size(case["w32"]) * (1 if what == "bwd" else 2) + (0 if what == "fwd" else 8))
        return {"bytes": n * each + 8 * case["T"] + params, "flops": n * {"fwd": 8, "bwd": 14, "both": 20}[what]}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        both = case["what"] == "both"
        return {"bytes": 4 * T * E * (2 if both else 1) + T * k * (12 if both else 8), "flops": T * E * (4 if both else 2)}
    if op in ("dispatch", "combine", "round_trip"):
        T, k, C = case["T"], case["k"], case["C"]
        if op == "combine":
            both, o, y = case["what"] == "both" and case["gates"], _size(case["out32"]), _size(case["y32"])
            moved = T * k * C * y + T * C * o * (2 if case["add"] else 1) + (T * C * o + T * k * C * y if both else 0)
            return {"bytes": moved + T * k * (12 if both else 8 if case["gates"] else 4), "flops": T * k * C * (6 if both else 2)}
        b = _size(case.get("f32", False))
        moved = T * C * b * (1 + k) + T * k * 12 + 4 * (case["E"] + 1)
        return {"bytes": moved + (2 * T * C * (1 + k) + T * k * 4 if op == "round_trip" else 0), "flops": T * k * C * 2 if op == "round_trip" else T * k}
    N, K, G = case["N"], case["K"], case["group"]
    codes = N * K // 2 + N * (K // G) * (_size(case["s32"]) + case["zeros"])
    if op == "int4_quantize":
        return {"bytes": 2 * N * K * _size(case["w32"]) + codes, "flops": 6 * N * K}
    if op == "int4_fwd":
        return {"bytes": codes + case["T"] * (2 * K + N * _size(case["f32"])), "flops": 2 * case["T"] * N * K}
    R, E = case["rows"], case["E"]
    busy = E * (1 - (1 - 1 / E) ** R)  # experts with rows, on average
    return {"bytes": busy * codes + 2 * R * K + (R + case["pad"]) * N * _size(case["f32"]) + 4 * (E + 1), "flops": 2 * R * N * K}


# ------------------------------------------------------- the definitions, 64 bits

def _exact_pairs(choice, E):
    """Offsets and rows by counting: the pairs of each expert in order, those without one last."""
    flat = choice.flatten().tolist()
    lists = [[] for _ in range(E + 1)]
    for i, e in enumerate(flat):
        lists[e if 0 <= e < E else E].append(i)
    order = [i for group in lists for i in group]
    edges = [0]
    for group in lists[:E]:
        edges.append(edges[-1] + len(group))
    row_of = [0] * len(flat)
    for r, i in enumerate(order):
        row_of[i] = r if r < edges[-1] else -1 - r
    made = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (edges, row_of, order)]
    return made[0], made[1].view(choice.shape), made[2]


def _nibbles(q):
    n = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=torch.float64, device=q.device)
    n[..., 0::2], n[..., 1::2] = q % 16, q // 16
    return n


def _meant(s, at, group):
    """The weights that codes, scales and zero points of one matrix stand for."""
    q, sc, z = ((v if at is None else v[at]) if v is not None else None for v in (s["q"], s["s"], s["z"]))
    z = torch.full(sc.shape, 8.0, dtype=torch.float64, device="cuda") if z is None else z.double()
    return (_nibbles(q) - z.repeat_interleave(group, -1)) * sc.double().repeat_interleave(group, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "layer_norm":
        x, w = s["x"].double(), s["w"].double()
        out = {}
        mean = x.sum(1) / case["C"]
        rstd = 1 / torch.sqrt((x * x).sum(1) / case["C"] - mean * mean + EPS)
        if case["what"] != "bwd":
            out.update(y=((x - mean[:, None]) * rstd[:, None]) * w + s["b"].double(), mean=mean, rstd=rstd)
        else:
            mean, rstd = s["mean"].double(), s["rstd"].double()
        if case["what"] != "fwd":
            xh, dy = (x - mean[:, None]) * rstd[:, None], s["dy"].double()
            a = torch.einsum("tc,c->t", dy, w) / case["C"]
            b = torch.einsum("tc,tc,c->t", dy, xh, w) / case["C"]
            out.update(dx=rstd[:, None] * (dy * w - a[:, None] - b[:, None] * xh), dw=torch.einsum("tc,tc->c", dy, xh), db=dy.sum(0))
        return out
    if op == "route":
        l, k = s["logits"].double(), case["k"]
        T, E = l.shape
        rest, gates, choice = l.clone(), [], []
        for _ in range(k):  # the largest of what is left, the lowest index among equals
            most = rest.amax(1, keepdim=True)
            at = torch.where(rest == most, torch.arange(E, device="cuda"), E).amin(1, keepdim=True)
            live = most > -INF
            gates.append(torch.where(live, most, -INF))
            choice.append(torch.where(live, at, -1))
            rest = rest.scatter(1, at, -INF)
        v, choice = torch.cat(gates, 1), torch.cat(choice, 1)
        norm = torch.logsumexp(v if case["renormalize"] else l, 1, keepdim=True)
        gates = torch.where(choice >= 0, (v - norm).exp(), 0.0)
        out = {"gates": gates, "choice": choice.int()}
        if case["what"] == "both":
            dg = torch.where(choice >= 0, s["d_gates"].double(), 0.0)
            full = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")  # d of each expert's gate; closed choices go to a spare column
            full.scatter_(1, torch.where(choice >= 0, choice, E), dg)
            p = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
            if case["renormalize"]:
                p.scatter_(1, torch.where(choice >= 0, choice, E), gates)
            else:
                p[:, :E] = torch.where(norm > -INF, (l - norm).exp(), 0.0)
            out["d_logits"] = (p * (full - (p * full).sum(1, keepdim=True)))[:, :E]
        return out
    if op in ("dispatch", "round_trip"):
        offsets, row_of, order = _exact_pairs(s["choice"], case["E"])
        have = torch.arange(order.numel(), device="cuda") < offsets[-1]
        rows = s["x"].double()[order.long() // case["k"]] * have[:, None]
        out = {"offsets": offsets, "row_of": row_of, "order": order, "rows": rows}
        if op == "round_trip":
            total = torch.zeros(case["T"], case["C"], dtype=torch.float64, device="cuda")
            weighted = s["y"].double() * s["gates"].double().flatten()[order.long()][:, None] * have[:, None]
            out["out"] = total.index_add_(0, order.long() // case["k"], weighted)
        return out
    if op == "combine":
        row_of, y = s["row_of"].long(), s["y"].double()
        total = torch.zeros(case["T"], case["C"], dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()
        gates = torch.ones(row_of.shape, dtype=torch.float64, device="cuda") if s["gates"] is None else s["gates"].double()
        d_y, d_gates, d = torch.zeros_like(y), torch.zeros_like(gates), s["d_out"].double()
        for j in range(case["k"]):
            t = (row_of[:, j] >= 0).nonzero()[:, 0]
            r = row_of[t, j]
            total[t] += gates[t, j][:, None] * y[r]
            d_y[r] = gates[t, j][:, None] * d[t]
            d_gates[t, j] = torch.einsum("tc,tc->t", d[t], y[r])
        out = {"out": total}
        if case["what"] == "both" and case["gates"]:
            out.update(d_y=d_y, d_gates=d_gates)
        return out
    if op == "int4_quantize":
        top = s["W"].double().view(case["N"], -1, case["group"])
        if case["zeros"]:
            scale = (top.amax(2).clamp_min(0) - top.amin(2).clamp_max(0)) / 15
            return {"W": None, "s": scale.clamp_min(1e-30), "z": None}
        return {"W": None, "s": (top.abs().amax(2) / 7).clamp_min(1e-30)}  # (the codes are a choice of rounding, not a value of 64 bits)
    if op == "int4_fwd":
        return s["X"].double() @ _meant(s, None, case["group"]).T
    out = torch.zeros(s["T"], case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, b = s["edges"][e], s["edges"][e + 1]
        if b > a:
            out[a:b] = s["X"][a:b].double() @ _meant(s, e, case["group"]).T
    return out
