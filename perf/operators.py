"""Cases for the operators of a training or serving step around the projections:

  grouped_*   products of ragged row groups with their expert's weights (forward,
              input gradient, weight gradient), group offsets on the device
  fp8_*       8-bit quantisation with one scale per 128 values, and the products of
              quantised operands (forward, input gradient, weight gradient)
  adamw_*     the AdamW update of many tensors, moments in 32 or 8 bits

``run`` computes a case in plain torch operations in 32 bits (``own`` false) or
through the framework's entry points (``own`` true); ``exact`` gives the same from
the definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128           # values that share one scale
TINY = 1e-30          # smallest block maximum a scale is derived from
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.95, 1e-8, 3e-4, 0.1


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding batch of 8 sequences, 8 experts each: bound by the weights it touches
        dict(name="grouped_fwd_decode", op="grouped_fwd", rows=64, pad=0, E=64, N=1024, K=4096, skew=0.3, kn=False, f32=False),
        # a prefill chunk over few experts with an odd row count, a padded buffer and [K, N] weights
        dict(name="grouped_fwd_prefill", op="grouped_fwd", rows=4031, pad=65, E=32, N=1024, K=4096, skew=0.8, kn=True, f32=False),
        # training: 16384 rows over 64 experts, down-projection's input gradient
        dict(name="grouped_dgrad_train", op="grouped_dgrad", rows=16384, pad=0, E=64, N=4096, K=2048, skew=0.5, kn=False, f32=False),
        # training: the same layer's weight gradients in FP32, as an optimizer reads them
        dict(name="grouped_wgrad_train", op="grouped_wgrad", rows=16384, pad=0, E=64, N=4096, K=2048, skew=0.5, kn=False, f32=True),
        # activations quantised for the forward pass and the weight gradient from one read
        dict(name="fp8_quantize_train", op="fp8_quantize", T=16384, C=4096, scaling="both", fmt="e4m3", f32=False),
        # decoding through the wide projection: bound by the 8-bit weights
        dict(name="fp8_fwd_decode", op="fp8_fwd", T=16, N=12288, K=4096, fmt="e4m3", f32=False),
        # a ragged prefill chunk through the square projection
        dict(name="fp8_fwd_prefill", op="fp8_fwd", T=4031, N=4096, K=4096, fmt="e4m3", f32=False),
        # training: the wide projection's input gradient, gradients in e5m2
        dict(name="fp8_dgrad_train", op="fp8_dgrad", T=16384, N=12288, K=4096, fmt="e5m2", f32=False),
        # training: a weight gradient over an odd number of tokens, FP32 out
        dict(name="fp8_wgrad_train", op="fp8_wgrad", T=16173, N=1024, K=4096, fmt="e4m3", f32=True),
        # the biases and norm scales of a small model: latency
        dict(name="adamw_small", op="adamw", bits=32, tensors=24, base=4096, spread=0, bf16_param=False, bf16_grad=False, copies=False),
        # FP32 master weights of a few projections, BF16 gradients and BF16 working copies
        dict(name="adamw_master", op="adamw", bits=32, tensors=8, base=12288 * 4096 // 2, spread=4, bf16_param=False, bf16_grad=True, copies=True),
        # the same with moments in 8 bits
        dict(name="adamw_8bit", op="adamw", bits=8, tensors=8, base=12288 * 4096 // 2, spread=4, bf16_param=False, bf16_grad=True, copies=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi, multiple):
    return max(multiple, _log(rng, lo, hi) // multiple * multiple)


def draw(rng):
    op = rng.choice(["grouped_fwd", "grouped_dgrad", "grouped_wgrad", "fp8_quantize", "fp8_fwd", "fp8_dgrad", "fp8_wgrad",
                     "adamw", "adamw"])
    if op.startswith("grouped"):
        N, K = _dim(rng, 64, 6144, 8), _dim(rng, 64, 6144, 8)
        E = min(_log(rng, 1, 256), max(1, (1 << 29) // (N * K)))
        return dict(op=op, rows=_log(rng, 1, 16384), pad=rng.choice([0, 0, rng.randrange(1, 200)]), E=E, N=N, K=K,
                    skew=round(rng.uniform(0.0, 1.0), 3), kn=rng.random() < 0.3, f32=rng.random() < 0.3)
    if op == "fp8_quantize":
        return dict(op=op, T=_log(rng, 1, 16384), C=_dim(rng, 64, 4096, 16), scaling=rng.choice(["row", "col", "block", "both"]),
                    fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), f32=rng.random() < 0.3)
    if op.startswith("fp8"):
        return dict(op=op, T=_log(rng, 1, 16384), N=_dim(rng, 64, 12288, 16), K=_dim(rng, 64, 4096, 16),
                    fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), f32=rng.random() < 0.3)
    tensors = _log(rng, 1, 200)
    return dict(op=op, bits=rng.choice([8, 32]), tensors=tensors, base=_log(rng, 16, (1 << 27) // tensors), spread=rng.choice([0, 2, 6]),
                bf16_param=rng.random() < 0.3, bf16_grad=rng.random() < 0.6, copies=rng.random() < 0.5)


# ----------------------------------------------------------------------- inputs

def _gen(seed, role, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 64 + role)
    return g


def _normal(shape, seed, role, scale=1.0, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat, g = out.view(-1), _gen(seed, role)
    for lo in range(0, flat.numel(), 1 << 26):  # a chunk at a time: no second copy in 32 bits
        n = min(1 << 26, flat.numel() - lo)
        flat[lo:lo + n] = torch.randn(n, device="cuda", generator=g).mul_(scale)
    return out


def _groups(case, seed):
    """Rows per expert: tokens pick experts from a skewed distribution; some get none."""
    g = _gen(seed, 1, "cpu")
    p = torch.softmax(torch.randn(case["E"], generator=g) * case["skew"], 0)
    picks = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    return torch.bincount(picks, minlength=case["E"]).tolist()


def _activations(shape, seed, role):
    """N(0, 1) with a few feature columns ten times larger, as activations have."""
    x = _normal(shape, seed, role)
    hot = torch.rand(shape[-1], device="cuda", generator=_gen(seed, role + 32)) < 0.01
    return torch.where(hot, x * 10, x)


def prepare(case, seed):
    op = case["op"]
    if op.startswith("grouped"):
        counts = _groups(case, seed)
        first = case["pad"] // 3  # part of the padding in front, the rest behind
        edges = [first]
        for c in counts:
            edges.append(edges[-1] + c)
        T, E, N, K = case["rows"] + case["pad"], case["E"], case["N"], case["K"]
        s = {"case": case, "counts": counts, "edges": edges, "T": T, "widest": max(1, max(counts)),
             "offsets": torch.tensor(edges, dtype=torch.int32, device="cuda")}
        if op != "grouped_dgrad":
            s["X"] = _activations((T, K), seed, 2)
        if op != "grouped_fwd":
            s["dY"] = _normal((T, N), seed, 3)
        if op != "grouped_wgrad":
            s["W"] = _normal((E, K, N) if case["kn"] else (E, N, K), seed, 4, 1.0 / math.sqrt(K))
        return s
    if op == "fp8_quantize":
        x = _activations((case["T"], case["C"]), seed, 2)
        return {"case": case, "x": x.float() if case["f32"] else x}
    if op.startswith("fp8"):
        T, N, K = case["T"], case["N"], case["K"]
        s = {"case": case}
        if op == "fp8_fwd":
            s["a"] = _by_rows(*_quantize(_activations((T, K), seed, 2), "row", case["fmt"]))
            s["b"] = _quantize(_normal((N, K), seed, 4, 1.0 / math.sqrt(K)), "block", "e4m3")
        elif op == "fp8_dgrad":
            s["a"] = _by_rows(*_quantize(_normal((T, N), seed, 3), "row", case["fmt"]))
            s["b"] = _quantize(_normal((N, K), seed, 4, 1.0 / math.sqrt(K)), "block", "e4m3")
        else:
            s["a"] = _quantize(_normal((T, N), seed, 3), "col", case["fmt"])
            s["b"] = _quantize(_activations((T, K), seed, 2), "col", "e4m3")
        return s
    return _prepare_adamw(case, seed)


def _sizes(case):
    """Elements of each tensor: the base size, larger and odd by turns where `spread` says so."""
    return [case["base"] if not case["spread"] or i % 2 == 0 else max(1, case["base"] // (1 + i % (case["spread"] + 1)) - i)
            for i in range(case["tensors"])]


def _prepare_adamw(case, seed):
    sizes, starts, total = _sizes(case), [], 0
    for n in sizes:  # each tensor starts on a whole block of its buffer
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK
    p_type = torch.bfloat16 if case["bf16_param"] else torch.float32
    g_type = torch.bfloat16 if case["bf16_grad"] else torch.float32
    p = _normal((total,), seed, 1, 0.02, p_type)
    g = _normal((total,), seed, 2, 1e-3, g_type)
    m = _normal((total,), seed, 3, 3e-4, torch.float32)
    v = _normal((total,), seed, 4, 1e-3, torch.float32).square_()
    copies = p.to(torch.bfloat16) if case["copies"] else None
    s = {"case": case, "sizes": sizes, "starts": starts, "total": total, "step": 100, "p": p, "copies": copies,
         "clip": torch.full((1,), 0.5, device="cuda")}
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, n in zip(starts, sizes):
        live[a:a + n] = True
    if case["bits"] == 8:
        s["m"], s["ms"] = _encode(torch.where(live, m, 0))
        s["v"], s["vs"] = _encode(torch.where(live, v, 0).sqrt())
    else:
        s["m"], s["v"] = torch.where(live, m, 0), torch.where(live, v, 0)
    s["g"], s["live"] = torch.where(live, g, 0), live

    def cut(x, per=1):
        return [x[a // per:-(-(a + n) // per)] for a, n in zip(starts, sizes)]
    s["grads"] = cut(s["g"])
    if own:
        import fp32_dense_projection_gb300 as dp
        eight = case["bits"] == 8
        s["opt"] = dp.AdamW(cut(p), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, state_bits=case["bits"],
                            copies=cut(copies) if copies is not None else None, exp_avg=cut(s["m"]), exp_avg_sq=cut(s["v"]),
                            exp_avg_scale=cut(s["ms"], BLOCK) if eight else None,
                            exp_avg_sq_scale=cut(s["vs"], BLOCK) if eight else None, step=s["step"])
    return s


# ------------------------------------------------------------------ plain forms

def _padded(s, x):
    """[E, widest, columns] in 32 bits: each group's rows, zeros after them."""
    at, ok = _places(s)
    return torch.where(ok[:, :, None], x[at.view(-1)].view(*at.shape, -1).float(), 0.0)


def _places(s):
    start = s["offsets"][:-1].long()
    count = (s["offsets"][1:] - s["offsets"][:-1]).long()
    i = torch.arange(s["widest"], device="cuda")
    ok = i[None, :] < count[:, None]
    return torch.where(ok, start[:, None] + i[None, :], 0), ok


def _scattered(s, y):
    """The rows of the padded groups back in their places; zeros elsewhere."""
    at, ok = _places(s)
    out = torch.zeros(s["T"] + 1, y.shape[-1], device="cuda")
    out[torch.where(ok, at, s["T"]).view(-1)] = y.view(-1, y.shape[-1])
    return out[:-1]


def _scales(x, scaling, top):
    """Scale of each block: max(|x|, TINY) / top, and the factor top / max."""
    T, C = x.shape
    rows = BLOCK if scaling in ("col", "block") else 1
    cols = BLOCK if scaling in ("row", "block") else 1
    a = torch.nn.functional.pad(x.abs(), (0, -C % cols, 0, -T % rows))
    a = a.view(-(-T // rows), rows, -(-C // cols), cols).amax((1, 3)).clamp_min(TINY)
    factor = (top / a).repeat_interleave(rows, 0)[:T].repeat_interleave(cols, 1)[:, :C]
    return a / top, factor


def _quantize(x, scaling, fmt):
    kind, top = FP8[fmt]
    x = x.float()
    s, factor = _scales(x, scaling, top)
    return (x * factor).clamp_(-top, top).to(kind), s


def _by_rows(q, s):
    """Row scales as the framework's quantisation lays them out: a column's in one piece."""
    return q, s.t().contiguous().t()


def _dequantize(q, s, scaling):
    T, C = q.shape
    rows = BLOCK if scaling in ("col", "block") else 1
    cols = BLOCK if scaling in ("row", "block") else 1
    return q.float() * s.repeat_interleave(rows, 0)[:T].repeat_interleave(cols, 1)[:, :C]


def _encode(x):
    """E4M3 codes of a moment, a scale for each 128 values; what is over zero stays over zero."""
    top = FP8["e4m3"][1]
    a = x.view(-1, BLOCK).abs().amax(1).clamp_min(TINY)
    y = (x.view(-1, BLOCK) * (top / a)[:, None]).view(-1).clamp_(-top, top)
    return y.to(torch.float8_e4m3fn), a / top


def _decode(q, s):
    return (q.float().view(-1, BLOCK) * s[:, None]).view(-1)


def _single(x):
    """A number rounded to 32 bits."""
    return float(torch.tensor(x, dtype=torch.float32))


def _plain_adamw(s):
    """The update on the whole buffer; the padding between the tensors has zero gradients and is put back."""
    case, eight = s["case"], s["case"]["bits"] == 8
    s["step"] += 1
    t = s["step"]
    g = s["g"].float() * s["clip"]
    m = _decode(s["m"], s["ms"]) if eight else s["m"]
    v = _decode(s["v"], s["vs"]).square() if eight else s["v"]
    m = m * _single(BETA1) + g * _single(1 - BETA1)
    v = v * _single(BETA2) + (g * g) * _single(1 - BETA2)
    root = v.sqrt()
    p = s["p"].float() * _single(1 - LR * DECAY)
    p = p - (m / (root * _single(1 / math.sqrt(1 - BETA2 ** t)) + _single(EPS))) * _single(LR / (1 - BETA1 ** t))
    s["p"].copy_(torch.where(s["live"], p, s["p"].float()))
    if s["copies"] is not None:
        s["copies"].copy_(s["p"])
    if eight:
        q, ms = _encode(m)
        s["m"].copy_(q)
        s["ms"].copy_(ms)
        top = FP8["e4m3"][1]
        a = root.view(-1, BLOCK).amax(1).clamp_min(TINY)
        y = (root.view(-1, BLOCK) * (top / a)[:, None]).view(-1).clamp_(max=top)
        s["v"].copy_(torch.where(root > 0, y.clamp_min(2.0 ** -9), y).to(torch.float8_e4m3fn))
        s["vs"].copy_(a / top)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {k: s[k] for k in ("p", "copies", "m", "ms", "v", "vs") if s.get(k) is not None}


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op.startswith("grouped"):
        out = torch.float32 if case["f32"] else torch.bfloat16
        if op == "grouped_wgrad":
            a, b = _padded(s, s["dY"]), _padded(s, s["X"])
            return (b.transpose(1, 2) @ a if case["kn"] else a.transpose(1, 2) @ b).to(out)
        W = s["W"].float()
        if op == "grouped_fwd":
            return _scattered(s, _padded(s, s["X"]) @ (W if case["kn"] else W.transpose(1, 2))).to(out)
        return _scattered(s, _padded(s, s["dY"]) @ (W.transpose(1, 2) if case["kn"] else W)).to(out)
    if op == "fp8_quantize":
        kinds = ["row", "col"] if case["scaling"] == "both" else [case["scaling"]]
        return [t for k in kinds for t in _quantize(s["x"], k, case["fmt"])]
    if op.startswith("fp8"):
        out = torch.float32 if case["f32"] else torch.bfloat16
        if op == "fp8_wgrad":
            return (_dequantize(*s["a"], "col").T @ _dequantize(*s["b"], "col")).to(out)
        a, b = _dequantize(*s["a"], "row"), _dequantize(*s["b"], "block")
        return (a @ (b.T if op == "fp8_fwd" else b)).to(out)
    return _plain_adamw(s)


def run(s):
    if not own:
        return _plain(s)
    import fp32_dense_projection_gb300 as dp
    case = s["case"]
    op = case["op"]
    if op == "adamw":
        s["opt"].step(s["grads"], grad_scale=s["clip"])
        return _adamw_outputs(s)
    if op == "fp8_quantize":
        return list(dp.fp8_quantize(s["x"], scaling=case["scaling"], dtype=FP8[case["fmt"]][0]))
    out = torch.float32 if case["f32"] else torch.bfloat16
    if op == "fp8_fwd":
        return dp.dp_gemm_fwd_fp8(*s["a"], *s["b"], out_dtype=out)
    if op == "fp8_dgrad":
        return dp.dp_gemm_dgrad_fp8(*s["a"], *s["b"], out_dtype=out)
    if op == "fp8_wgrad":
        return dp.dp_gemm_wgrad_fp8(*s["a"], *s["b"], out_dtype=out)
    layout = "kn" if case["kn"] else "nk"
    if op == "grouped_fwd":
        return dp.dp_gemm_fwd_grouped(s["X"], s["W"], s["offsets"], out_dtype=out, weight_layout=layout)
    if op == "grouped_dgrad":
        return dp.dp_gemm_dgrad_grouped(s["dY"], s["W"], s["offsets"], out_dtype=out, weight_layout=layout)
    return dp.dp_gemm_wgrad_grouped(s["dY"], s["X"], s["offsets"], out_dtype=out, weight_layout=layout)


# ------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        moments = 4 + 16.0 / BLOCK if case["bits"] == 8 else 16
        each = (4 if case["bf16_param"] else 8) + (2 if case["bf16_grad"] else 4) + moments + (2 if case["copies"] else 0)
        return {"bytes": n * each, "flops": n * 16}
    if op == "fp8_quantize":
        n, T, C = case["T"] * case["C"], case["T"], case["C"]
        scales = {"row": T * -(-C // BLOCK), "col": -(-T // BLOCK) * C, "block": -(-T // BLOCK) * -(-C // BLOCK)}
        scales["both"] = scales["row"] + scales["col"]
        return {"bytes": n * ((4 if case["f32"] else 2) + (2 if case["scaling"] == "both" else 1)) + 4 * scales[case["scaling"]],
                "flops": 3 * n}
    size = 4 if case["f32"] else 2
    if op.startswith("fp8"):
        T, N, K = case["T"], case["N"], case["K"]
        read = {"fp8_fwd": T * K + N * K, "fp8_dgrad": T * N + N * K, "fp8_wgrad": T * (N + K)}[op]
        return {"bytes": read * (1 + 4 / BLOCK) + size * {"fp8_fwd": T * N, "fp8_dgrad": T * K, "fp8_wgrad": N * K}[op],
                "flops": 2 * T * N * K}
    R, T, E, N, K = case["rows"], case["rows"] + case["pad"], case["E"], case["N"], case["K"]
    busy = E * (1 - (1 - 1 / E) ** R)  # experts with rows, on average
    moved = {"grouped_fwd": 2 * R * K + 2 * busy * N * K + size * T * N, "grouped_dgrad": 2 * R * N + 2 * busy * N * K + size * T * K,
             "grouped_wgrad": 2 * R * (N + K) + size * E * N * K}[op]
    return {"bytes": moved + 4 * (E + 1), "flops": 2 * R * N * K}


# ------------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("grouped"):
        E, N, K, e = case["E"], case["N"], case["K"], s["edges"]
        if op == "grouped_wgrad":
            out = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
            for i in range(E):
                out[i] = s["dY"][e[i]:e[i + 1]].double().T @ s["X"][e[i]:e[i + 1]].double()
            return out.transpose(1, 2).contiguous() if case["kn"] else out
        rows = s["X"] if op == "grouped_fwd" else s["dY"]
        out = torch.zeros(s["T"], N if op == "grouped_fwd" else K, dtype=torch.float64, device="cuda")
        for i in range(E):
            W = s["W"][i].double()
            W = W.T if case["kn"] else W  # [N, K]
            out[e[i]:e[i + 1]] = rows[e[i]:e[i + 1]].double() @ (W.T if op == "grouped_fwd" else W)
        return out
    if op == "fp8_quantize":
        top = FP8[case["fmt"]][1]
        x, got = s["x"].double(), []
        for kind in (["row", "col"] if case["scaling"] == "both" else [case["scaling"]]):
            parts = [x] if kind == "row" else x.split(BLOCK, 0)
            if kind == "col":
                a = torch.stack([p.abs().amax(0) for p in parts])
            else:
                a = torch.cat([torch.stack([c.abs().amax(1) if kind == "row" else c.abs().max()[None] for c in p.split(BLOCK, 1)], 1)
                               for p in parts])
            got += [None, a.clamp_min(TINY) / top]  # (the codes are a choice of rounding, not a value of 64 bits)
        return got
    if op.startswith("fp8"):
        (qa, sa), (qb, sb) = s["a"], s["b"]
        T = qa.shape[0]
        total = 0
        if op == "fp8_wgrad":
            for k in range(0, T, BLOCK):
                a, b = qa[k:k + BLOCK].double() * sa[k // BLOCK].double(), qb[k:k + BLOCK].double() * sb[k // BLOCK].double()
                total = total + a.T @ b
            return total
        N, K = qb.shape
        wide = sb.double().repeat_interleave(BLOCK, 0)[:N]  # [N, K blocks]
        if op == "fp8_fwd":
            for k in range(0, K, BLOCK):
                total = total + (qa[:, k:k + BLOCK].double() * sa[:, k // BLOCK:k // BLOCK + 1].double()) @ \
                    (qb[:, k:k + BLOCK].double() * wide[:, k // BLOCK:k // BLOCK + 1]).T
            return total
        wide = wide.repeat_interleave(BLOCK, 1)[:, :K]
        for n in range(0, N, BLOCK):
            total = total + (qa[:, n:n + BLOCK].double() * sa[:, n // BLOCK:n // BLOCK + 1].double()) @ \
                (qb[n:n + BLOCK].double() * wide[n:n + BLOCK])
        return total
    t, g = s["step"] + 1, s["g"].double() * s["clip"].double()
    if case["bits"] == 8:
        m = s["m"].double() * s["ms"].double().repeat_interleave(BLOCK)
        v = (s["v"].double() * s["vs"].double().repeat_interleave(BLOCK)) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    p = s["p"].double()
    p = torch.where(s["live"], p - LR * DECAY * p - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS), p)
    got = {"p": p, "copies": p if case["copies"] else None}
    if case["bits"] == 8:
        top = FP8["e4m3"][1]
        got.update(m=None, ms=m.view(-1, BLOCK).abs().amax(1).clamp_min(TINY) / top,
                   v=None, vs=v.sqrt().view(-1, BLOCK).amax(1).clamp_min(TINY) / top)
    else:
        got.update(m=m, v=v)
    return {k: x for k, x in got.items() if x is not None or case["bits"] == 8 and k in ("m", "v")}
