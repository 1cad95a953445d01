"""The 4-bit decoder block, operator by operator, at the sizes it is used with.

  quantize  rows of bf16 or fp32 as 4-bit integers with one scale (and, in the affine form, one offset) per group of
            32, 64 or 128 columns, and back: how weights get there, and what they stand for afterwards.
  gemm      Y[b, n] = sum_k X[b, k] W[n, k] (+ bias[n]) over such weights and bf16 tokens, from one token to a prompt.
  norm      the join between two blocks: p = x / sqrt(mean(x^2) + eps) * post_gain (the norm after a block; or p = x),
            h = residual_scale * r + block_scale * gate * p, y = h / sqrt(mean(h^2) + eps) * gain (the norm before the
            next block; or none), y in bf16, fp32 or 8-bit integers with a scale per token.
  block     them together, as a decode step runs them: join, gate and up in one product, silu(g) * u, down, join.

A group p of 4-bit weights: scale s = max(max|p| / 7, 2^-126), p is about s q; affine: s = max(max p / 15 - min p / 15,
2^-126), m = (min p / 2 + max p / 2) + s / 2, p is about s q + m.  s (before m and q are formed) and m are rounded to
the type they are kept in; q is the fp32 quotient p / s or (p - m) / s rounded to the nearest integer, ties to even,
and held to -8 .. 7.  A row's integers lie two to a byte, the even column in the low half, as q + 8; rows start at
multiples of 16 bytes.  Scales and offsets lie group by group: [groups, rows].  Integers come back as the values that
they stand for.
"""
from __future__ import annotations

import torch

own = False

EPS = 1e-5
TINY = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4, "i8": 1, "none": 0}


def listed():
    return [
        # a gate matrix taken to 4 bits at model load, one bf16 scale per 128 columns
        {"name": "quantize, gate weights", "op": "quantize", "b": 14336, "cols": 4096, "x": "bf16", "group": 128, "affine": False, "scales": "bf16"},
        # a small fp32 matrix of odd width (a head, an adapter), small groups with offsets
        {"name": "quantize, odd rows", "op": "quantize", "b": 37, "cols": 1001, "x": "f32", "group": 32, "affine": True, "scales": "f32"},
        # one decode step of one sequence: the gate product, bound by the weight read
        {"name": "gemm, one token", "op": "gemm", "b": 1, "rows": 14336, "cols": 4096, "group": 128, "affine": False, "scales": "bf16", "out": "bf16", "bias": False},
        # a served batch's down product: few rows, a long sum, weights that came with offsets
        {"name": "gemm, 16 tokens down", "op": "gemm", "b": 16, "rows": 4096, "cols": 14336, "group": 64, "affine": True, "scales": "bf16", "out": "f32", "bias": False},
        # ragged in every size, with offsets, a bias and a short last group
        {"name": "gemm, ragged", "op": "gemm", "b": 77, "rows": 1000, "cols": 4100, "group": 32, "affine": True, "scales": "f32", "out": "f32", "bias": True},
        # a large served batch, or a chunk of a prompt
        {"name": "gemm, 256 tokens", "op": "gemm", "b": 256, "rows": 14336, "cols": 4096, "group": 128, "affine": False, "scales": "bf16", "out": "bf16", "bias": False},
        # a long prompt's gate product: bound by the matrix cores
        {"name": "gemm, prompt", "op": "gemm", "b": 4096, "rows": 14336, "cols": 4096, "group": 128, "affine": False, "scales": "bf16", "out": "bf16", "bias": False},
        # one decode step of one sequence: the join of two blocks; latency is all of it
        {"name": "norm, one token", "op": "norm", "b": 1, "cols": 4096, "x": "bf16", "res": "bf16", "post": True, "gate": "vector", "branch": 1.0, "keep": 1.0, "out": "bf16"},
        # a prompt's join, in front of 8-bit products
        {"name": "norm, prompt", "op": "norm", "b": 2048, "cols": 4096, "x": "bf16", "res": "bf16", "post": True, "gate": "vector", "branch": 1.0, "keep": 1.0, "out": "i8"},
        # an fp32 stream of a wider model with a gate per token and scaled branches; an odd number of tokens
        {"name": "norm, fp32 stream", "op": "norm", "b": 1111, "cols": 8192, "x": "bf16", "res": "f32", "post": True, "gate": "token", "branch": 0.5, "keep": 0.875, "out": "bf16"},
        # a whole block of one sequence's decode step, and of a served batch's
        {"name": "block, one token", "op": "block", "b": 1, "rows": 14336, "cols": 4096, "group": 128, "affine": False, "scales": "bf16"},
        {"name": "block, 16 tokens", "op": "block", "b": 16, "rows": 14336, "cols": 4096, "group": 64, "affine": True, "scales": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A size from lo to hi, spread over its logarithm; most of them are odd ones or no multiple of anything."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "gemm", "norm", "norm", "block"))
    if op == "norm":
        return {"op": op, "b": _spread(rng, 1, 2048), "cols": _spread(rng, 64, 8192), "x": rng.choice(("bf16", "f32")),
                "res": rng.choice(("bf16", "f32")), "post": rng.random() < 0.75, "gate": rng.choice(("none", "vector", "token")),
                "branch": rng.choice((1.0, 0.5, 0.25)), "keep": rng.choice((1.0, 0.875)),
                "out": rng.choice(("i8", "bf16", "f32", "none"))}
    four = {"group": rng.choice((32, 64, 128)), "affine": rng.random() < 0.5, "scales": rng.choice(("bf16", "f32"))}
    if op == "quantize":
        return {"op": op, "b": _spread(rng, 1, 14336), "cols": _spread(rng, 64, 4096), "x": rng.choice(("bf16", "f32")), **four}
    if op == "gemm":
        return {"op": op, "b": _spread(rng, 1, 4096), "rows": _spread(rng, 64, 14336), "cols": _spread(rng, 64, 4096), **four,
                "out": rng.choice(("bf16", "f32")), "bias": rng.random() < 0.5}
    return {"op": op, "b": _spread(rng, 1, 64), "rows": _spread(rng, 256, 14336), "cols": _spread(rng, 128, 4096), **four}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _tokens(b, cols, gen, dtype):
    """Activations of b tokens: N(0, 1) with a channel in 256 twenty times as large, as residual streams have; the last
    token of a batch of eight or more is padding (zeros)."""
    x = _randn(gen, b, cols)
    loud = torch.rand(cols, generator=gen, device="cuda") < 1 / 256
    x = torch.where(loud, 20 * x, x)
    if b >= 8:
        x[-1] = 0
    return x.to(dtype)


def _weights(rows, cols, group, gen):
    """Weights N(0, 0.02), the groups of columns off centre by 0.005 in the mean."""
    w = 0.02 * _randn(gen, rows, cols)
    shift = 0.005 * _randn(gen, rows, (cols + group - 1) // group)
    return w + shift.repeat_interleave(group, 1)[:, :cols]


def _rows4(rows, cols):
    """Packed 4-bit rows as the framework lays them out: each starts at a multiple of 16 bytes."""
    return torch.zeros(rows, (cols + 31) // 32 * 16, dtype=torch.uint8, device="cuda")[:, : (cols + 1) // 2]


def _ints4(w, group, affine, kind):
    """A matrix's integers [rows, cols] (whole numbers, held in fp32) and the scales and offsets [groups, rows] as they are kept."""
    rows, cols = w.shape
    groups = (cols + group - 1) // group
    pad = groups * group - cols
    if affine:
        top = torch.nn.functional.pad(w, (0, pad), value=float("-inf")).view(rows, groups, group).amax(2)
        low = torch.nn.functional.pad(w, (0, pad), value=float("inf")).view(rows, groups, group).amin(2)
        scale = (top / 15 - low / 15).clamp_min(TINY).to(kind)
        offset = ((low / 2 + top / 2) + scale.float() / 2).to(kind)
    else:
        top = torch.nn.functional.pad(w, (0, pad)).view(rows, groups, group).abs().amax(2)
        scale, offset = (top / 7).clamp_min(TINY).to(kind), None
    of = w if offset is None else w - offset.float().repeat_interleave(group, 1)[:, :cols]
    q = torch.round(of / scale.float().repeat_interleave(group, 1)[:, :cols]).clamp(-8, 7)
    return q, scale.t().contiguous(), None if offset is None else offset.t().contiguous()


def _in4(w, group, affine, kind):
    """A matrix in 4 bits: packed rows, scales, offsets."""
    q, scale, offset = _ints4(w, group, affine, kind)
    u = (q + 8).to(torch.uint8)
    if u.shape[1] % 2:
        u = torch.nn.functional.pad(u, (0, 1), value=8)
    packed = _rows4(*w.shape)
    packed.copy_(u[:, ::2] | (u[:, 1::2] << 4))
    return packed, scale, offset


def prepare(case, seed):
    op, b, cols = case["op"], case["b"], case["cols"]
    gen, s = _gen(seed), dict(case)
    four = (case.get("group"), case.get("affine"), TYPES.get(case.get("scales")))
    if op == "quantize":
        s["X"] = _weights(b, cols, case["group"], gen).to(TYPES[case["x"]])
        s["Q"] = _rows4(b, cols)
        s["scale"] = torch.empty((cols + case["group"] - 1) // case["group"], b, dtype=TYPES[case["scales"]], device="cuda")
        s["offset"] = torch.empty_like(s["scale"]) if case["affine"] else None
        s["Y"] = torch.empty(b, cols, dtype=torch.bfloat16, device="cuda")
    elif op == "gemm":
        s["W"], s["scale"], s["offset"] = _in4(_weights(case["rows"], cols, case["group"], gen), *four)
        s["X"] = _tokens(b, cols, gen, torch.bfloat16)
        s["bias"] = _randn(gen, case["rows"]) if case["bias"] else None
        s["Y"] = torch.empty(b, case["rows"], dtype=TYPES[case["out"]], device="cuda")
    elif op == "norm":
        s["X"] = _tokens(b, cols, gen, TYPES[case["x"]])
        s["R"] = _tokens(b, cols, gen, TYPES[case["res"]])
        s["H"] = torch.empty_like(s["R"])
        s["post_gain"] = (1 + 0.2 * _randn(gen, cols)).to(TYPES[case["x"]]) if case["post"] else None
        s["gain"] = (1 + 0.2 * _randn(gen, cols)).to(TYPES[case["x"]]) if case["out"] != "none" else None
        shape = {"none": None, "vector": (cols,), "token": (b, cols)}[case["gate"]]
        s["gate"] = None if shape is None else (0.5 + 0.5 * _randn(gen, *shape)).to(torch.bfloat16)
        s["scale"] = torch.empty(b, device="cuda") if case["out"] == "i8" else None
        s["Q"] = torch.empty(b, (cols + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :cols] if case["out"] == "i8" else None
        s["Y"] = None if case["out"] == "none" else torch.empty(b, cols, dtype=TYPES.get(case["out"], torch.bfloat16), device="cuda")
    else:
        rows = case["rows"]
        s["X"] = _tokens(b, cols, gen, torch.bfloat16)
        s["R"] = _tokens(b, cols, gen, torch.bfloat16)
        for name in ("post1", "gain1", "post2", "gain2"):
            s[name] = (1 + 0.2 * _randn(gen, cols)).to(torch.bfloat16)
        s["gate"] = (0.5 + 0.5 * _randn(gen, cols)).to(torch.bfloat16)
        s["W"], s["w_scale"], s["w_offset"] = _in4(_weights(2 * rows, cols, case["group"], gen), *four)  # gate, then up
        s["D"], s["d_scale"], s["d_offset"] = _in4(_weights(cols, rows, case["group"], gen), *four)
        for name, width in (("H1", cols), ("N1", cols), ("GU", 2 * rows), ("A", rows), ("Z", cols), ("H2", cols), ("N2", cols)):
            s[name] = torch.empty(b, width, dtype=torch.bfloat16, device="cuda")
    return s


# -- plain forms ----------------------------------------------------------------

def _values4(packed, cols, group, scale, offset):
    """What packed 4-bit rows stand for, in fp32."""
    q = (torch.stack((packed & 15, packed >> 4), 2).view(packed.shape[0], -1)[:, :cols].float()) - 8
    v = q * scale.t().float().repeat_interleave(group, 1)[:, :cols]
    return v if offset is None else v + offset.t().float().repeat_interleave(group, 1)[:, :cols]


def _gemm(packed, group, scale, offset, X, bias=None):
    y = X.float() @ _values4(packed, X.shape[1], group, scale, offset).t()
    return y if bias is None else y + bias


def _rstd(v):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _join(X, R, post_gain, gate, branch, keep):
    """The stream behind a block, as it is kept."""
    p = X.float()
    if post_gain is not None:
        p = p * _rstd(p) * post_gain.float()
    if gate is not None:
        p = p * gate.float()
    return (keep * R.float() + branch * p).to(R.dtype)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["X"].float()
        q, scale, offset = _ints4(x, s["group"], s["affine"], s["scale"].dtype)
        v = q * scale.t().float().repeat_interleave(s["group"], 1)[:, : x.shape[1]]
        if offset is not None:
            v = v + offset.t().float().repeat_interleave(s["group"], 1)[:, : x.shape[1]]
        return v.to(torch.bfloat16), scale, offset
    if op == "gemm":
        return _gemm(s["W"], s["group"], s["scale"], s["offset"], s["X"], s["bias"]).to(s["Y"].dtype)
    if op == "norm":
        kept = _join(s["X"], s["R"], s["post_gain"], s["gate"], s["branch"], s["keep"])
        if s["out"] == "none":
            return kept
        h = kept.float()
        p = h * s["gain"].float()
        if s["out"] != "i8":
            return kept, (p * _rstd(h)).to(s["Y"].dtype)
        step = (p.abs().amax(1, keepdim=True) / 127).clamp_min(TINY)
        scale = step * _rstd(h)
        return kept, (torch.round(p * (1 / step)) * scale).to(torch.bfloat16), scale[:, 0]
    h = _join(s["X"], s["R"], s["post1"], s["gate"], 1.0, 1.0)
    n = (h.float() * _rstd(h.float()) * s["gain1"].float()).to(torch.bfloat16)
    gu = _gemm(s["W"], s["group"], s["w_scale"], s["w_offset"], n).to(torch.bfloat16).float()
    g, u = gu[:, : s["rows"]], gu[:, s["rows"]:]
    a = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
    z = _gemm(s["D"], s["group"], s["d_scale"], s["d_offset"], a).to(torch.bfloat16)
    h = _join(z, h, s["post2"], s["gate"], 1.0, 1.0)
    return h, (h.float() * _rstd(h.float()) * s["gain2"].float()).to(torch.bfloat16)


# -- the framework's kernels ------------------------------------------------------

def _kernels(s):
    import decode_gemv_canonical_amd as uw

    op = s["op"]
    if op == "quantize":
        uw.uw_i4_quantize(s["X"], s["Q"], s["scale"], s["offset"], group=s["group"])
        uw.uw_i4_dequantize(s["Q"], s["scale"], s["Y"], s["offset"], group=s["group"])
        return s["Y"], s["scale"], s["offset"]
    if op == "gemm":
        uw.uw_i4_gemm(s["W"], s["scale"], s["X"], s["Y"], offset=s["offset"], group=s["group"], bias=s["bias"])
        return s["Y"]
    if op == "norm":
        uw.uw_block_norm(s["X"], s["R"], post_gain=s["post_gain"], post_norm=s["post"], gate=s["gate"], block_scale=s["branch"],
                         residual_scale=s["keep"], residual_out=s["H"], gain=s["gain"], Y=s["Y"] if s["Q"] is None else s["Q"],
                         scale=s["scale"], eps=EPS)
        if s["out"] == "none":
            return s["H"]
        if s["out"] != "i8":
            return s["H"], s["Y"]
        uw.uw_i8_dequantize(s["Q"], s["scale"], s["Y"])
        return s["H"], s["Y"], s["scale"]
    uw.uw_block_norm(s["X"], s["R"], post_gain=s["post1"], gate=s["gate"], residual_out=s["H1"], gain=s["gain1"], Y=s["N1"], eps=EPS)
    uw.uw_i4_gemm(s["W"], s["w_scale"], s["N1"], s["GU"], offset=s["w_offset"], group=s["group"])
    uw.uw_silu_mul(s["GU"][:, : s["rows"]], s["GU"][:, s["rows"]:], s["A"])
    uw.uw_i4_gemm(s["D"], s["d_scale"], s["A"], s["Z"], offset=s["d_offset"], group=s["group"])
    uw.uw_block_norm(s["Z"], s["H1"], post_gain=s["post2"], gate=s["gate"], residual_out=s["H2"], gain=s["gain2"], Y=s["N2"], eps=EPS)
    return s["H2"], s["N2"]


def run(state):
    return _kernels(state) if own else _plain(state)


def work(case):
    op, b, cols = case["op"], case["b"], case["cols"]
    n = b * cols

    def four(rows, width):
        """Bytes of a matrix in 4 bits."""
        per = BYTES[case["scales"]] * (2 if case["affine"] else 1)
        return rows * ((width + 1) // 2) + rows * ((width + case["group"] - 1) // case["group"]) * per

    if op == "quantize":  # the weights in; the packed rows, then the bf16 values that they stand for, out
        return {"bytes": n * BYTES[case["x"]] + four(b, cols) + 2 * n, "flops": 4 * n}
    if op == "gemm":
        rows = case["rows"]
        return {"bytes": four(rows, cols) + 2 * n + 4 * rows * case["bias"] + b * rows * BYTES[case["out"]],
                "flops": 2 * b * rows * cols}
    if op == "norm":
        gate = {"none": 0, "vector": 2 * cols, "token": 2 * n}[case["gate"]]
        gains = cols * BYTES[case["x"]] * (case["post"] + (case["out"] != "none"))
        # 8-bit outputs: the integers and their scales, then the bf16 values that they stand for
        out = n * (1 + 2) + 4 * b if case["out"] == "i8" else n * BYTES[case["out"]]
        return {"bytes": n * BYTES[case["x"]] + 2 * n * BYTES[case["res"]] + gate + gains + out, "flops": 14 * n}
    rows = case["rows"]
    return {"bytes": four(2 * rows, cols) + four(cols, rows) + 10 * cols + 4 * 2 * n, "flops": 6 * b * rows * cols}


# -- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, cols = case["op"], case["cols"]

    def spread(per_group, width):
        """One value per group and row as one per column and row."""
        at = torch.arange(width, device="cuda") // case["group"]
        return per_group.double()[at].T

    def meaning(packed, width, scale, offset):
        column = torch.arange(width, device="cuda")
        half = packed[:, column // 2].int()
        value = torch.where(column % 2 == 0, half % 16, half // 16).double() - 8
        value = value * spread(scale, width)
        return value if offset is None else value + spread(offset, width)

    def product(packed, scale, offset, tokens):
        return torch.mm(tokens.double(), meaning(packed, tokens.shape[1], scale, offset).T.contiguous())

    def length(rows):
        return torch.sqrt(torch.sum(rows ** 2, dim=1) / rows.shape[1] + EPS).unsqueeze(1)

    def joined(block, stream, after, gate, branch, keep):
        v = block.double()
        if after is not None:
            v = v / length(v) * after.double()
        if gate is not None:
            v = v * gate.double()
        return keep * stream.double() + branch * v

    if op == "quantize":
        x, size = s["X"].double(), case["group"]
        parts = [x[:, i: i + size] for i in range(0, cols, size)]
        most = torch.stack([p.max(1).values for p in parts])
        least = torch.stack([p.min(1).values for p in parts])
        kind, offset = TYPES[case["scales"]], None
        if case["affine"]:
            scale = torch.maximum((most - least) / 15, torch.full_like(most, TINY)).to(kind)
            offset = ((least + most + scale.double()) / 2).to(kind)
            x = x - spread(offset, cols)
        else:
            scale = torch.maximum(torch.maximum(most, -least) / 7, torch.full_like(most, TINY)).to(kind)
        ints = torch.round((x / spread(scale, cols)).float()).double()  # the definition rounds the quotient to fp32 first
        ints = torch.minimum(torch.maximum(ints, torch.full_like(ints, -8)), torch.full_like(ints, 7))
        values = ints * spread(scale, cols)
        if offset is None:
            return values, scale.double(), None
        return values + spread(offset, cols), scale.double(), offset.double()
    if op == "gemm":
        y = product(s["W"], s["scale"], s["offset"], s["X"])
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "norm":
        stream = joined(s["X"], s["R"], s["post_gain"], s["gate"], case["branch"], case["keep"])
        if case["out"] == "none":
            return stream
        h = stream.to(s["R"].dtype).double()  # the norm reads the stream as it is kept
        rows = h * s["gain"].double()
        if case["out"] != "i8":
            return stream, rows / length(h)
        step = torch.clamp(torch.max(torch.abs(rows), dim=1, keepdim=True).values / 127, min=TINY)
        return stream, torch.round(rows / step) * step / length(h), (step / length(h))[:, 0]
    bf16 = torch.bfloat16  # each operator writes bf16, and the next reads that
    h = joined(s["X"], s["R"], s["post1"], s["gate"], 1, 1).to(bf16).double()
    n = (h / length(h) * s["gain1"].double()).to(bf16)
    first, second = product(s["W"], s["w_scale"], s["w_offset"], n).to(bf16).double().split(case["rows"], dim=1)
    a = (first * torch.sigmoid(first) * second).to(bf16)
    z = product(s["D"], s["d_scale"], s["d_offset"], a).to(bf16)
    stream = joined(z, h, s["post2"], s["gate"], 1, 1)
    h = stream.to(bf16).double()
    return stream, h / length(h) * s["gain2"].double()
