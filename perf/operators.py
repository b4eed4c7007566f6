"""Operators of the block-scaled 8-bit expert path and the grouped softmax gate: the cases
they are measured at, their inputs, their plain forms and their values in 64 bits.

  quantize  rows of activations (or 128 x 128 blocks of a weight) to e4m3 codes with one
            power-of-two scale for each block of 128
  matmul    y = a w^T with e4m3 codes on both sides, one scale for each row and 128 inputs of
            a, and for each 128 x 128 block of w
  experts   SwiGLU experts over dispatched tokens with e4m3 weights: quantise the tokens,
            gate and up products, silu(gate) * up, quantise again, down product
  route     softmax over all experts, groups limited by their best expert, top-k, an optional
            bias for balance, weights renormalised or not

With ``own`` false ``run`` computes each operator from elementary torch operations; with it
true it makes the calls a user of the package makes.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one decoded token's hidden row on its way into the experts: a latency
        {"name": "quantize_token", "op": "quantize", "rows": 1, "n": 7168, "ld": 7168,
         "block_rows": 1, "dtype": "bf16"},
        # a prefill chunk's hidden rows, read out of a wider buffer
        {"name": "quantize_prefill", "op": "quantize", "rows": 8191, "n": 7168, "ld": 7424,
         "block_rows": 1, "dtype": "bf16"},
        # a weight matrix laid out once in 128 x 128 blocks, from fp32 master weights
        {"name": "quantize_weight", "op": "quantize", "rows": 2112, "n": 7168, "ld": 7168,
         "block_rows": 128, "dtype": "f32"},
        # one token through a projection with an odd number of outputs
        {"name": "matmul_token", "op": "matmul", "M": 1, "N": 2112, "K": 7168, "out": "bf16"},
        # a decode batch through the down projection of a dense block
        {"name": "matmul_batch", "op": "matmul", "M": 128, "N": 7168, "K": 2048, "out": "bf16"},
        # ragged everywhere: rows, outputs and a last block of 80 inputs, kept in fp32
        {"name": "matmul_ragged", "op": "matmul", "M": 333, "N": 577, "K": 1488, "out": "f32"},
        # a prefill chunk through a gate/up projection
        {"name": "matmul_prefill", "op": "matmul", "M": 8192, "N": 4096, "K": 7168,
         "out": "bf16"},
        # one decoded token: its experts' weights are the whole cost
        {"name": "experts_token", "op": "experts", "T": 1, "d": 7168, "I": 2048, "E": 64, "K": 8,
         "shared": True},
        # a decode batch that touches nearly every expert
        {"name": "experts_batch", "op": "experts", "T": 64, "d": 7168, "I": 2048, "E": 64, "K": 8,
         "shared": True},
        # prefill of a few thousand tokens over the experts of one device
        {"name": "experts_prefill", "op": "experts", "T": 4000, "d": 7168, "I": 2048, "E": 32,
         "K": 8, "shared": True},
        # one token's gate
        {"name": "route_token", "op": "route", "rows": 1, "E": 256, "K": 8, "G": 8, "tg": 4,
         "bias": True, "norm": True, "dtype": "f32"},
        # the gate of a prefill chunk: 160 experts in 8 groups, the best 3 groups, 6 experts
        {"name": "route_prefill", "op": "route", "rows": 16384, "E": 160, "K": 6, "G": 8, "tg": 3,
         "bias": False, "norm": False, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "matmul", "experts", "route"))
    if op == "quantize":
        n = 16 * rng.randint(1, 448)
        return {"op": op, "rows": _log(rng, 1, 8191), "n": n, "ld": n + 8 * rng.randint(0, 32),
                "block_rows": rng.choice((1, 1, BLOCK)), "dtype": rng.choice(("bf16", "f32"))}
    if op == "matmul":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 4096),
                "K": 16 * _log(rng, 8, 448), "out": rng.choice(("bf16", "bf16", "f32"))}
    if op == "experts":
        E = rng.choice((8, 16, 32, 48))
        return {"op": op, "T": _log(rng, 1, 4000), "d": 128 * _log(rng, 2, 40),
                "I": 128 * _log(rng, 1, 12), "E": E, "K": rng.randint(1, 8),
                "shared": rng.random() < 0.7}
    G = rng.choice((1, 1, 4, 8))
    E = G * rng.randint(4, 64)
    tg = rng.randint(1, G)
    return {"op": op, "rows": _log(rng, 1, 16384), "E": E,
            "K": rng.randint(1, min(8, tg * (E // G))), "G": G, "tg": tg,
            "bias": rng.random() < 0.5, "norm": rng.random() < 0.5,
            "dtype": rng.choice(("f32", "f32", "bf16"))}


def _blocks(n):
    return -(-n // BLOCK)


def work(c):
    if c["op"] == "quantize":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["rows"] * c["n"]
        return {"bytes": n * (e + 1) + 4 * -(-c["rows"] // c["block_rows"]) * _blocks(c["n"]),
                "flops": 3 * n}
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K + N * K + M * N * (2 if c["out"] == "bf16" else 4)
                + 4 * _blocks(K) * (M + _blocks(N)), "flops": 2 * M * N * K}
    if c["op"] == "experts":
        T, d, I, E, K = c["T"], c["d"], c["I"], c["E"], c["K"]
        hit = E * (1.0 - (1.0 - K / E) ** T) + (1 if c["shared"] else 0)
        slots = T * K + (T if c["shared"] else 0)
        return {"bytes": int(hit * 3 * d * I * (1 + 4 / BLOCK ** 2)) + 2 * T * d + 2 * slots * d
                + 4 * T * K, "flops": 6 * slots * d * I}
    e = 2 if c["dtype"] == "bf16" else 4
    return {"bytes": c["rows"] * (c["E"] * e + 8 * c["K"]) + 4 * c["E"],
            "flops": 4 * c["rows"] * c["E"]}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _codes(shape, g):
    """e4m3 codes of normal values, the largest near the type's end."""
    return (_randn(shape, g, torch.bfloat16) * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _weight(shape, g):
    """Codes [.., N, K] and fp32 scales [.., ceil(N/128), ceil(K/128)] of a weight whose rows
    have about unit norm; the blocks' scales are any numbers, as checkpoints have them."""
    *lead, N, K = shape
    s = torch.rand(*lead, _blocks(N), _blocks(K), generator=g, device="cuda") + 0.5
    return _codes(shape, g), s / (100.0 * math.sqrt(K))


def _activations(rows, n, ld, g, dtype):
    """Hidden rows: normal values, a few channels many times larger, as trained layers have."""
    x = _randn((rows, ld), g)
    x *= 1.0 + 15.0 * (torch.rand(ld, generator=g, device="cuda") < 0.01)
    return x.to(dtype)[:, :n]


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c}
    if c["op"] == "quantize":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["x"] = _activations(c["rows"], c["n"], c["ld"], g, dt)
    elif c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        s["a"] = _codes((M, K), g)
        s["a_scale"] = torch.exp2(torch.randint(-9, -5, (M, _blocks(K)), generator=g,
                                                device="cuda").float())
        s["w"], s["w_scale"] = _weight((N, K), g)
    elif c["op"] == "experts":
        T, d, I, E, K = c["T"], c["d"], c["I"], c["E"], c["K"]
        s["x"] = _activations(T, d, d, g, torch.bfloat16)
        liking = _randn((T, E), g) + 0.5 * _randn((E,), g)  # some experts are hit more often
        inds = liking.topk(K, dim=1).indices.to(torch.int32)
        flat = inds.reshape(-1).long()
        s["perm"] = torch.sort(flat, stable=True).indices.to(torch.int32)
        counts = torch.bincount(flat, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())  # rows of the busiest expert
        s["experts"] = {k: _weight(sh, g) for k, sh in
                        (("gate", (E, I, d)), ("up", (E, I, d)), ("down", (E, d, I)))}
        s["shared"] = {k: _weight(sh, g) for k, sh in
                       (("gate", (1, I, d)), ("up", (1, I, d)), ("down", (1, d, I)))} \
            if c["shared"] else None
    else:
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["logits"] = (1.5 * _randn((c["rows"], c["E"]), g)).to(dt)
        s["bias"] = 0.01 * _randn((c["E"],), g) if c["bias"] else None
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------

def _plain_quantize(x, block_rows=1):
    """fp32 [.., rows, n] -> (e4m3 codes, fp32 scales): the smallest power of two s with
    amax / s <= 448 for each block."""
    *lead, rows, n = x.shape
    R, B = -(-rows // block_rows), _blocks(n)
    p = torch.nn.functional.pad(x, (0, B * BLOCK - n, 0, R * block_rows - rows))
    p = p.reshape(*lead, R, block_rows, B, BLOCK)
    amax = p.abs().amax(dim=(-1, -3))
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = (torch.where(m <= 0.875, e - 9, e - 8)).clamp_min(-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    q = (p / scale[..., :, None, :, None]).reshape(*lead, R * block_rows, B * BLOCK)
    return q[..., :rows, :n].to(torch.float8_e4m3fn), scale


def _values(codes, scale, block_rows=1):
    """fp32 values of codes with a scale for each block."""
    *_, rows, n = codes.shape
    s = scale.repeat_interleave(BLOCK, -1)[..., :n]
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, -2)[..., :rows, :]
    return codes.float() * s


def _plain_swiglu(x, gate, up, down):
    """fp32 rows [E, m, d] through the experts' weights, the rows quantised before each
    product; fp32 [E, m, d]."""
    x = _values(*_plain_quantize(x))
    a = torch.matmul(x, _values(*gate, BLOCK).transpose(-1, -2))
    b = torch.matmul(x, _values(*up, BLOCK).transpose(-1, -2))
    h = a / (1.0 + torch.exp(-a)) * b
    return torch.matmul(_values(*_plain_quantize(h)), _values(*down, BLOCK).transpose(-1, -2))


def _plain_experts(s):
    c = s["c"]
    E, K, d, P = c["E"], c["K"], c["d"], c["T"] * c["K"]
    off, perm, x = s["offsets"].long(), s["perm"].long(), s["x"].float()
    # slot j of expert e lies in row j - offsets[e] of its batch of `most` rows
    j = torch.arange(P, device="cuda")
    e = torch.searchsorted(off[1:], j, right=True)
    at = e * s["most"] + j - off[e]
    rows = torch.zeros(E * s["most"], d, device="cuda")
    rows[at] = x[perm // K]
    y = _plain_swiglu(rows.reshape(E, s["most"], d), *(s["experts"][k] for k in ("gate", "up", "down")))
    y = y.reshape(-1, d)[at]
    if s["shared"] is not None:
        z = _plain_swiglu(x[None], *(s["shared"][k] for k in ("gate", "up", "down")))
        y = torch.cat([y, z[0]])
    return y.to(torch.bfloat16)


def _plain_route(s):
    c = s["c"]
    E, G, K = c["E"], c["G"], c["K"]
    l = s["logits"].double()  # close scores have to keep their order
    p = torch.exp(l - l.amax(dim=1, keepdim=True))
    p = p / p.sum(dim=1, keepdim=True)
    v = p if s["bias"] is None else p + s["bias"].double()
    if c["tg"] < G:
        best = v.reshape(-1, G, E // G).amax(dim=2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices
        keep = torch.zeros_like(best, dtype=torch.bool).scatter(1, order[:, :c["tg"]], True)
        v = torch.where(keep.repeat_interleave(E // G, dim=1), v, -math.inf)
    inds = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :K]
    w = p.gather(1, inds)
    if c["norm"] and K > 1:
        w = w / w.sum(dim=1, keepdim=True)
    return inds.to(torch.int32), (w * 2.5).float()


def _plain(s):
    c = s["c"]
    if c["op"] == "quantize":
        return _plain_quantize(s["x"].float(), c["block_rows"])
    if c["op"] == "matmul":
        y = torch.matmul(_values(s["a"], s["a_scale"]), _values(s["w"], s["w_scale"], BLOCK).t())
        return y.to(torch.bfloat16) if c["out"] == "bf16" else y
    return _plain_experts(s) if c["op"] == "experts" else _plain_route(s)


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(s):
    if not own:
        return _plain(s)
    from deepseek_moe_layer_gb300 import binding
    c = s["c"]
    if c["op"] == "quantize":
        return binding.quantize_blocks(s["x"], block_rows=c["block_rows"])
    if c["op"] == "matmul":
        return binding.matmul_blocks(s["a"], s["a_scale"], s["w"], s["w_scale"],
                                     out_dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    if c["op"] == "experts":
        dicts = [None if w is None else
                 {"bits": binding.MOE_BITS_E4M3, "gate": w["gate"][0], "gate_s": w["gate"][1],
                  "up": w["up"][0], "up_s": w["up"][1], "down": w["down"][0], "down_s": w["down"][1]}
                 for w in (s["experts"], s["shared"])]
        return binding.grouped_swiglu(s["x"], s["offsets"], s["perm"], c["K"], *dicts)
    return binding.route_softmax_grouped(s["logits"], c["K"], c["G"], c["tg"], c["norm"], 2.5,
                                         bias=s["bias"])


# ---------------------------------------------------------------------------------------
# values in 64 bits
# ---------------------------------------------------------------------------------------

def exact(c, seed):
    def quantize(x, block_rows=1):
        """float64 [rows, n] -> (e4m3 numbers, scales), both float64: each block of a 128-column
        strip is scaled by 2^ceil(log2(amax / 448)) and rounded to 4 significant bits (multiples
        of 2^-9 below 2^-6), ties to even."""
        rows, n = x.shape
        q = torch.empty_like(x)
        scales = torch.ones(-(-rows // block_rows), _blocks(n), dtype=torch.float64, device=x.device)
        for b in range(_blocks(n)):
            strip = x[:, b * BLOCK:(b + 1) * BLOCK]
            top = strip.abs().amax(dim=1)
            top = torch.nn.functional.pad(top, (0, scales.shape[0] * block_rows - rows))
            top = top.reshape(-1, block_rows).amax(dim=1)
            e = torch.floor(torch.log2(top.clamp_min(1e-300) / E4M3_MAX)) - 1  # from below, then up
            for _ in range(3):
                e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)
            scale = torch.where(top > 0, torch.exp2(e.clamp_min(-126)), 1.0)
            scales[:, b] = scale
            v = strip / scale.repeat_interleave(block_rows)[:rows, None]
            ulp = torch.exp2((torch.frexp(v)[1] - 4).clamp_min(-9).double())
            q[:, b * BLOCK:(b + 1) * BLOCK] = torch.round(v / ulp) * ulp
        return q, scales

    def product(q, qs, w, ws):
        """Sum over the 128-wide blocks of the inputs of (q_b w_b^T) * scale * scale."""
        n, k = w.shape
        ws = ws.double().repeat_interleave(BLOCK, 0)[:n]
        wide = torch.empty(n, k, dtype=torch.float64, device=w.device)
        for b in range(_blocks(k)):
            at = slice(b * BLOCK, (b + 1) * BLOCK)
            wide[:, at] = w[:, at].double() * ws[:, b:b + 1]
        qd = q.double().clone()
        for b in range(_blocks(k)):
            qd[:, b * BLOCK:(b + 1) * BLOCK] *= qs[:, b:b + 1].double()
        return qd @ wide.t()

    def swiglu(q, qs, w, e):
        part = {k: (w[k][0][e], w[k][1][e]) for k in ("gate", "up", "down")}
        a = product(q, qs, *part["gate"])
        h = a * torch.sigmoid(a) * product(q, qs, *part["up"])
        return product(*quantize(h), *part["down"])

    s = prepare(c, seed)
    if c["op"] == "quantize":
        return quantize(s["x"].double(), c["block_rows"])
    if c["op"] == "matmul":
        return product(s["a"], s["a_scale"], s["w"], s["w_scale"])
    if c["op"] == "experts":
        q, qs = quantize(s["x"].double())
        off, tok = s["offsets"].tolist(), s["perm"].long() // c["K"]
        out = [swiglu(q[tok[off[e]:off[e + 1]]], qs[tok[off[e]:off[e + 1]]], s["experts"], e)
               for e in range(c["E"]) if off[e + 1] > off[e]]
        if s["shared"] is not None:
            out.append(swiglu(q, qs, s["shared"], 0))
        return torch.cat(out)
    # the K best experts one after the other, each by its value and then its index
    p = torch.softmax(s["logits"].double(), dim=1)
    v = p.clone() if s["bias"] is None else p + s["bias"].double()
    rows, (E, G) = torch.arange(c["rows"], device="cuda"), (c["E"], c["G"])
    first = lambda t: (t == t.amax(dim=1, keepdim=True)).to(torch.int8).argmax(dim=1)  # noqa: E731
    best = v.view(-1, G, E // G).amax(dim=2)
    out = torch.ones(c["rows"], G, dtype=torch.bool, device="cuda")
    for _ in range(c["tg"]):
        g = first(best)
        best[rows, g], out[rows, g] = -math.inf, False
    v.view(-1, G, E // G)[out] = -math.inf
    inds = []
    for _ in range(c["K"]):
        inds.append(first(v))
        v[rows, inds[-1]] = -math.inf
    inds = torch.stack(inds, dim=1)
    w = p[rows[:, None], inds]
    if c["norm"] and c["K"] > 1:
        w = w / w.sum(dim=1, keepdim=True)
    return inds.to(torch.int32), w * 2.5
