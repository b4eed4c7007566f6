"""Operators of sparse attention over a latent cache, around the indexer's selection: the cases
they are measured at, their inputs, their plain forms and their values in 64 bits.

  append     rows of new tokens into a paged cache: normalised, rotated by their positions,
             rounded (to bf16, or to e4m3 codes with a power-of-two scale per 128 columns), and
             the rotated parts of the same tokens' queries
  scores     the indexer's scores of every cached position a token may see:
             key_scale * sum over heads of weight * relu(query . key)
  attention  attention whose keys and values are one cached row per position (512 latent columns,
             64 rotated ones; the values are the latent columns), over all positions a token may
             see or over selected ones

With ``own`` false ``run`` computes each operator from elementary torch operations; with it
true it makes the calls a user of the package makes.
"""
import math

import torch

own = False

LATENT, ROT = 512, 64
WIDTH = LATENT + ROT
IDX = 128          # columns of an index key
E4M3_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
# append: T tokens of one or more sequences; "latent" rows are 512 RMS-normalised + 64 rotated
# columns, "index" rows 128 layer-normalised columns whose first 64 are rotated.
# scores, attention: B sequences of `tokens` new tokens each (ragged: fewer and fewer), the first
# with n positions in the cache and the others with less; a token sees the positions up to its own.

def listed():
    return [
        # one decoded token's latent row and its 128 heads' rotated queries: a latency
        {"name": "append_token", "op": "append", "kind": "latent", "T": 1, "heads": 128,
         "page": 64, "cache": "bf16", "interleaved": True, "start": 131071},
        # a prefill chunk of latent rows and queries
        {"name": "append_prefill", "op": "append", "kind": "latent", "T": 8192, "heads": 128,
         "page": 64, "cache": "bf16", "interleaved": True, "start": 8192},
        # an odd number of index keys into an 8-bit cache, no queries
        {"name": "append_index", "op": "append", "kind": "index", "T": 4001, "heads": 0,
         "page": 64, "cache": "e4m3", "interleaved": False, "start": 777},
        # one decoded token: a latency
        {"name": "scores_token", "op": "scores", "B": 1, "tokens": 1, "ragged": False, "n": 4096,
         "heads": 64, "page": 64, "cache": "bf16"},
        # a decode batch with long contexts: the keys' bytes are the whole cost
        {"name": "scores_decode", "op": "scores", "B": 64, "tokens": 1, "ragged": False, "n": 32768,
         "heads": 64, "page": 64, "cache": "e4m3"},
        # chunks of a few prompts, odd everywhere, small pages
        {"name": "scores_ragged", "op": "scores", "B": 3, "tokens": 501, "ragged": True, "n": 5003,
         "heads": 32, "page": 16, "cache": "bf16"},
        # a prefill chunk behind a long context: tensor work
        {"name": "scores_prefill", "op": "scores", "B": 1, "tokens": 4096, "ragged": False,
         "n": 16384, "heads": 64, "page": 64, "cache": "e4m3"},
        # one decoded token over its whole context: a latency, few rows and one long axis
        {"name": "attention_token", "op": "attention", "B": 1, "tokens": 1, "ragged": False,
         "n": 4096, "heads": 128, "page": 64, "k": 0},
        # a decode batch over whole contexts of many lengths
        {"name": "attention_decode", "op": "attention", "B": 64, "tokens": 1, "ragged": False,
         "n": 16384, "heads": 128, "page": 64, "k": 0},
        # a few drafted tokens per sequence, few heads, small pages, odd lengths
        {"name": "attention_draft", "op": "attention", "B": 17, "tokens": 4, "ragged": False,
         "n": 3001, "heads": 16, "page": 16, "k": 0},
        # a decode batch over the 2048 positions the indexer selected
        {"name": "attention_selected", "op": "attention", "B": 64, "tokens": 1, "ragged": False,
         "n": 16384, "heads": 128, "page": 64, "k": 2048},
        # a prefill chunk, each token over its own 2048 selected positions
        {"name": "attention_prefill", "op": "attention", "B": 1, "tokens": 2048, "ragged": False,
         "n": 8192, "heads": 128, "page": 64, "k": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "scores", "attention"))
    page = rng.choice((1, 16, 48, 64, 64, 128))
    if op == "append":
        kind = rng.choice(("latent", "index"))
        return {"op": op, "kind": kind, "T": _log(rng, 1, 8192),
                "heads": rng.choice((0, 1, 16, 64, 128)), "page": page,
                "cache": "bf16" if kind == "latent" else rng.choice(("bf16", "e4m3")),
                "interleaved": rng.random() < 0.5, "start": _log(rng, 1, 1000000)}
    c = {"op": op, "B": _log(rng, 1, 64), "tokens": rng.choice((1, 1, 2, 5, _log(rng, 2, 2048))),
         "ragged": rng.random() < 0.3}
    if op == "scores":
        c.update(n=_log(rng, c["tokens"], 32768), heads=rng.choice((8, 16, 32, 64)), page=page,
                 cache=rng.choice(("bf16", "e4m3")))
        most = 1 << 26  # pairs of a token and a position
    else:
        c.update(n=_log(rng, c["tokens"], 16384), heads=rng.choice((1, 16, 24, 64, 128)), page=page,
                 k=rng.choice((0, 0, 2048, _log(rng, 1, 2048))))
        most = 1 << 22
    while c["B"] > 1 and c["B"] * c["tokens"] * c["n"] > most:
        c["B"] -= 1
    while c["tokens"] > 1 and c["tokens"] * c["n"] > most:
        c["tokens"] //= 2
    return c


def _shape(c):
    """Per sequence: its new tokens, and its positions with them."""
    B, tokens, n = c["B"], c["tokens"], c["n"]
    new = [max(1, tokens - (b * tokens // (B + 1) if c["ragged"] else 0)) for b in range(B)]
    return new, [max(new[b], n - b * (3 * n // 4) // B) for b in range(B)]


def _visible(c):
    """Positions that each token may see, in the tokens' order."""
    return [n - t + i + 1 for t, n in zip(*_shape(c)) for i in range(t)]


def work(c):
    if c["op"] == "append":
        w = WIDTH if c["kind"] == "latent" else IDX
        row = 2 * w if c["cache"] == "bf16" else w + 4
        return {"bytes": c["T"] * (2 * w + row + 4 * c["heads"] * ROT + 8),
                "flops": c["T"] * (6 * w + 3 * c["heads"] * ROT)}
    new, length = _shape(c)
    T, H, seen = sum(new), c["heads"], _visible(c)
    if c["op"] == "scores":
        e = 2 if c["cache"] == "bf16" else 1
        return {"bytes": sum(length) * (IDX * e + (4 if e == 1 else 0)) + T * H * (IDX * e + 4)
                + 4 * T * c["n"], "flops": 2 * sum(seen) * H * IDX}
    rows, pairs = sum(length), sum(seen)
    if c["k"]:
        pairs = sum(min(c["k"], s) for s in seen)
        rows = sum(min(n, t * c["k"]) for t, n in zip(new, length))
    return {"bytes": rows * WIDTH * 2 + T * H * (WIDTH + LATENT) * 2 + 4 * T * c["k"],
            "flops": 2 * pairs * H * (WIDTH + LATENT)}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _pages(c, g):
    """Block table int32 [B, pages of the longest], -1 behind a sequence's last page, and the
    number of pages of the cache (some belong to nobody)."""
    need = [-(-n // c["page"]) for n in _shape(c)[1]]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["B"], max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table, total


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c}
    if c["op"] == "append":
        latent = c["kind"] == "latent"
        T, w = c["T"], WIDTH if latent else IDX
        # the projection that made the row made other columns beside it
        s["x"] = _randn((T, w + 1536 if latent else w), g).to(torch.bfloat16)[:, :w]
        pages = -(-2 * T // c["page"]) + 1
        s["slots"] = torch.randperm(pages * c["page"], generator=g, device="cuda")[:T]
        s["positions"] = _ints(range(c["start"], c["start"] + T))
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, ROT, 2, device="cuda").double() / ROT)).float()
        s["weight"] = 1.0 + 0.1 * _randn((LATENT if latent else IDX,), g)
        s["bias"] = None if latent else 0.1 * _randn((IDX,), g)
        old = _randn((pages, c["page"], w), g)
        if c["cache"] == "bf16":
            s["cache"], s["scales"] = old.to(torch.bfloat16), None
        else:
            s["cache"] = (100.0 * old).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s["scales"] = torch.full((pages, c["page"], 1), 0.03125, device="cuda")
        if c["heads"]:
            # the rotated part of the queries as their projection leaves it (behind 128 other
            # columns of a head), and its place in the queries that the attention reads
            s["q"] = _randn((T, c["heads"], 128 + ROT), g).to(torch.bfloat16)[..., 128:]
            s["q_out"] = torch.zeros(T, c["heads"], WIDTH if latent else IDX, dtype=torch.bfloat16,
                                     device="cuda")
        return s
    new, length = _shape(c)
    T, H = sum(new), c["heads"]
    s["table"], pages = _pages(c, g)
    s["lengths"] = _ints(_visible(c))
    s["cu"] = None if max(new) == 1 else _ints([sum(new[:b]) for b in range(c["B"] + 1)])
    if c["op"] == "scores":
        keys, q = _randn((pages, c["page"], IDX), g), _randn((T, H, IDX), g)
        w = _randn((T, H), g) / math.sqrt(H * IDX)
        if c["cache"] == "bf16":
            s["keys"], s["q"], s["scales"] = keys.to(torch.bfloat16), q.to(torch.bfloat16), None
        else:
            f8 = lambda t: (100.0 * t).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)  # noqa: E731
            s["keys"], s["q"], w = f8(keys), f8(q), w / 100.0
            s["scales"] = torch.exp2(torch.randint(-8, -5, (pages, c["page"], 1), generator=g,
                                                   device="cuda").float())
        s["w"] = w
        return s
    s["cache"] = _randn((pages, c["page"], WIDTH), g).to(torch.bfloat16)
    s["q"] = _randn((T, H, WIDTH), g).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(128 + ROT)
    s["inds"] = None
    if c["k"]:
        # neighbouring tokens like much the same positions
        k, n = c["k"], c["n"]
        inds = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        at = 0
        for t, m in zip(new, length):
            liking = _randn((1, m), g) + 0.7 * _randn((t, m), g)
            see = s["lengths"][at:at + t, None]
            liking.masked_fill_(torch.arange(m, device="cuda") >= see, -math.inf)
            best = liking.topk(min(k, m), dim=1).indices
            best = torch.where(best < see, best, n).sort(dim=1).values  # ascending, then the padding
            inds[at:at + t, :min(k, m)] = torch.where(best < n, best, -1).to(torch.int32)
            at += t
        s["inds"] = inds
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------

def _rotate(x, positions, inv_freq, interleaved):
    """fp32 [T, .., R] with the pairs of each row turned by positions * inv_freq (in 64 bits)."""
    a = positions.double()[:, None] * inv_freq.double()
    a = a.reshape(a.shape[0], *([1] * (x.dim() - 2)), a.shape[1])
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    if interleaved:
        u, v = x[..., 0::2], x[..., 1::2]
        return torch.stack((u * cos - v * sin, v * cos + u * sin), dim=-1).reshape(x.shape)
    u, v = x.chunk(2, dim=-1)
    return torch.cat((u * cos - v * sin, v * cos + u * sin), dim=-1)


def _plain_quantize(x):
    """fp32 [T, 128] -> (e4m3 codes, fp32 scale [T, 1]): the smallest power of two s with
    amax / s <= 448."""
    amax = x.abs().amax(dim=1, keepdim=True)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp_min(-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    return (x / scale).to(torch.float8_e4m3fn), scale


def _plain_append(s):
    c = s["c"]
    x, w = s["x"].float(), s["weight"]
    turn = lambda t: _rotate(t, s["positions"], s["inv_freq"], c["interleaved"])  # noqa: E731
    if c["kind"] == "latent":
        a = x[:, :LATENT]
        a = a * torch.rsqrt((a * a).mean(dim=1, keepdim=True) + EPS) * w
        x = torch.cat((a, turn(x[:, LATENT:])), dim=1)
    else:
        x = x - x.mean(dim=1, keepdim=True)
        x = x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS) * w + s["bias"]
        x = torch.cat((turn(x[:, :ROT]), x[:, ROT:]), dim=1)
    flat = s["cache"].view(-1, x.shape[1])
    out = [s["cache"]]
    if c["cache"] == "bf16":
        flat[s["slots"]] = x.to(torch.bfloat16)
    else:
        codes, scale = _plain_quantize(x)
        flat.view(torch.uint8)[s["slots"]] = codes.view(torch.uint8)
        s["scales"].view(-1, 1)[s["slots"]] = scale
        out.append(s["scales"])
    if c["heads"]:
        at = slice(LATENT, None) if c["kind"] == "latent" else slice(0, ROT)
        s["q_out"][..., at] = turn(s["q"].float()).to(torch.bfloat16)
        out.append(s["q_out"])
    return tuple(out)


def _rows(s, cache, b, n):
    """The first n cached rows of sequence b, [n, width]."""
    c = s["c"]
    m = -(-n // c["page"])
    bits = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    rows = bits[s["table"][b, :m].long()].reshape(m * c["page"], -1)[:n]
    return rows.view(cache.dtype)


def _spans(c, most):
    """(sequence, its positions, first token, tokens) in runs of at most `most` pairs."""
    at = 0
    for b, (t, n) in enumerate(zip(*_shape(c))):
        step = max(1, most // n)
        for i in range(0, t, step):
            yield b, n, at + i, min(step, t - i)
        at += t


def _plain_scores(s):
    c = s["c"]
    T, H, n = s["q"].shape[0], c["heads"], c["n"]
    out = torch.full((T, n), -math.inf, device="cuda")
    for b, m, t0, t in _spans(c, (1 << 27) // H):
        k = _rows(s, s["keys"], b, m).float()
        q = s["q"][t0:t0 + t].float().reshape(t * H, IDX)
        p = torch.matmul(q, k.t()).clamp_min_(0.0).reshape(t, H, m)
        v = torch.matmul(s["w"][t0:t0 + t, None, :], p)[:, 0]
        if s["scales"] is not None:
            v = v * _rows(s, s["scales"], b, m)[:, 0]
        see = s["lengths"][t0:t0 + t, None]
        out[t0:t0 + t, :m] = torch.where(torch.arange(m, device="cuda") < see, v, -math.inf)
    return out


def _plain_attention(s):
    c = s["c"]
    H, k = c["heads"], c["k"]
    q, out = s["q"], torch.empty(*s["q"].shape[:2], LATENT, dtype=torch.bfloat16, device="cuda")
    for b, m, t0, t in _spans(c, (1 << 27) // H):
        if k:
            t1 = t0 + t
            for i in range(t0, t1, 128):  # tokens that are gathered together
                j = s["inds"][i:min(i + 128, t1)].long()
                rows = _rows(s, s["cache"], b, m)[j.clamp_min(0)].float()     # [tokens, k, WIDTH]
                z = torch.matmul(q[i:i + j.shape[0]].float(), rows.transpose(1, 2)) * s["scale"]
                z = z.masked_fill(j[:, None, :] < 0, -math.inf)
                p = torch.exp(z - z.amax(dim=2, keepdim=True))
                o = torch.matmul(p, rows[..., :LATENT]) / p.sum(dim=2, keepdim=True)
                out[i:i + j.shape[0]] = o.to(torch.bfloat16)
            continue
        rows = _rows(s, s["cache"], b, m).float()
        z = torch.matmul(q[t0:t0 + t].float().reshape(t * H, WIDTH), rows.t()) * s["scale"]
        hide = torch.arange(m, device="cuda") >= s["lengths"][t0:t0 + t, None]
        z = z.reshape(t, H, m).masked_fill(hide[:, None], -math.inf)
        p = torch.exp(z - z.amax(dim=2, keepdim=True))
        o = torch.matmul(p.reshape(t * H, m), rows[:, :LATENT]).reshape(t, H, LATENT)
        out[t0:t0 + t] = (o / p.sum(dim=2, keepdim=True)).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(s):
    c = s["c"]
    if not own:
        return {"append": _plain_append, "scores": _plain_scores,
                "attention": _plain_attention}[c["op"]](s)
    from deepseek_moe_layer_gb300 import binding
    if c["op"] == "append":
        latent, q, q_at = c["kind"] == "latent", None, None
        if c["heads"]:
            q, q_at = s["q"], s["q_out"][..., LATENT:] if latent else s["q_out"][..., :ROT]
        binding.cache_append(s["x"], s["slots"], s["cache"], scales=s["scales"],
                             norm_weight=s["weight"], norm_bias=s["bias"], eps=EPS,
                             positions=s["positions"], inv_freq=s["inv_freq"],
                             rope_at=LATENT if latent else 0, interleaved=c["interleaved"],
                             q=q, q_out=q_at)
        return tuple(s[k] for k in ("cache", "scales", "q_out") if s.get(k) is not None)
    if c["op"] == "scores":
        return binding.indexer_scores(s["q"], s["w"], s["keys"], s["table"], s["lengths"], c["n"],
                                      key_scales=s["scales"], cu_tokens=s["cu"])
    return binding.latent_attention(s["q"], s["cache"], s["table"], s["lengths"], s["scale"],
                                    inds=s["inds"], cu_tokens=s["cu"])


# ---------------------------------------------------------------------------------------
# values in 64 bits
# ---------------------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    dev = s.get("x", s.get("q")).device
    if c["op"] == "append":
        w, T = s["x"].shape[1], c["T"]
        angle = torch.outer(s["positions"].double(), s["inv_freq"].double())
        turn = torch.polar(torch.ones_like(angle), angle)

        def rotated(v):  # float64 [T, .., ROT]: each pair is a complex number
            pair = v.unflatten(-1, (-1, 2)) if c["interleaved"] else \
                v.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_complex(pair.contiguous())
            z = z * turn.reshape(T, *([1] * (v.dim() - 2)), -1)
            pair = torch.view_as_real(z)
            return (pair if c["interleaved"] else pair.transpose(-1, -2)).flatten(-2)

        r = s["x"].double()
        n = s["weight"].numel()
        head = r[:, :n]
        if s["bias"] is not None:
            head = head - head.sum(1, keepdim=True) / n
        head = head / ((head ** 2).sum(1, keepdim=True) / n + EPS).sqrt() * s["weight"].double()
        if s["bias"] is not None:
            head = head + s["bias"].double()
        r = torch.cat((head, r[:, n:]), 1)
        at = LATENT if c["kind"] == "latent" else 0
        r[:, at:at + ROT] = rotated(r[:, at:at + ROT])
        cache = s["cache"].float().double().reshape(-1, w)
        out = []
        if s["scales"] is None:
            cache[s["slots"]] = r
            out.append(cache.reshape(s["cache"].shape))
        else:
            top = r.abs().amax(1)
            e = torch.floor(torch.log2(top / E4M3_MAX)) - 1  # from below, then up
            for _ in range(3):
                e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)
            scale = torch.exp2(e)[:, None]
            v = r / scale
            ulp = torch.exp2((torch.frexp(v)[1] - 4).clamp_min(-9).double())
            cache[s["slots"]] = torch.round(v / ulp) * ulp
            scales = s["scales"].double().reshape(-1, 1)
            scales[s["slots"]] = scale
            out += [cache.reshape(s["cache"].shape), scales.reshape(s["scales"].shape)]
        if c["heads"]:
            full = s["q_out"].double()
            full[..., at:at + ROT] = rotated(s["q"].double())
            out.append(full)
        return tuple(out)

    T, H = s["q"].shape[:2]
    owner = [b for b, t in enumerate(_shape(c)[0]) for _ in range(t)]
    pos = torch.arange(s["table"].shape[1] * c["page"], device=dev)
    slot = s["table"].long()[:, pos // c["page"]] * c["page"] + pos % c["page"]  # [B, positions]
    lens = s["lengths"].tolist()
    if c["op"] == "scores":
        keys = s["keys"].float().reshape(-1, IDX)
        out = torch.full((T, c["n"]), -math.inf, dtype=torch.float64, device=dev)
        held, b = None, -1
        for t in range(T):
            if owner[t] != b:
                b = owner[t]
                at = slot[b, :max(l for l, o in zip(lens, owner) if o == b)]
                held = keys[at].double()
                if s["scales"] is not None:
                    held *= s["scales"].reshape(-1)[at].double()[:, None]
            z = held[:lens[t]] @ s["q"][t].double().t()
            out[t, :lens[t]] = (z * (z > 0)) @ s["w"][t].double()
        return out
    rows = s["cache"].reshape(-1, WIDTH)
    out = torch.zeros(T, H, LATENT, dtype=torch.float64, device=dev)
    for t in range(T):
        if s["inds"] is None:
            at = slot[owner[t], :lens[t]]
        else:
            at = slot[owner[t], s["inds"][t][s["inds"][t] >= 0].long()]
        kv = rows[at].double()
        p = torch.softmax(kv @ s["q"][t].double().t() * s["scale"], dim=0)
        out[t] = p.t() @ kv[:, :LATENT]
    return out
