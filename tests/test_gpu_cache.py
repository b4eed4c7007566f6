"""GPU parity of the operators over a paged cache (moe_cache_append, moe_indexer_scores,
moe_latent_attention) against plain evaluations in 64 bits.

Bounds, u = 2^-24 the rounding of fp32:
  append     a normalised column: the sums over W columns are off by W u relative, the root by a few
             u; a rotated pair by its angle's error (2^-25 turns to position 2^26, 2^-20 beyond) times
             the pair.  With `amp` the magnitudes that meet in a column:
             |y - ref| <= (W + 32) u amp + angle error * pair, then the rounding to bf16 (2^-8 |y|) or to
             e4m3 (half a step).
  scores     products of bf16 or e4m3 numbers are exact in fp32; 128 of them are added with up to
             2^-23 each (truncation counts as one unit), heads by a multiply-add each:
             |y - ref| <= s (sum_h |w_h| 128 2^-23 sum_k |q_hk k_k| + (H + 4) u sum_h |w_h| relu_h).
  attention  scores off by d = (576 2^-23 + 4 u) scale sum |q c| and, in base 2, by (|score| + 8) 2u; p
             rounded to bf16 once (2^-8), so with A = sum_j p_j |c_j|:
             |o - ref| <= 2^-8 |ref| + (2^-8 + 4 d + n u) A, the sums' n u among them.
"""
import math
import threading

import pytest
import torch

from deepseek_moe_layer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF, F8, F32, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32
U = 2.0 ** -24
INF = float("inf")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(*shape, g, dtype=F32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def ints(v, dtype=I32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def close(y, ref, tol, what=""):
    y, ref = y.double(), ref.double()
    same = (y == ref) | (y.isnan() & ref.isnan())
    bad = ~(((y - ref).abs() <= tol) | same)
    assert not bad.any(), (f"{what}: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{float(y[bad][0])} for {float(ref[bad][0])}")


# ---- append -----------------------------------------------------------------------------------

def rotate64(v, pos, freq, interleaved):
    """(rotated float64 [T, .., R], magnitude of each column's pair)."""
    a = (pos.double()[:, None] * freq.double()).reshape(len(pos), *([1] * (v.dim() - 2)), -1)
    c, s = torch.cos(a), torch.sin(a)
    x, y = (v[..., 0::2], v[..., 1::2]) if interleaved else v.chunk(2, -1)
    join = (lambda p, q: torch.stack((p, q), -1).flatten(-2)) if interleaved else \
        (lambda p, q: torch.cat((p, q), -1))
    pair = x.abs() + y.abs()
    return join(x * c - y * s, y * c + x * s), join(pair, pair)


def append64(x, weight, bias, eps, pos, freq, at, interleaved):
    """(rows in 64 bits, the bound of the fp32 evaluation)."""
    x = x.double()
    T, W = x.shape
    y, amp = x.clone(), torch.zeros_like(x)
    if weight is not None:
        n = weight.numel()
        h = x[:, :n]
        mean = h.mean(1, keepdim=True) if bias is not None else 0.0
        r = ((h - mean) ** 2).mean(1, keepdim=True).add(eps).rsqrt()
        y[:, :n] = (h - mean) * r * weight.double()
        spread = h.abs() + (h.abs().mean(1, keepdim=True) if bias is not None else 0.0)
        # (an error of the mean moves the deviations, and with them r)
        amp[:, :n] = spread * r * weight.double().abs() * (1 + (spread * r).amax(1, keepdim=True) *
                                                           (bias is not None))
        if bias is not None:
            y[:, :n] += bias.double()
            amp[:, :n] += bias.double().abs()
    tol = (W + 32) * U * amp
    if freq is not None:
        R = 2 * freq.numel()
        turn = 2.0 ** -25 if int(pos.abs().max()) < 1 << 26 else 2.0 ** -20
        rot, pair = rotate64(y[:, at:at + R], pos, freq, interleaved)
        _, err = rotate64(tol[:, at:at + R], pos * 0, freq, interleaved)
        tol[:, at:at + R] = err + (2 * math.pi * turn + 8 * U) * pair
        y[:, at:at + R] = rot
    return y, tol


def check_rows(got, scales, y, tol):
    if scales is None:
        close(got, y, 2.0 ** -8 * y.abs() + tol * 1.01, "rows")
        return
    T, W = y.shape
    b = y.reshape(T, -1, 128)
    top, t = b.abs().amax(-1), tol.reshape(T, -1, 128).amax(-1)
    s = scales.double()
    assert torch.equal(torch.frexp(scales)[0], torch.full_like(scales, 0.5)), "a power of two"
    # the smallest that holds the largest magnitude, give or take the evaluation's error
    assert bool(((top - t <= 448 * s) & ((top + t > 224 * s) | (s == 2.0 ** -126))).all())
    v = b / s[..., None]
    step = torch.exp2((torch.frexp(v)[1] - 4).clamp_min(-9).double())
    close(got.float().double().reshape(b.shape) * s[..., None], b,
          (step / 2 + 1e-12) * s[..., None] + 2 * tol.reshape(b.shape), "codes")


APPEND = [
    # T, W, norm columns, bias, R, at, interleaved, page, pages, 8 bits, heads, extra columns of x
    (1, 576, 512, False, 64, 512, True, 64, 2, False, 128, 1536),
    (37, 576, 512, False, 64, 512, False, 16, 7, False, 3, 0),
    (200, 128, 128, True, 64, 0, False, 64, 9, True, 0, 0),
    (65, 128, 128, True, 64, 0, True, 1, 300, False, 64, 8),
    (9, 1024, 1024, True, 1024, 0, False, 48, 2, True, 1, 0),
    (5, 8, 0, False, 0, 0, True, 3, 5, False, 0, 16),
    (33, 24, 8, False, 16, 8, True, 5, 9, False, 7, 0),
    (300, 256, 0, False, 128, 64, False, 64, 6, True, 2, 0),
    (64, 640, 600, True, 32, 592, True, 64, 2, False, 130, 0),
]


@pytest.mark.parametrize("T,W,n,bias,R,at,il,page,pages,f8,H,extra", APPEND)
def test_append(T, W, n, bias, R, at, il, page, pages, f8, H, extra):
    g = gen(T + W)
    x = (randn(T, W + extra, g=g) * 3 + 0.5).to(BF)[:, :W]
    weight = 1 + 0.2 * randn(n, g=g) if n else None
    b = 0.3 * randn(n, g=g) if bias else None
    freq = torch.exp2(-torch.rand(R // 2, generator=g, device=DEV) * 13) if R else None
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV).to(I32) if R else None
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T]
    slots[::5] = -1                      # without a place
    slots[1::7] += pages * page          # outside the cache
    cache = randn(pages, page, W, g=g).to(F8 if f8 else BF)
    scales = torch.full((pages, page, W // 128), 7.0, device=DEV) if f8 else None
    before = cache.clone()
    q = randn(T, H, R + 8, g=g, dtype=BF)[..., 8:] if H else None
    wide = torch.full((T, H, R + 24), 9.0, dtype=BF, device=DEV) if H else None
    out = binding.cache_append(x, slots, cache, scales=scales, norm_weight=weight, norm_bias=b,
                               positions=pos, inv_freq=freq, rope_at=at, interleaved=il, q=q,
                               q_out=wide[..., 16:16 + R] if H else None)
    y, tol = append64(x, weight, b, 1e-6, pos, freq, at, il)
    ok = (slots >= 0) & (slots < pages * page)
    once = (slots[:, None] == slots[ok]).sum(1) == 1  # (a slot that two tokens name holds either's)
    named = slots[ok]
    ok &= once
    at_ = slots[ok]
    flat = cache.view(torch.uint8).reshape(pages * page, -1).view(cache.dtype)
    check_rows(flat[at_].float() if f8 else flat[at_],
               scales.reshape(pages * page, -1)[at_] if f8 else None, y[ok], tol[ok])
    rest = torch.ones(pages * page, dtype=torch.bool, device=DEV)
    rest[named] = False
    old = before.view(torch.uint8).reshape(pages * page, -1)
    assert torch.equal(cache.view(torch.uint8).reshape(pages * page, -1)[rest], old[rest])
    if f8:
        assert bool((scales.reshape(pages * page, -1)[rest] == 7.0).all())
    if H:
        assert out[1].data_ptr() == wide[..., 16:16 + R].data_ptr()
        ref, pair = rotate64(q.double(), pos, freq, il)
        close(wide[..., 16:16 + R], ref, 2.0 ** -8 * ref.abs() + (2 * math.pi * 2.0 ** -25 + 8 * U) * pair, "q")
        assert bool((wide[..., :16] == 9.0).all()) and bool((wide[..., 16 + R:] == 9.0).all())


@pytest.mark.parametrize("first", [0, 1 << 20, (1 << 24) + 1, (1 << 26) - 70, (1 << 31) - 65, -100, -(1 << 31)])
def test_append_far_positions(first):
    T, R = 64, 64
    g = gen(3)
    pos = (first + torch.arange(T, device=DEV)).to(I32)
    freq = (10000.0 ** (-torch.arange(0, R, 2, device=DEV).double() / R)).float()
    x = randn(T, R, g=g, dtype=BF)
    cache = torch.zeros(1, T, R, dtype=BF, device=DEV)
    q = randn(T, 2, R, g=g, dtype=BF)
    keep = q.clone()
    _, qo = binding.cache_append(x, torch.arange(T, device=DEV), cache, positions=pos, inv_freq=freq, q=q, q_out=q)
    assert qo is q
    y, tol = append64(x, None, None, 0, pos.long(), freq, 0, True)
    check_rows(cache[0], None, y, tol)
    turn = 2.0 ** -25 if abs(first) + T < 1 << 26 else 2.0 ** -20
    ref, pair = rotate64(keep.double(), pos.long(), freq, True)
    close(q, ref, 2.0 ** -8 * ref.abs() + (2 * math.pi * turn + 8 * U) * pair, "q in place")


def turns64(pos, freq):
    """pos * f / (2 pi) behind the point, from whole numbers: float64 [positions, frequencies]."""
    bits = 320

    def arctan_of_inverse(n):
        term = total = (1 << bits) // n
        k = 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total

    two_pi = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))  # Machin's formula, in units of 2^-320
    out = []
    for p in pos:
        for f in freq:
            m, d = f.as_integer_ratio()  # d a power of two
            out.append((p * m << 2 * bits) // (d * two_pi) % (1 << bits) / (1 << bits))
    return torch.tensor(out, dtype=torch.float64).reshape(len(pos), len(freq))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("first,top", [(112736, 1.0), ((1 << 20) - 7, 1.0), (65710802, 1.0), ((1 << 26) - 40, 1.0),
                                       ((1 << 31) - 16, 1.0), (-(1 << 31), 1.0), ((1 << 31) - 16, 63.0)])
def test_append_angles(first, top, interleaved):
    """The angle itself: of every pair (u, v), u = 1 .. 2 and v are chosen so that u cos a - v sin a is almost 0,
    where the rounding to bf16 hides nothing.  Off by 2^-25 turns, and by 2 units of cos and sin and two
    roundings of the products: (2^-23 + 2 2^-24) of the pair."""
    T, R = 16, 64
    g = torch.Generator().manual_seed(first % 1000)
    freq = (torch.rand(R // 2, generator=g) ** 2 * top).float()
    freq[0], freq[1], freq[2] = 1.0, 0.7498942, 0.0013335214
    pos = [first + t for t in range(T)]
    a = turns64(pos, [float(f) for f in freq]) * 2 * math.pi
    c, s = torch.cos(a), torch.sin(a)
    u = 1 + torch.arange(128, dtype=torch.float64) / 128
    u = u.expand(T, R // 2, 128)
    v = (u * (c / s)[..., None]).clamp(-1e4, 1e4).to(BF).double()
    left = (u * c[..., None] - v * s[..., None]).abs() / (u + v.abs())
    best = left.argmin(-1, keepdim=True)
    u, v = u.gather(-1, best)[..., 0], v.gather(-1, best)[..., 0]
    join = (lambda p, q: torch.stack((p, q), -1).flatten(-2)) if interleaved else (lambda p, q: torch.cat((p, q), -1))
    x = join(u, v).to(DEV, BF)
    ref = join(u * c - v * s, v * c + u * s).to(DEV)
    pair = join(u + v.abs(), u + v.abs()).to(DEV)
    cache = torch.zeros(1, T, R, dtype=BF, device=DEV)
    _, q = binding.cache_append(x, torch.arange(T, device=DEV), cache, positions=ints(pos), inv_freq=freq.to(DEV),
                                interleaved=interleaved, q=x[:, None])
    tol = 2.0 ** -8 * ref.abs() + (2 * math.pi * 2.0 ** -25 + 2.0 ** -22) * pair
    close(cache[0], ref, tol, "rows")
    close(q[:, 0], ref, tol, "q")


def test_append_frequencies_without_a_value():
    x = torch.ones(4, 16, dtype=BF, device=DEV)
    freq = torch.tensor([0.0, INF, -INF, float("nan"), -0.5, 1e-40, 0.5, 1e-12], device=DEV)
    cache = torch.zeros(1, 4, 16, dtype=BF, device=DEV)
    binding.cache_append(x, torch.arange(4, device=DEV), cache, positions=ints([0, 1, 3, 1000]), inv_freq=freq)
    y = cache[0].view(4, 8, 2)
    assert bool(y[:, 1:4].isnan().all()) and bool((y[:, [0, 5, 7]] == 1.0).all())
    assert torch.equal(y[:, 4], y[:, 6].flip(-1)) and not torch.equal(y[1:, 4], y[1:, 6])


def test_append_not_finite():
    x = torch.ones(4, 128, dtype=BF, device=DEV)
    x[0, 5], x[1, 5], x[2, 5] = float("nan"), INF, -INF
    cache = torch.zeros(1, 4, 128, dtype=F8, device=DEV)
    scales = torch.zeros(1, 4, 1, device=DEV)
    binding.cache_append(x, torch.arange(4, device=DEV), cache, scales=scales)
    v = cache.float()[0]
    assert bool(v[:3, 5].isnan().all())
    v[:3, 5] = 256.0
    assert bool((v == 256.0).all()) and bool((scales == 2.0 ** -8).all())
    w = torch.ones(128, device=DEV)
    out = torch.zeros(1, 4, 128, dtype=BF, device=DEV)
    binding.cache_append(x, torch.arange(4, device=DEV), out, norm_weight=w)
    assert bool(out[0, 0].isnan().all()) and bool(out[0, 3].isfinite().all())
    zero = torch.zeros(1, 128, dtype=BF, device=DEV)  # a row of zeros: divided by the root of eps
    binding.cache_append(zero, ints([2], torch.int64), out, norm_weight=w)
    assert bool((out[0, 2] == 0).all())


def test_append_no_tokens():
    cache = torch.ones(2, 4, 64, dtype=BF, device=DEV)
    r = binding.cache_append(torch.zeros(0, 64, dtype=BF, device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV), cache)
    assert r is cache and bool((cache == 1).all())


@pytest.mark.parametrize("f8", [False, True])
def test_append_to_a_cache_without_pages(f8):
    g = gen(22)
    x, q, slots = randn(5, 128, g=g, dtype=BF), randn(5, 3, 64, g=g, dtype=BF), torch.arange(-1, 4, device=DEV)
    freq, pos = torch.rand(32, generator=g, device=DEV), ints([0, 1, 70, 5000, 100000])
    empty = torch.empty(0, 16, 128, dtype=F8 if f8 else BF, device=DEV)
    scales = torch.empty(0, 16, 1, device=DEV) if f8 else None
    cache, out = binding.cache_append(x, slots, empty, scales=scales, positions=pos, inv_freq=freq, q=q)
    assert cache is empty
    ref, pair = rotate64(q.double(), pos, freq, True)
    close(out, ref, 2.0 ** -8 * ref.abs() + (2 * math.pi * 2.0 ** -25 + 8 * U) * pair, "q")


# ---- a paged cache ------------------------------------------------------------------------------

class Batch:
    """Sequences of `lens` cached positions with `new` tokens at their ends, in scattered pages.  Rows that
    belong to nobody, and those behind a sequence's end in its last page, hold NaN."""

    def __init__(self, lens, new, page, width, g, dtype=BF, spare=3, scale=1.0):
        self.lens, self.new, self.page = lens, new, page
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g, device=DEV).to(I32)
        self.table = torch.full((len(lens), max(max(need), 1) + 1), -7, dtype=I32, device=DEV)
        rows = (randn(self.pages * page, width, g=g) * scale)
        used = torch.zeros(self.pages * page, dtype=torch.bool, device=DEV)
        at, self.slots = 0, []
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            j = torch.arange(n, device=DEV)
            s = self.table[b].long()[j // page] * page + j % page
            used[s] = True
            self.slots.append(s)
        rows[~used] = float("nan")
        self.rows = rows.clamp(-448, 448).to(dtype) if dtype is F8 else rows.to(dtype)
        self.cache = self.rows.view(self.pages, page, width)
        self.T = sum(new)
        self.cu = ints([sum(new[:b]) for b in range(len(new) + 1)])
        self.lengths = ints([max(0, n - t + i + 1) for n, t in zip(lens, new) for i in range(t)])

    def tokens(self):
        t = 0
        for b, n in enumerate(self.new):
            for _ in range(n):
                yield t, b, self.slots[b][:int(self.lengths[t])]
                t += 1

    def cu_or_none(self):
        return None if all(n == 1 for n in self.new) else self.cu


# ---- scores -------------------------------------------------------------------------------------

def scores_check(out, bt, q, w, ks, n):
    rows = bt.rows.float().double()
    for t, b, s in bt.tokens():
        s = s[:n]
        assert bool((out[t, len(s):n] == -INF).all()), f"token {t}: positions that it may not see"
        if len(s) == 0:
            continue
        k, qt, wt = rows[s], q[t].float().double(), w[t].double()
        z, mag = k @ qt.t(), k.abs() @ qt.abs().t()
        sc = ks.reshape(-1)[s].double() if ks is not None else 1.0
        ref = (z.clamp_min(0) @ wt) * sc
        tol = (128 * 2.0 ** -23 * (mag @ wt.abs()) + (len(wt) + 4) * U * (z.clamp_min(0) @ wt.abs())) * \
            (sc.abs() if ks is not None else 1.0)
        close(out[t, :len(s)], ref, tol + 1e-37, f"token {t}")


SCORES = [
    # lens, new tokens, page, heads, 8 bits, positions of a row (None: the longest sequence)
    ([1], [1], 1, 1, False, None),
    ([4096], [1], 64, 64, False, None),
    ([127, 128, 129, 1, 3000], [1, 1, 1, 1, 1], 64, 64, True, None),
    ([300, 17, 5], [3, 17, 1], 16, 32, False, None),
    ([500, 260, 77], [40, 33, 9], 48, 16, True, None),
    ([1000, 640], [70, 5], 64, 128, True, 900),
    ([333, 200], [21, 30], 7, 24, False, 1111),
    ([700], [129], 64, 80, True, None),
    ([257, 64, 900], [0, 2, 50], 128, 8, False, None),
    ([0, 40, 0], [1, 1, 1], 16, 64, True, 50),
    ([2000] * 9, [4] * 9, 64, 64, False, 2048),
    ([5], [5], 64, 100, False, None),
]


@pytest.mark.parametrize("lens,new,page,H,f8,n", SCORES)
def test_scores(lens, new, page, H, f8, n):
    g = gen(sum(lens) + H)
    bt = Batch(lens, new, page, 128, g, F8 if f8 else BF, scale=100.0 if f8 else 1.0)
    n = n or max(max(lens), 1)
    q = (randn(bt.T, H, 128, g=g) * (60 if f8 else 1)).clamp(-448, 448).to(F8 if f8 else BF)
    w = randn(bt.T, H, g=g)
    ks = (torch.rand(bt.pages, page, 1, generator=g, device=DEV) + 0.5) * 0.01 if f8 else None
    wide = torch.full((bt.T, n + 5), 3.0, device=DEV)
    out = binding.indexer_scores(q, w, bt.cache, bt.table, bt.lengths, n, key_scales=ks,
                                 cu_tokens=bt.cu_or_none(), out=wide[:, :n])
    assert out.data_ptr() == wide.data_ptr() and bool((wide[:, n:] == 3.0).all())
    scores_check(out, bt, q, w, ks, n)
    again = binding.indexer_scores(q, w, bt.cache, bt.table, bt.lengths, n, key_scales=ks,
                                   cu_tokens=bt.cu_or_none())
    assert torch.equal(again, out)
    binding.device_status()


def test_scores_rows_behind_the_last_sequence_and_pages_that_are_not_there():
    g = gen(5)
    bt = Batch([300, 200], [3, 2], 16, 128, g)
    T = bt.T + 4  # padded
    lengths = torch.cat([bt.lengths, ints([300] * 4)])
    q, w = randn(T, 64, 128, g=g, dtype=BF), randn(T, 64, g=g)
    out = torch.full((T, 300), 5.0, device=DEV)
    binding.indexer_scores(q, w, bt.cache, bt.table, lengths, 300, cu_tokens=bt.cu, out=out)
    assert bool((out[bt.T:] == 5.0).all())
    scores_check(out, bt, q, w, None, 300)
    for bad in (-1, bt.pages, 2 ** 31 - 1, -2 ** 31):
        table = bt.table.clone()
        table[0, 2] = bad
        got = binding.indexer_scores(q, w, bt.cache, table, lengths, 300, cu_tokens=bt.cu, out=torch.empty_like(out))
        assert bool((got[:3, 32:48] == -INF).all())
        keep = torch.ones(300, dtype=torch.bool, device=DEV)
        keep[32:48] = False
        assert torch.equal(got[:3, keep], out[:3, keep]) and torch.equal(got[3:5], out[3:5])


@pytest.mark.parametrize("f8", [False, True])
def test_scores_of_a_cache_without_pages(f8):
    g = gen(21)
    dtype = F8 if f8 else BF
    q, w = randn(3, 64, 128, g=g).to(dtype), randn(3, 64, g=g)
    keys = torch.empty(0, 16, 128, dtype=dtype, device=DEV)
    ks = torch.empty(0, 16, 1, device=DEV) if f8 else None
    out = binding.indexer_scores(q, w, keys, torch.zeros(3, 20, dtype=I32, device=DEV), ints([300, 1, 77]), 310,
                                 key_scales=ks)
    assert bool((out == -INF).all())
    binding.device_status()


def test_scores_not_finite():
    g = gen(6)
    bt = Batch([200], [1], 64, 128, g)
    q, w = randn(1, 64, 128, g=g, dtype=BF), torch.ones(1, 64, device=DEV)
    bt.rows[bt.slots[0][7], 3] = float("nan")
    out = binding.indexer_scores(q, w, bt.cache, bt.table, bt.lengths, 200)
    assert bool(out[0, 7].isnan()) and int(out.isnan().sum()) == 1
    w[0, 5] = float("nan")
    assert bool(binding.indexer_scores(q, w, bt.cache, bt.table, bt.lengths, 200).isnan().all())


@pytest.mark.parametrize("H", [5, 20, 33, 50, 64])
def test_scores_infinite_key(H):
    # the products of all heads are infinite: +inf where a head's is and its weight is not 0, 0 where
    # all are -inf; what pads the heads to a multiple of 16 must not be in it
    g = gen(7)
    bt = Batch([200], [1], 64, 128, g)
    q, w = randn(1, H, 128, g=g, dtype=BF), torch.rand(1, H, generator=g, device=DEV) + 0.5
    q[0, :, 3] = 1.0
    for value, want in ((INF, INF), (-INF, 0.0)):
        bt.rows[bt.slots[0][7], 3] = value
        out = binding.indexer_scores(q, w, bt.cache, bt.table, bt.lengths, 200)
        assert float(out[0, 7]) == want and int(out.isfinite().sum()) == 200 - (want == INF)


def test_scores_longest_row():
    # 2^31 - 512 positions, of which 130 are there
    g = gen(8)
    bt = Batch([130], [1], 64, 128, g)
    n = 2 ** 31 - 512
    q, w = randn(1, 64, 128, g=g, dtype=BF), randn(1, 64, g=g)
    out = binding.indexer_scores(q, w, bt.cache, bt.table, bt.lengths, n, out=torch.zeros(1, n, device=DEV))
    scores_check(out[:, :5000], bt, q, w, None, 5000)
    assert all(bool((part == -INF).all()) for part in out[0, 130:].split(1 << 28))


def test_ends_of_sequences_that_do_not_ascend():
    # no results to speak of, but calls that end and rows behind the last end as they were
    g = gen(9)
    bt = Batch([300, 200, 90], [3, 2, 4], 16, 576, g)
    keys = bt.cache[..., :128].contiguous()
    q, qi, w = (randn(9, 16, n, g=g, dtype=BF) for n in (576, 128, 1))
    for cu in ([5, 9, 2, 7], [1000000, -5, 1000000, 7], [-9, 2, 2 ** 31 - 1, 3], [7, 7, 7, 7], [4, 3, 2, -1]):
        kept = max(0, min(9, cu[3]))
        o = torch.full((9, 16, 512), 5.0, dtype=BF, device=DEV)
        binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, cu_tokens=ints(cu), out=o)
        s = torch.full((9, 300), 5.0, device=DEV)
        binding.indexer_scores(qi, w[..., 0].float().contiguous(), keys, bt.table, bt.lengths, 300,
                               cu_tokens=ints(cu), out=s)
        assert bool((s[kept:] == 5.0).all()) and (kept > 0 or bool((o == 5.0).all()))
        binding.device_status()


# ---- attention ----------------------------------------------------------------------------------

def attention_check(out, lse, bt, q, scale, inds=None):
    rows = bt.rows.double()
    for t, b, s in bt.tokens():
        if inds is not None:
            j = inds[t][:int(bt.lengths[t])]
            j = j[(j >= 0) & (j < int(bt.lengths[t]))].long()
            s = bt.slots[b][j]
        if len(s) == 0:
            assert bool((out[t] == 0).all()) and (lse is None or bool((lse[t] == -INF).all()))
            continue
        c, qt = rows[s], q[t].double()
        z, mag = qt @ c.t() * scale, qt.abs() @ c.abs().t() * abs(scale)
        d = ((576 * 2.0 ** -23 + 4 * U) * mag + (z.abs() + 8) * 2 * U).amax(1, keepdim=True)
        p = torch.softmax(z, 1)
        ref, A = p @ c[:, :512], p @ c[:, :512].abs()
        close(out[t], ref, 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 4 * d + len(s) * U) * A, f"token {t}")
        if lse is not None:
            want = torch.logsumexp(z, 1)
            close(lse[t], want, 2 * d[:, 0] + (len(s) + 16) * U + 4 * U * want.abs(), f"lse of token {t}")


ATTENTION = [
    # lens, new tokens, page, heads, k (0: all positions), scale of the scores
    ([1], [1], 64, 128, 0, 1.0),
    ([4096], [1], 64, 128, 0, 1.0),
    ([127, 128, 129, 1, 700], [1] * 5, 64, 128, 0, 1.0),
    ([0, 60, 0, 300], [1] * 4, 16, 64, 0, 1.0),
    ([900, 40], [3, 5], 48, 16, 0, 1.0),
    ([300, 77, 513], [20, 9, 1], 7, 24, 0, 2.0),
    ([140], [140], 64, 3, 0, 1.0),
    ([260], [130], 128, 1, 0, 1.0),
    ([500, 333], [2, 4], 64, 100, 0, 4.0),
    ([600, 100, 0, 50], [0, 2, 1, 0], 1, 128, 0, 1.0),
    ([3000], [3], 64, 128, 257, 1.0),
    ([500, 90], [5, 2], 16, 16, 64, 1.0),
    ([64, 2000], [1, 1], 64, 128, 2048, 1.0),
    ([200], [200], 64, 64, 33, 1.0),
    ([700] * 90, [1] * 90, 64, 128, 0, 1.0),
    ([2300, 100, 1500, 40, 5, 1999], [1] * 6, 64, 128, 0, 8.0),
]


def select(bt, k, g):
    inds = torch.full((bt.T, k), -1, dtype=I32, device=DEV)
    for t, b, s in bt.tokens():
        n = len(s)
        pick = torch.randperm(n, generator=g, device=DEV)[:k].sort().values if n else torch.zeros(0, device=DEV)
        inds[t, :len(pick)] = pick.to(I32)
    return inds


@pytest.mark.parametrize("lens,new,page,H,k,sharp", ATTENTION)
def test_attention(lens, new, page, H, k, sharp):
    g = gen(sum(lens) + H + k)
    bt = Batch(lens, new, page, 576, g)
    wide = randn(bt.T, H + 1, 584, g=g, dtype=BF)
    q = wide[:, 1:, 8:]  # tokens and heads strided
    scale = sharp / math.sqrt(192)
    inds = select(bt, k, g) if k else None
    args = dict(inds=inds, cu_tokens=bt.cu_or_none(), want_lse=True)
    out, lse = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, scale, **args)
    attention_check(out, lse, bt, q, scale, inds)
    given = torch.empty_like(out)
    again, lse2 = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, scale, out=given, **args)
    assert again is given and torch.equal(again, out) and torch.equal(lse2, lse)
    binding.device_status()


@pytest.mark.parametrize("rise", [3.0, 40.0, -40.0])
def test_attention_rising_maximum(rise):
    """Scores that climb (or fall) along the positions move the running maximum in every tile, and in
    some rows only; large ones make p of all but the last positions 0."""
    g = gen(8)
    bt = Batch([1500, 800], [1, 1], 64, 576, g, scale=0.05)
    for b, s in enumerate(bt.slots):
        bt.rows[s, 540] = (torch.arange(len(s), device=DEV) * (rise / 64)).to(BF)
    q = randn(2, 128, 576, g=g, dtype=BF)
    q[:, ::3, 540] = 0.0
    q[:, 1::3, 540] = 1.0
    out, lse = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.5, want_lse=True)
    attention_check(out, lse, bt, q, 0.5)


def test_attention_hidden_rows_may_hold_anything():
    """What a token may not see changes no bit of its output: rows behind its length that later tokens
    of the segment see, rows that are not selected, pages that are not there."""
    g = gen(9)
    bt = Batch([200], [6], 64, 576, g)
    q = randn(6, 16, 576, g=g, dtype=BF)
    ref = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, cu_tokens=bt.cu)
    for v in (float("nan"), INF, -INF, torch.finfo(BF).min):
        bt2 = bt.rows.clone()
        bt2[bt.slots[0][197], :] = v  # seen by the last three tokens
        got = binding.latent_attention(q, bt2.view(bt.cache.shape), bt.table, bt.lengths, 0.1, cu_tokens=bt.cu)
        assert torch.equal(got[:3], ref[:3])
        if math.isnan(v):
            assert bool(got[3:].isnan().all())
    bt = Batch([400, 400], [1, 1], 64, 576, g)
    q = randn(2, 128, 576, g=g, dtype=BF)
    inds = select(bt, 64, g)
    ref = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, inds=inds)
    rows = bt.rows.clone()
    for b in range(2):
        hidden = torch.ones(400, dtype=torch.bool, device=DEV)
        hidden[inds[b].long()] = False
        rows[bt.slots[b][hidden]] = float("nan")
    got = binding.latent_attention(q, rows.view(bt.cache.shape), bt.table, bt.lengths, 0.1, inds=inds)
    assert torch.equal(got, ref)


def test_attention_pages_that_are_not_there():
    g = gen(10)
    bt = Batch([300, 150], [2, 1], 16, 576, g)
    q = randn(3, 128, 576, g=g, dtype=BF)
    for bad in (-1, bt.pages, 2 ** 31 - 1, -2 ** 31):
        table = bt.table.clone()
        table[0, 3:5] = bad
        out = binding.latent_attention(q, bt.cache, table, bt.lengths, 0.1, cu_tokens=bt.cu)
        keep = torch.ones(300, dtype=torch.bool, device=DEV)
        keep[48:80] = False
        for t in range(2):
            c = bt.rows[bt.slots[0][:299 + t][keep[:299 + t]]].double()
            p = torch.softmax(q[t].double() @ c.t() * 0.1, 1)
            ref, A = p @ c[:, :512], p @ c[:, :512].abs()
            close(out[t], ref, 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 1e-4) * A, f"token {t}")
        table[:] = bad
        out, lse = binding.latent_attention(q, bt.cache, table, bt.lengths, 0.1, cu_tokens=bt.cu, want_lse=True)
        assert bool((out == 0).all()) and bool((lse == -INF).all())
    empty = torch.empty(0, 16, 576, dtype=BF, device=DEV)  # a cache without pages
    out = binding.latent_attention(q, empty, bt.table, bt.lengths, 0.1, cu_tokens=bt.cu)
    assert bool((out == 0).all())


def test_attention_entries_of_a_selection():
    g = gen(11)
    bt = Batch([100, 100, 20], [1, 1, 1], 64, 576, g)
    q = randn(3, 32, 576, g=g, dtype=BF)
    inds = torch.full((3, 40), -1, dtype=I32, device=DEV)
    inds[0, :6] = ints([5, 200, -3, 7, 2 ** 31 - 1, 5])  # two that are not there, one twice
    inds[2, :30] = torch.arange(30, dtype=I32, device=DEV)  # entries from the 20th on are not looked at
    out, lse = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, inds=inds, want_lse=True)
    c = bt.rows[bt.slots[0][ints([5, 7, 5]).long()]].double()
    p = torch.softmax(q[0].double() @ c.t() * 0.1, 1)
    close(out[0], p @ c[:, :512], 2.0 ** -8 * (p @ c[:, :512]).abs() + (2.0 ** -8 + 1e-4) * (p @ c[:, :512].abs()))
    assert bool((out[1] == 0).all()) and bool((lse[1] == -INF).all())
    c = bt.rows[bt.slots[2]].double()
    p = torch.softmax(q[2].double() @ c.t() * 0.1, 1)
    close(out[2], p @ c[:, :512], 2.0 ** -8 * (p @ c[:, :512]).abs() + (2.0 ** -8 + 1e-4) * (p @ c[:, :512].abs()))


def test_attention_rows_behind_the_last_sequence():
    g = gen(12)
    bt = Batch([300, 90], [3, 2], 64, 576, g)
    T = bt.T + 5
    lengths = torch.cat([bt.lengths, ints([90] * 5)])
    q = randn(T, 128, 576, g=g, dtype=BF)
    out = torch.full((T, 128, 512), 5.0, dtype=BF, device=DEV)
    binding.latent_attention(q, bt.cache, bt.table, lengths, 0.1, cu_tokens=bt.cu, out=out)
    assert bool((out[bt.T:] == 5.0).all())
    attention_check(out, None, bt, q, 0.1)


def test_attention_not_finite_scores():
    g = gen(13)
    bt = Batch([300], [1], 64, 576, g)
    q = randn(1, 128, 576, g=g, dtype=BF)
    ref = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1)
    q2 = q.clone()
    q2[0, 17, 3] = float("nan")
    out = binding.latent_attention(q2, bt.cache, bt.table, bt.lengths, 0.1)
    assert bool(out[0, 17].isnan().all())
    assert torch.equal(out[0, :17], ref[0, :17]) and torch.equal(out[0, 18:], ref[0, 18:])
    # scores that are all alike, and a scale of 0: the mean
    out = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.0)
    mean = bt.rows[bt.slots[0], :512].double()
    close(out[0], mean.mean(0).expand(128, 512), (2.0 ** -8 + 300 * U) * 2 * mean.abs().mean(0))


@pytest.mark.parametrize("lens", [[100, 5], [4096], [2000] * 12, [3000] * 2, [1, 128, 129]])
@pytest.mark.parametrize("k", [0, 300])
def test_attention_scores_of_minus_infinity(lens, k):
    """Scores that are all -inf have no softmax: NaN, in one piece and in many, told from no positions (0).  With
    one finite score among them, wherever it lies, the output is that row."""
    g = gen(23)
    bt = Batch(lens, [1] * len(lens), 64, 576, g)
    q = randn(bt.T, 20, 576, g=g, dtype=BF)
    q[:, :, 540] = -1.0
    q[:, 5, 540] = 0.0  # 0 * inf
    inds = select(bt, k, g) if k else None
    rows = bt.rows.clone()
    for s in bt.slots:
        rows[s, 540] = INF

    def run(lengths=bt.lengths):
        return binding.latent_attention(q, rows.view(bt.cache.shape), bt.table, lengths, 0.1, inds=inds, want_lse=True)

    out, lse = run()
    assert bool(out.isnan().all())
    lse[:, 5] = -INF  # (NaN there)
    assert bool((lse == -INF).all())
    out, lse = run(torch.zeros_like(bt.lengths))
    assert bool((out == 0).all()) and bool((lse == -INF).all())
    heads = [h for h in range(20) if h != 5]
    for where in (0.0, 0.4, 0.99):
        at = [int(where * len(s)) if inds is None else int(inds[t][int(where * min(k, len(s)))])
              for t, s in enumerate(bt.slots)]
        for s, j in zip(bt.slots, at):
            rows[s[j], 540] = 1.0
        out, lse = run()
        c = torch.stack([rows[s[j]] for s, j in zip(bt.slots, at)])
        assert torch.equal(out[:, heads], c[:, None, :512].expand(-1, 19, -1))
        z = (q.double() * c[:, None].double()).sum(-1) * 0.1
        mag = (q.double() * c[:, None].double()).abs().sum(-1) * 0.1
        close(lse[:, heads], z[:, heads], ((576 * 2.0 ** -23 + 4 * U) * mag + 40 * U * (z.abs() + 8))[:, heads], "lse")
        for s, j in zip(bt.slots, at):
            rows[s[j], 540] = INF
    binding.device_status()


@pytest.mark.parametrize("lens,new,H", [
    ([3001, 2000, 2700, 1500, 1, 2999, 900, 2222, 128, 129, 1777, 2048, 2600, 3000, 640, 2500, 1999], [4] * 17, 16),
    ([5000, 5000], [1, 1], 128), ([9000, 100, 3000], [1, 2, 9], 32), ([2560] * 30, [1] * 30, 128),
    ([1280 + 128 * i for i in range(20)], [1] * 20, 64), ([640] * 50 + [4000], [1] * 51, 128),
    ([0, 8000, 0, 7000, 0], [1, 1, 1, 1, 1], 100),
])
def test_attention_of_a_few_long_sequences(lens, new, H):
    # segments of several tiles, fewer than CTA pairs: pieces of one segment each, or runs across them
    g = gen(sum(lens))
    bt = Batch(lens, new, 64, 576, g)
    q = randn(bt.T, H, 576, g=g, dtype=BF)
    out, lse = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, cu_tokens=bt.cu_or_none(), want_lse=True)
    attention_check(out, lse, bt, q, 0.1)
    again = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, cu_tokens=bt.cu_or_none())
    assert torch.equal(again, out)
    binding.device_status()


@pytest.mark.parametrize("shape", ["even", "one long", "many short", "drafts"])
@pytest.mark.parametrize("count", [75, 76, 77, 151, 152, 153, 305])
def test_runs_of_the_list_of_tiles(count, shape):
    # as many sequences as there are CTA pairs or CTAs, one fewer and one more: runs that begin and end
    # at, before and behind the borders of sequences
    g = gen(count)
    lens = {"even": [256] * count, "one long": [9000] + [130] * (count - 1), "drafts": [300] * count,
            "many short": [(37 * i) % 129 for i in range(count)]}[shape]
    new = [1 + i % 3 if shape == "drafts" else 1 for i in range(count)]
    bt = Batch(lens, new, 32, 576, g)
    q, qi, w = randn(bt.T, 20, 576, g=g, dtype=BF), randn(bt.T, 32, 128, g=g, dtype=BF), randn(bt.T, 32, g=g)
    out, lse = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, cu_tokens=bt.cu_or_none(), want_lse=True)
    attention_check(out, lse, bt, q, 0.1)
    keys = bt.cache[..., :128].contiguous()
    n = max(lens)
    s = binding.indexer_scores(qi, w, keys, bt.table, bt.lengths, n, cu_tokens=bt.cu_or_none())
    bt.rows = keys.view(-1, 128)
    scores_check(s, bt, qi, w, None, n)
    binding.device_status()


@pytest.mark.parametrize("H,before,prompt,behind", [(128, 40, 150, 41), (16, 3, 260, 90), (64, 0, 130, 130), (20, 130, 33, 0)])
def test_one_prompt_beside_decoding_sequences(H, before, prompt, behind):
    # one sequence with many new tokens among sequences with one each: groups and segments of every kind
    g = gen(24 + H)
    lens = [(97 * i) % 700 + 1 for i in range(before)] + [prompt + 200] + [(61 * i) % 900 + 1 for i in range(behind)]
    bt = Batch(lens, [1] * before + [prompt] + [1] * behind, 32, 576, g)
    q, qi, w = randn(bt.T, H, 576, g=g, dtype=BF), randn(bt.T, H, 128, g=g, dtype=BF), randn(bt.T, H, g=g)
    out, lse = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, cu_tokens=bt.cu, want_lse=True)
    attention_check(out, lse, bt, q, 0.1)
    inds = select(bt, 130, g)
    attention_check(binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, inds=inds, cu_tokens=bt.cu), None,
                    bt, q, 0.1, inds)
    keys = bt.cache[..., :128].contiguous()
    s = binding.indexer_scores(qi, w, keys, bt.table, bt.lengths, max(lens), cu_tokens=bt.cu)
    bt.rows = keys.view(-1, 128)
    scores_check(s, bt, qi, w, None, max(lens))
    binding.device_status()


# ---- a cache behind 32-bit offsets, graphs, streams, failed launches ------------------------------

def test_rows_behind_32_bit_offsets():
    """4.2 million rows of 576: their bytes, and their elements, pass 2^32 and 2^31."""
    g = gen(14)
    page, pages = 64, 66000
    cache = torch.empty(pages, page, 576, dtype=BF, device=DEV)
    last = pages - 1
    slots = torch.arange(last * page, last * page + 50, device=DEV)
    x = randn(50, 576, g=g, dtype=BF)
    binding.cache_append(x, slots, cache)
    assert torch.equal(cache[last, :50], x)
    table, n = ints([[last]]), ints([50])
    q = randn(1, 128, 576, g=g, dtype=BF)
    small = binding.latent_attention(q, cache[last:].clone(), ints([[0]]), n, 0.1)
    assert torch.equal(binding.latent_attention(q, cache, table, n, 0.1), small)
    keys = cache.view(-1)[:pages * page * 4 * 128].view(-1, page, 128)  # 17 million index keys
    at = keys.shape[0] - 1
    keys[at] = randn(page, 128, g=g, dtype=BF)
    qi, w = randn(1, 64, 128, g=g, dtype=BF), randn(1, 64, g=g)
    one = binding.indexer_scores(qi, w, keys[at:].clone(), ints([[0]]), n, 64)
    assert torch.equal(binding.indexer_scores(qi, w, keys, ints([[at]]), n, 64), one)


def _serving(g):
    """A decode step's buffers: caches of latent rows and index keys with room for one more token."""
    lens = [900, 33, 2100]
    s = {"lat": Batch(lens, [1, 1, 1], 64, 576, g), "key": Batch(lens, [1, 1, 1], 64, 128, g)}
    s["key"].table = s["lat"].table  # one block table for both
    s["key"].slots = s["lat"].slots
    for b in (s["lat"], s["key"]):
        b.rows.copy_(randn(*b.rows.shape, g=g).to(BF))
    s.update(x=randn(3, 576, g=g, dtype=BF), xk=randn(3, 128, g=g, dtype=BF),
             q=randn(3, 128, 192, g=g, dtype=BF), qa=randn(3, 128, 576, g=g, dtype=BF),
             qi=randn(3, 64, 128, g=g, dtype=BF), w=randn(3, 64, g=g) / 64,
             norm=1 + 0.1 * randn(512, g=g), kw=1 + 0.1 * randn(128, g=g), kb=0.1 * randn(128, g=g),
             freq=(10000.0 ** (-torch.arange(0, 64, 2, device=DEV).double() / 64)).float(),
             pos=ints([n - 1 for n in lens]), slots=torch.stack([v[-1] for v in s["lat"].slots]))
    return s


def _step(s, k):
    """One token of each sequence: into the caches, scores, selection, attention."""
    lat, key = s["lat"], s["key"]
    binding.cache_append(s["x"], s["slots"], lat.cache, norm_weight=s["norm"], positions=s["pos"],
                         inv_freq=s["freq"], rope_at=512, q=s["q"][..., 128:], q_out=s["qa"][..., 512:])
    binding.cache_append(s["xk"], s["slots"], key.cache, norm_weight=s["kw"], norm_bias=s["kb"],
                         positions=s["pos"], inv_freq=s["freq"], interleaved=False,
                         q=s["qi"][..., :64], q_out=s["qi"][..., :64])
    sc = binding.indexer_scores(s["qi"], s["w"], key.cache, lat.table, lat.lengths, max(lat.lens))
    inds = binding.indexer_topk(sc, k, lengths=lat.lengths)
    return sc, inds, binding.latent_attention(s["qa"], lat.cache, lat.table, lat.lengths, 0.07, inds=inds)


def test_a_step_of_them_together():
    s = _serving(gen(15))
    s["qi0"] = s["qi"].clone()
    sc, inds, out = _step(s, 512)
    lat, key = s["lat"], s["key"]
    y, tol = append64(s["x"], s["norm"], None, 1e-6, s["pos"], s["freq"], 512, True)
    check_rows(lat.rows[s["slots"]], None, y, tol)
    y, tol = append64(s["xk"], s["kw"], s["kb"], 1e-6, s["pos"], s["freq"], 0, False)
    check_rows(key.rows[s["slots"]], None, y, tol)
    scores_check(sc, key, s["qi"], s["w"], None, 2100)
    for t, n in enumerate(lat.lens):
        want = torch.topk(sc[t], min(512, n)).indices.sort().values
        assert torch.equal(inds[t, :min(512, n)].long(), want) and bool((inds[t, min(512, n):] == -1).all())
    attention_check(out, None, lat, s["qa"], 0.07, inds)
    # a selection of everything is attention over everything
    s["qi"].copy_(s["qi0"])
    sc, inds, out = _step(s, 4096)
    dense = binding.latent_attention(s["qa"], lat.cache, lat.table, lat.lengths, 0.07)
    A = dense.float().abs().amax()
    assert float((out.float() - dense.float()).abs().amax()) <= 2.0 ** -6 * float(A)
    binding.device_status()


def test_captured_steps():
    """Two captured graphs of the same step, replayed in turn and with inputs that changed in between."""
    s = _serving(gen(16))
    qi = s["qi"].clone()
    for _ in range(2):
        s["qi"].copy_(qi)
        _step(s, 256)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            s["qi"].copy_(qi)
            graphs.append((gr, _step(s, 256)))
    for seed in (1, 2):
        g = gen(seed)
        s["x"].copy_(randn(3, 576, g=g))
        s["q"].copy_(randn(3, 128, 192, g=g))
        s["lat"].lengths.copy_(ints([850 + seed, 20 + seed, 2000 + seed]))
        s["qi"].copy_(qi)
        want = _step(s, 256)
        for gr, got in graphs:
            for t in got:
                t.zero_()
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
    binding.device_status()


def test_calls_on_streams_of_their_own():
    g = gen(17)
    bt = Batch([3000, 1200], [1, 1], 64, 576, g)
    kt = Batch([3000, 1200], [1, 1], 64, 128, g)
    q = [randn(2, 128, 576, g=g, dtype=BF) for _ in range(4)]
    qi = [randn(2, 64, 128, g=g, dtype=BF) for _ in range(4)]
    w = randn(2, 64, g=g)
    want = [binding.latent_attention(v, bt.cache, bt.table, bt.lengths, 0.1) for v in q]
    wants = [binding.indexer_scores(v, w, kt.cache, kt.table, kt.lengths, 3000) for v in qi]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [None] * 8

    def work(i):
        for _ in range(5):
            got[i] = binding.latent_attention(q[i], bt.cache, bt.table, bt.lengths, 0.1, stream=streams[i])
            got[4 + i] = binding.indexer_scores(qi[i], w, kt.cache, kt.table, kt.lengths, 3000, stream=streams[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(got, want + wants):
        assert torch.equal(a, b)
    binding.device_status()


def test_failed_launches():
    g = gen(18)
    bt = Batch([3000], [1], 64, 576, g)
    q = randn(1, 128, 576, g=g, dtype=BF)
    want = binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1)
    out = torch.full_like(want, 5.0)
    key = torch.zeros(1, 64, 128, dtype=BF, device=DEV)
    sc = torch.full((1, 64), 5.0, device=DEV)
    try:
        binding.set_fault(binding.MOE_FAULT_LAUNCH, 0)
        with pytest.raises(binding.MoeError, match="attention kernel: injected"):
            binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, out=out)
        with pytest.raises(binding.MoeError, match="scores kernel: injected"):
            binding.indexer_scores(torch.zeros(1, 8, 128, dtype=BF, device=DEV), torch.zeros(1, 8, device=DEV),
                                   key, ints([[0]]), ints([64]), 64, out=sc)
        with pytest.raises(binding.MoeError, match="append kernel: injected"):
            binding.cache_append(torch.ones(1, 128, dtype=BF, device=DEV), ints([0], torch.int64), key)
        torch.cuda.synchronize()
        assert bool((out == 5.0).all()) and bool((sc == 5.0).all()) and bool((key == 0).all())
        binding.set_fault(binding.MOE_FAULT_LAUNCH, 1)
        with pytest.raises(binding.MoeError, match="attention join: injected"):
            binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, out=out)
    finally:
        binding.set_fault(binding.MOE_FAULT_NONE)
    assert torch.equal(binding.latent_attention(q, bt.cache, bt.table, bt.lengths, 0.1, out=out), want)
    binding.device_status()
