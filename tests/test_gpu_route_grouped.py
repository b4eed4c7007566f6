"""GPU parity of the group-limited softmax gate (moe_route_softmax_grouped) against a plain
evaluation in 64 bits: the experts and their order equal, the weights within the fp32 bound
derived at check()."""
import numpy as np
import pytest
import torch

from deepseek_moe_layer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def reference(logits, bias, K, G, tg, norm, scale):
    l = logits.double().cpu().numpy()
    l = np.where(np.isnan(l), -np.inf, l)
    rows, E = l.shape
    m = l.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(m == np.inf, (l == np.inf).astype(float),
                     np.where(m == -np.inf, 0.0, np.exp(l - np.where(np.isinf(m), 0, m))))
    z = e.sum(axis=1, keepdims=True)
    p = np.divide(e, z, out=np.zeros_like(e), where=z > 0)
    # without a bias the order is the logits' (equal to p's wherever p tells them apart)
    v = l.copy() if bias is None else p + bias.double().cpu().numpy()[None]
    v = np.where(np.isnan(v), -np.inf, v)
    inds = np.empty((rows, K), np.int32)
    for r in range(rows):
        best = v[r].reshape(G, E // G).max(axis=1)
        kept = sorted(range(G), key=lambda g: (-best[g], g))[:tg]
        cand = [x for x in range(E) if x // (E // G) in kept]
        inds[r] = sorted(cand, key=lambda x: (-v[r, x], x))[:K]
    w = np.take_along_axis(p, inds, axis=1)
    if norm and K > 1:
        s = w.sum(axis=1, keepdims=True)
        w = np.divide(w, s, out=np.zeros_like(w), where=s > 0)
    return inds, w * scale


def check(logits, K, G, tg, norm, scale=2.5, bias=None):
    inds, scores = binding.route_softmax_grouped(logits, K, G, tg, norm, scale, bias=bias)
    torch.cuda.synchronize()
    ri, rw = reference(logits, bias, K, G, tg, norm, scale)
    assert np.array_equal(inds.cpu().numpy(), ri)
    # fp32: l - m off by 2^-24 |l - m| <= 2^-24 * 104 before exp underflows; expf two steps;
    # Z at most 32 + 5 additions, again for the K weights; the products and quotients: below
    # (104 + 4 + 37 + 37 + 6) * 2^-24 < 2^-16 of the weight; subnormal p off by 2^-149 each
    got = scores.double().cpu().numpy()
    assert np.all(np.abs(got - rw) <= 2.0 ** -16 * np.abs(rw) + abs(scale) * 2.0 ** -126)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("rows,E,K,G,tg,norm", [
    (1, 1, 1, 1, 1, True), (3, 2, 2, 2, 2, True), (7, 8, 3, 4, 2, False), (64, 33, 5, 3, 2, True),
    (50, 60, 4, 1, 1, False), (200, 160, 6, 8, 3, False), (128, 256, 8, 8, 4, True),
    (40, 250, 8, 10, 9, True), (33, 288, 8, 32, 3, True), (20, 512, 32, 4, 1, False),
    (9, 1024, 32, 16, 5, True), (5, 992, 7, 31, 1, True), (300, 64, 1, 64 // 4, 1, True)])
def test_shapes(rows, E, K, G, tg, norm, with_bias, dtype):
    g = torch.Generator(device=DEV).manual_seed(rows + E)
    logits = (2 * torch.randn(rows, E, generator=g, device=DEV)).to(dtype)
    bias = 0.02 * torch.randn(E, generator=g, device=DEV) if with_bias else None
    check(logits, K, G, tg, norm, bias=bias)


@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lowest_index(with_bias):
    g = torch.Generator(device=DEV).manual_seed(5)
    logits = torch.randint(-2, 3, (300, 48), generator=g, device=DEV).float()
    bias = torch.zeros(48, device=DEV) if with_bias else None
    check(logits, 6, 6, 3, True, bias=bias)
    check(torch.zeros(4, 48, device=DEV), 6, 6, 3, True, bias=bias)


def test_bias_gaps_that_fp32_cannot_tell():
    """v_j equal to about 2^-30 of itself for many experts: the order is that of 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(6)
    rows, E = 64, 64
    base = torch.randn(E, generator=g, device=DEV)
    logits = base[None].repeat(rows, 1)
    p = torch.softmax(base.double(), 0)
    bias = (0.5 - p).float()  # p + bias = 0.5 to within fp32's rounding of the bias
    logits += 1e-6 * torch.randn(rows, E, generator=g, device=DEV)
    for G, tg in ((1, 1), (8, 3)):
        check(logits, 8, G, tg, False, bias=bias)


@pytest.mark.parametrize("with_bias", [False, True])
def test_rows_with_infinities_and_nan(with_bias):
    inf, nan = float("inf"), float("nan")
    E = 40
    l = torch.linspace(-3, 3, E).repeat(8, 1)
    l[0] = -inf                      # nothing left: weights 0, lowest experts
    l[1, 5:] = -inf                  # five experts left
    l[2, 7] = inf
    l[3, [3, 9]] = inf
    l[4, [0, 39]] = nan
    l[5] = nan
    l[6] = torch.finfo(torch.float32).min
    l[7] = torch.linspace(-1e4, 1e4, E)
    bias = torch.zeros(E) if with_bias else None
    for norm in (False, True):
        check(l.to(DEV), 6, 4, 2, norm, bias=bias.to(DEV) if with_bias else None)
        check(l.to(DEV), 6, 1, 1, norm, bias=bias.to(DEV) if with_bias else None)


def test_nan_bias_is_chosen_last():
    g = torch.Generator(device=DEV).manual_seed(7)
    bias = torch.zeros(16, device=DEV)
    bias[2] = float("nan")
    check(torch.randn(30, 16, generator=g, device=DEV), 4, 4, 2, True, bias=bias)
    check(torch.randn(30, 16, generator=g, device=DEV), 16, 1, 1, True, bias=bias)


def test_leading_dims_and_large_batch():
    g = torch.Generator(device=DEV).manual_seed(8)
    l = torch.randn(3, 700, 96, generator=g, device=DEV)
    i1, s1 = binding.route_softmax_grouped(l, 4, 3, 2, True, 1.0)
    i2, s2 = binding.route_softmax_grouped(l.view(-1, 96), 4, 3, 2, True, 1.0)
    assert i1.shape == (3, 700, 4) and torch.equal(i1.view(-1, 4), i2) and torch.equal(s1.view(-1, 4), s2)
    check(l.view(-1, 96)[:500], 4, 3, 2, True, 1.0)


def dominant_rows(E, K, G, seed, rows=256):
    """Rows whose border between K and K + 1 lies between two experts of tiny probability some
    2^-24 apart, and an expert of probability near 1 whose bias puts its value beside theirs: what
    fp32 leaves of that value is off by many times the gap, in either direction."""
    r = np.random.default_rng(seed)
    eg = E // G
    base = r.normal(0, 0.3, E)
    J = int(r.integers(E // 2, E))
    base[J] = np.log(E) + r.uniform(1.5, 4.0)
    base = base.astype(np.float32).astype(np.float64)
    p = np.exp(base - base.max())
    p /= p.sum()
    c = 0.01
    want = c - 0.001 * (1 + r.random(E))
    rest = [x for x in r.permutation(E) if x != J]
    a, b, top = rest[0], rest[1], rest[2:1 + K]
    gap = 2.0 ** -24 * r.uniform(1.0, 2.0)
    want[a], want[b] = c + gap / 2, c - gap / 2
    want[J] = c + 2.0 ** -24 * r.uniform(-1, 2)
    want[top] = c + 0.1 + 0.01 * r.random(len(top))
    bias = (want - p).astype(np.float32)
    logits = np.repeat(base.astype(np.float32)[None], rows, 0)
    # the dominant logit a few steps of fp32 to either side: its value moves past the border
    step = np.spacing(logits[0, J])
    logits[:, J] += (step * r.integers(-3, 4, rows)).astype(np.float32)
    logits[:, a] += (1e-5 * r.normal(size=rows)).astype(np.float32)
    return torch.from_numpy(logits).to(DEV), torch.from_numpy(bias).to(DEV)


@pytest.mark.parametrize("E,K,G,tg", [(32, 1, 1, 1), (32, 3, 4, 4), (64, 1, 8, 8), (160, 6, 1, 1),
                                      (160, 1, 1, 1), (256, 8, 8, 8), (288, 2, 1, 1), (1024, 4, 1, 1)])
def test_bias_hides_a_dominant_expert(E, K, G, tg):
    """An expert that fp32 ranks behind the first K + 1 is chosen where 64 bits choose it."""
    for seed in range(24):
        logits, bias = dominant_rows(E, K, G, 1000 * E + seed)
        check(logits, K, G, tg, False, bias=bias)


def test_order_among_experts_without_probability():
    """Beside a +inf logit every finite one has p = 0: without a bias the logits still order them,
    with a bias of zeros their values are equal and the lower index comes first."""
    l = torch.tensor([[float("inf"), 1.0, 5.0, 2.0]], device=DEV)
    inds, scores = binding.route_softmax_grouped(l, 2, 1, 1, False, 1.0)
    assert inds.tolist() == [[0, 2]] and scores.tolist() == [[1.0, 0.0]]
    inds, scores = binding.route_softmax_grouped(l, 2, 1, 1, False, 1.0, bias=torch.zeros(4, device=DEV))
    assert inds.tolist() == [[0, 1]] and scores.tolist() == [[1.0, 0.0]]
