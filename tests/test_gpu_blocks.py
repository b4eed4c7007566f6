"""GPU parity of the block-scaled e4m3 path (moe_quantize_blocks, moe_matmul_blocks, the
MOE_BITS_E4M3 experts of moe_grouped_swiglu) against plain evaluations in 64 bits.

Quantisation is one rounding of an exact quotient: codes and scales are compared bit for bit.

Products: e4m3 products are exact in fp32 (4 x 4 significant bits).  A block's 128 products are
added in fp32 in some order, each addition off by at most one unit (truncation counts as one),
and the blocks by a multiply-add each after a product of the two scales, so with S the sum of
the magnitudes of all scaled products  |y - ref| <= (128 * 2^-23 + (blocks + 2) * 2^-24) S,
plus 2^-8 |y| for a bf16 result.

Experts: h is quantised again, so an h that its own error bound lets cross a rounding border may
land one e4m3 step away; every such h adds its step times |w_down| to the bound.
"""
import numpy as np
import pytest
import torch

from deepseek_moe_layer_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
F8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ---------------------------------------------------------------------------------------
# 64-bit references
# ---------------------------------------------------------------------------------------

def step64(v):
    """Spacing of e4m3 at |v|: 2^(floor(log2 |v|) - 3), 2^-9 below 2^-6."""
    return torch.exp2((torch.frexp(v)[1] - 4).clamp_min(-9).double())


def scale64(amax):
    s = torch.exp2(torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448)) + 1)
    for _ in range(3):  # the smallest power of two with amax / s <= 448
        s = torch.where(amax <= 448 * s / 2, s / 2, s)
    return torch.where(amax > 0, s.clamp_min(2.0 ** -126), torch.ones_like(s))


def quantize64(x, block_rows=1):
    """x [rows, n] -> (values in units of the scale, scale spread to x's shape, scales)."""
    rows, n = x.shape
    R, B = -(-rows // block_rows), -(-n // 128)
    x = x.double()
    fin = torch.where(torch.isfinite(x), x, 0.0).abs()
    fin = torch.nn.functional.pad(fin, (0, B * 128 - n, 0, R * block_rows - rows))
    s = scale64(fin.view(R, block_rows, B, 128).amax(dim=(1, 3)))
    wide = s.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :n]
    v = torch.where(torch.isfinite(x), x / wide, float("nan"))
    return torch.round(v / step64(v)) * step64(v), wide, s


def spread(scale, rows, cols, block_rows):
    return scale.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def product64(av, wv, blocks):
    """(a w^T, error bound of the fp32 result) of float64 values (scales included)."""
    S = av.abs() @ wv.abs().t()
    return av @ wv.t(), (128 * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24) * S


def check_within(got, ref, tol):
    got, ref = got.double(), ref.double()
    bad = ~((got - ref).abs() <= tol)
    bad &= ~(torch.isnan(got) & torch.isnan(ref))
    assert not bool(bad.any()), (int(bad.sum()), float((got - ref).abs()[bad].max()),
                                 bad.nonzero()[:4].tolist())


# ---------------------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------------------

def check_quantize(x, block_rows):
    codes, scales = binding.quantize_blocks(x, block_rows=block_rows)
    v, _, s = quantize64(x, block_rows)
    assert torch.equal(scales.double(), s)
    c = codes.double()
    assert torch.equal(torch.isnan(c), torch.isnan(v))
    assert torch.equal(torch.nan_to_num(c), torch.nan_to_num(v))
    assert torch.equal(torch.signbit(codes.float())[~torch.isnan(v)], torch.signbit(v)[~torch.isnan(v)])


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,pad", [(1, 16, 0), (1, 7168, 0), (3, 144, 8), (127, 128, 16),
                                        (129, 272, 0), (300, 1040, 24), (257, 2048, 0)])
def test_quantize_rows_and_blocks(rows, n, pad, dtype, block_rows):
    g = gen(rows * 7 + n)
    x = torch.randn(rows, n + pad, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g, device=DEV).float())
    check_quantize(x.to(dtype)[:, :n], block_rows)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_special_values(dtype, block_rows):
    tiny = torch.finfo(dtype).tiny
    rows = [torch.zeros(256), torch.full((256,), -0.0), torch.full((256,), 448.0),
            torch.full((256,), torch.finfo(dtype).max), torch.full((256,), tiny),
            torch.full((256,), tiny / 8), torch.full((256,), float("nan")),
            torch.full((256,), float("-inf"))]
    mixed = torch.linspace(-3, 3, 256)
    for at, v in ((5, float("inf")), (130, float("nan")), (140, float("-inf"))):
        mixed = mixed.clone()
        mixed[at] = v
        rows.append(mixed)
    # borders of the scale: 448 s and its neighbour, and every tie between two codes
    rows.append(torch.tensor([448.0, 450.0] + [0.0] * 126 + [896.0, 900.0] + [0.0] * 126))
    ties = torch.arange(128) * 0.5 + 16.25
    rows.append(torch.cat([ties, -ties]))
    x = torch.stack(rows).to(DEV).to(dtype)
    for i in range(x.shape[0]):
        check_quantize(x[i:i + 1], block_rows)
    check_quantize(x, block_rows)


def test_quantize_leaves_outputs_of_empty_input():
    codes, scales = binding.quantize_blocks(torch.empty(0, 256, device=DEV))
    assert codes.shape == (0, 256) and scales.shape == (0, 2)


# ---------------------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------------------

def codes_of(shape, g, mag=60.0):
    return (torch.randn(shape, generator=g, device=DEV) * mag).clamp(-448, 448).to(F8)


def operands(M, N, K, seed, pad=0):
    g = gen(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    a = codes_of((M, K + pad), g)[:, :K]
    w = codes_of((N, K), g)
    sa = torch.rand(M, kb, generator=g, device=DEV) * 0.02 + 1e-3
    sw = torch.rand(nb, kb, generator=g, device=DEV) * 0.02 + 1e-3
    return a, sa, w, sw


def check_matmul(a, sa, w, sw, dtype):
    (M, K), N = a.shape, w.shape[0]
    y = binding.matmul_blocks(a, sa, w, sw, out_dtype=dtype)
    torch.cuda.synchronize()
    binding.device_status()
    ref, tol = product64(a.double() * spread(sa, M, K, 1), w.double() * spread(sw, N, K, 128),
                         sa.shape[1])
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    check_within(y, ref, tol)
    return y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,pad", [
    (1, 1, 16, 0), (1, 256, 128, 0), (2, 577, 1488, 16), (31, 64, 144, 0), (33, 130, 384, 0),
    (96, 2112, 7168, 0), (97, 256, 640, 0), (128, 512, 256, 128), (129, 257, 272, 0),
    (300, 1025, 2048, 0), (1000, 4096, 512, 0), (5000, 136, 128, 0)])
def test_matmul_shapes(M, N, K, pad, dtype):
    check_matmul(*operands(M, N, K, M + N + K, pad), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    # many tiles of one CTA each: of 32 rows, of 128 rows, with and without a ragged last column
    (5, 40000, 256), (30, 39001, 144), (2500, 2304, 256), (2470, 2401, 272),
    # two, four and eight CTAs on a tile, k-blocks that do not divide evenly
    (32, 8192, 1424), (128, 8192, 640), (20, 4097, 2064), (260, 1600, 1680), (17, 700, 7168),
    (3, 256, 4112), (128, 256, 5264), (100, 131, 4000)])
def test_matmul_tile_forms(M, N, K, dtype):
    check_matmul(*operands(M, N, K, M + N + K), dtype)


def test_matmul_every_row_and_column_lands_in_its_place():
    """One-hot rows pick single weight columns: exact, and wrong as soon as a row, a column, a
    block or its scale is taken from elsewhere."""
    M, N, K = 300, 520, 400
    g = gen(3)
    k = torch.randint(0, K, (M,), generator=g, device=DEV)
    a = torch.zeros(M, K, device=DEV).scatter_(1, k[:, None], 1.0).to(F8)
    w = codes_of((N, K), g)
    sa = torch.exp2(torch.randint(-3, 4, (M, 4), generator=g, device=DEV).float())
    sw = torch.exp2(torch.randint(-3, 4, (5, 4), generator=g, device=DEV).float())
    y = binding.matmul_blocks(a, sa, w, sw, out_dtype=torch.float32)
    ref = (w.double() * spread(sw, N, K, 128)).t()[k] * sa.double().gather(1, (k // 128)[:, None])
    assert torch.equal(y.double(), ref)


def test_matmul_takes_strided_rows_and_a_given_output():
    a, sa, w, sw = operands(70, 96, 256, 8, pad=64)
    out = torch.full((72, 96), 5.0, dtype=torch.float32, device=DEV)
    y = binding.matmul_blocks(a, sa, w, sw, out=out[1:71])
    assert y.data_ptr() == out[1:71].data_ptr()
    assert torch.equal(y, binding.matmul_blocks(a.contiguous(), sa, w, sw, out_dtype=torch.float32))
    assert bool((out[0] == 5).all()) and bool((out[71] == 5).all())
    # an output that starts off a 32-byte border
    buf = torch.full((70 * 96 + 1,), 5.0, dtype=torch.float32, device=DEV)
    z = binding.matmul_blocks(a, sa, w, sw, out=buf[1:].view(70, 96))
    assert torch.equal(z, y) and float(buf[0]) == 5.0


def test_cpu_tensors_are_refused():
    a, sa, w, sw = operands(4, 16, 128, 1)
    with pytest.raises(ValueError):
        binding.matmul_blocks(a.cpu(), sa.cpu(), w.cpu(), sw.cpu())
    with pytest.raises(ValueError):
        binding.matmul_blocks(a, sa, w.cpu(), sw)
    with pytest.raises(ValueError):
        binding.quantize_blocks(torch.randn(4, 128))
    with pytest.raises(ValueError):
        binding.route_softmax_grouped(torch.randn(4, 16), 2, 4, 2, True, 1.0)


def test_matmul_nan_stays_in_its_row_and_column():
    a, sa, w, sw = operands(200, 300, 512, 11)
    a, w = a.clone(), w.clone()
    a.view(torch.uint8)[7, 130] = 0x7F
    w.view(torch.uint8)[290, 3] = 0xFF
    y = binding.matmul_blocks(a, sa, w, sw)
    bad = torch.isnan(y)
    want = torch.zeros_like(bad)
    want[7, :] = True
    want[:, 290] = True
    assert torch.equal(bad, want)


def test_matmul_same_bits_on_other_streams_in_graphs_and_beside_each_other():
    sets = [operands(64, 2112, 1024, 5), operands(700, 384, 640, 6), operands(1, 512, 7168, 7)]
    want = [binding.matmul_blocks(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(binding.matmul_blocks(*s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    graphs, outs = [], []
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(binding.matmul_blocks(*s))
        graphs.append(gr)
    for o in outs:
        o.zero_()
    for gr, st in zip(graphs, streams):
        with torch.cuda.stream(st):
            gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------------------

def weight(E, N, K, g):
    s = (torch.rand(E, N // 128, K // 128, generator=g, device=DEV) + 0.5) / (60 * K ** 0.5)
    return codes_of((E, N, K), g), s


def make_experts(E, d, I, g):
    out = {"bits": binding.MOE_BITS_E4M3}
    for k, (n, m) in (("gate", (I, d)), ("up", (I, d)), ("down", (d, I))):
        out[k], out[k + "_s"] = weight(E, n, m, g)
    return out


def expert_ref(x, ex, e):
    """float64 SwiGLU of the rows x through expert e and its error bound."""
    rows, d = x.shape
    I = ex["gate"].shape[1]
    w = {k: ex[k][e].double() * spread(ex[k + "_s"][e], *ex[k].shape[1:], 128)
         for k in ("gate", "up", "down")}
    v, s, _ = quantize64(x)
    a, ta = product64(v * s, w["gate"], d // 128)
    b, tb = product64(v * s, w["up"], d // 128)
    si = a * torch.sigmoid(a)
    h = si * b
    # |silu'| <= 1.1; expf's and the quotient's own errors stay below 2^-20 of silu
    th = 1.1 * ta * (b.abs() + tb) + si.abs() * tb + 2.0 ** -20 * h.abs()
    q, hs, _ = quantize64(h)
    # what one step away costs: an h within th of a border between two codes, or a block whose
    # scale its largest h may change (then any of its codes may be rounded at twice the step)
    u = h / hs
    step = step64(u)
    border = ((torch.floor(u / step) + 0.5) * step - u).abs()
    near = border <= th / hs + 1e-300
    near |= step64(u.abs() + th / hs) != step
    amax = h.abs().view(rows, I // 128, 128).amax(2)
    tmax = (h.abs() + th).view(rows, I // 128, 128).amax(2)
    tmin = (h.abs() - th).clamp_min(0).view(rows, I // 128, 128).amax(2)
    moved = (scale64(tmax) != scale64(amax)) | (scale64(tmin) != scale64(amax))
    near |= moved.repeat_interleave(128, 1)
    off = torch.where(near, 2 * step * hs, 0.0)
    y, ty = product64(q * hs, w["down"], I // 128)
    return y, ty + off @ w["down"].abs().t()


def dispatch(T, E, K, g, skew=0.0, drop=False):
    like = torch.randn(T, E, generator=g, device=DEV) + skew * torch.randn(E, generator=g, device=DEV)
    inds = like.topk(K, dim=1).indices.to(torch.int32)
    if drop:  # pairs without an expert are not dispatched
        inds[torch.rand(T, K, generator=g, device=DEV) < 0.3] = -1
    return inds


def check_experts(T, d, I, E, K, shared, seed, skew=0.0, drop=False):
    g = gen(seed)
    x = (torch.randn(T, d, generator=g, device=DEV) *
         (1 + 15 * (torch.rand(d, generator=g, device=DEV) < 0.01))).to(torch.bfloat16)
    ex = make_experts(E, d, I, g)
    sh = make_experts(1, d, I, g) if shared else None
    inds = dispatch(T, E, K, g, skew, drop)
    counts, offsets, perm, inv = binding.permute(inds, E)
    y = binding.grouped_swiglu(x, offsets, perm, K, ex, sh)
    torch.cuda.synchronize()
    binding.device_status()
    off = offsets.tolist()
    tok = perm.long() // K
    for e in range(E):
        if off[e + 1] > off[e]:
            at = slice(off[e], off[e + 1])
            ref, tol = expert_ref(x[tok[at]], ex, e)
            check_within(y[at], ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs())
    if shared:
        ref, tol = expert_ref(x, sh, 0)
        check_within(y[T * K:], ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs())


@pytest.mark.parametrize("T,d,I,E,K,shared", [
    (1, 128, 128, 4, 1, False), (1, 256, 128, 8, 8, True), (5, 640, 384, 8, 2, True),
    (64, 256, 256, 16, 4, True), (33, 1024, 128, 5, 3, False), (300, 384, 256, 6, 2, True),
    (700, 512, 384, 4, 4, True), (1500, 256, 128, 3, 2, False)])
def test_experts(T, d, I, E, K, shared):
    check_experts(T, d, I, E, K, shared, T + d)


@pytest.mark.parametrize("T,d,I,E,K,shared", [
    # many tiles of 32 rows, some experts with more rows than one; then of 128 rows
    (64, 512, 1024, 40, 4, True), (100, 256, 2048, 48, 7, False), (1200, 640, 1024, 8, 4, True),
    # few tiles, several CTAs on each: of 32 rows and of 128
    (2, 2048, 256, 16, 3, True), (40, 1152, 128, 6, 2, True), (200, 1408, 128, 2, 2, False)])
def test_experts_tile_forms(T, d, I, E, K, shared):
    check_experts(T, d, I, E, K, shared, T + d + I)


def test_experts_skewed_and_undispatched():
    check_experts(400, 256, 256, 32, 4, True, 1, skew=3.0)
    check_experts(200, 256, 128, 8, 3, True, 2, drop=True)
    check_experts(3000, 256, 128, 8, 3, True, 3, drop=True)  # by the inverse dispatch


@pytest.mark.parametrize("T,shared", [(3, True), (3, False), (900, True), (4200, False)])
def test_experts_with_nothing_dispatched(T, shared):
    """Every pair without an expert: only the shared rows are computed."""
    g = gen(T)
    d, I, E, K = 256, 128, 5, 2
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    ex, sh = make_experts(E, d, I, g), make_experts(1, d, I, g) if shared else None
    inds = torch.full((T, K), -1, dtype=torch.int32, device=DEV)
    _, offsets, perm, _ = binding.permute(inds, E)
    y = binding.grouped_swiglu(x, offsets, perm, K, ex, sh)
    torch.cuda.synchronize()
    binding.device_status()
    if shared:
        ref, tol = expert_ref(x, sh, 0)
        check_within(y[T * K:], ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs())


def test_experts_same_bits_on_another_stream_and_twice():
    g = gen(31)
    d, I, E, K = 512, 256, 8, 3
    ex, sh = make_experts(E, d, I, g), make_experts(1, d, I, g)
    cases = []
    for T in (1, 50, 1700):
        x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
        _, offsets, perm, _ = binding.permute(dispatch(T, E, K, g), E)
        cases.append((x, offsets, perm, binding.grouped_swiglu(x, offsets, perm, K, ex, sh)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):  # all at once, each on a stream and a workspace of its own
        got = []
        for (x, o, p, _), st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(binding.grouped_swiglu(x, o, p, K, ex, sh, stream=st))
        torch.cuda.synchronize()
        for c, y in zip(cases, got):
            assert torch.equal(c[3], y)


def test_weights_quantised_by_the_library_serve_as_experts():
    """bf16 weights through moe_quantize_blocks (128 x 128) into the experts' format."""
    g = gen(41)
    d, I, E, K, T = 256, 256, 3, 2, 20
    ex = {"bits": binding.MOE_BITS_E4M3}
    for k, (n, m) in (("gate", (I, d)), ("up", (I, d)), ("down", (d, I))):
        w = (torch.randn(E, n, m, generator=g, device=DEV) / m ** 0.5).to(torch.bfloat16)
        q = [binding.quantize_blocks(w[e], block_rows=128) for e in range(E)]
        ex[k] = torch.stack([c.view(torch.uint8) for c, _ in q]).view(F8)
        ex[k + "_s"] = torch.stack([s for _, s in q])
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    _, offsets, perm, _ = binding.permute(dispatch(T, E, K, g), E)
    y = binding.grouped_swiglu(x, offsets, perm, K, ex)
    off, tok = offsets.tolist(), perm.long() // K
    for e in range(E):
        at = slice(off[e], off[e + 1])
        ref, tol = expert_ref(x[tok[at]], ex, e)
        check_within(y[at], ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs())


def test_experts_rows_behind_the_last_slot_are_left_alone():
    g = gen(9)
    T, d, I, E, K = 40, 256, 128, 4, 2
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    ex = make_experts(E, d, I, g)
    inds = torch.full((T, K), -1, dtype=torch.int32, device=DEV)
    inds[:7, 0] = 2
    _, offsets, perm, _ = binding.permute(inds, E)
    out = torch.full((T * K, d), 7.0, dtype=torch.bfloat16, device=DEV)
    need = binding.grouped_swiglu_workspace_bytes(T, d, I, E, K, False)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    import ctypes
    ew = binding.expert_weights(ex)
    binding._check(binding.lib().moe_grouped_swiglu(
        binding._ptr(x), T, d, I, E, K, binding._ptr(offsets), binding._ptr(perm),
        ctypes.byref(ew), None, binding._ptr(out), binding._ptr(ws), need, binding._stream()))
    torch.cuda.synchronize()
    assert bool((out[7:] == 7.0).all()) and not bool((out[:7] == 7.0).all())


def test_failed_launches_leave_outputs_and_recover():
    """The host-side fault hook at each launch of the new calls: an error, the outputs of the
    launches not made as they were, and the same call right afterwards."""
    g = gen(51)
    x = torch.randn(40, 256, generator=g, device=DEV)
    codes = torch.full((40, 256), 1.0, device=DEV).to(F8)
    scales = torch.full((40, 2), 3.0, device=DEV)
    ops = operands(40, 96, 256, 2)
    out = torch.full((40, 96), 5.0, device=DEV)
    logits = torch.randn(40, 16, generator=g, device=DEV)
    inds = torch.full((40, 2), 9, dtype=torch.int32, device=DEV)
    ex = make_experts(4, 256, 128, g)
    _, offsets, perm, _ = binding.permute(dispatch(40, 4, 2, g), 4)
    xb = x.to(torch.bfloat16)
    before = binding.get_fault()
    try:
        for at, call in ((0, lambda: binding.quantize_blocks(x, codes=codes, scales=scales)),
                         (0, lambda: binding.matmul_blocks(*ops, out=out)),
                         (0, lambda: binding.route_softmax_grouped(logits, 2, 4, 2, True, 1.0, inds=inds)),
                         (0, lambda: binding.grouped_swiglu(xb, offsets, perm, 2, ex)),
                         (1, lambda: binding.grouped_swiglu(xb, offsets, perm, 2, ex)),
                         (2, lambda: binding.grouped_swiglu(xb, offsets, perm, 2, ex))):
            binding.set_fault(binding.MOE_FAULT_LAUNCH, at)
            with pytest.raises(binding.MoeError) as e:
                call()
            assert e.value.code == binding.MOE_ERR_CUDA and "injected" in str(e.value)
        torch.cuda.synchronize()
        assert bool((codes.float() == 1).all()) and bool((scales == 3).all())
        assert bool((out == 5).all()) and bool((inds == 9).all())
    finally:
        binding.set_fault(*before)
    check_quantize(x, 1)
    check_matmul(*ops, torch.float32)
    check_experts(40, 256, 128, 4, 2, False, 52)


def test_layer_of_the_parts():
    """moe_forward(_ex) with e4m3 experts is its parts: the gate on the layer's own logits, the
    dispatch, the experts and the combine give the same bits, for both gates."""
    g = gen(21)
    d, I, E, K = 512, 256, 16, 4
    ex, sh = make_experts(E, d, I, g), make_experts(1, d, I, g)
    wr = (torch.randn(E, d, generator=g, device=DEV) / d ** 0.5).to(torch.bfloat16)
    bias = 0.05 * torch.randn(E, generator=g, device=DEV)
    wg = (torch.randn(d, generator=g, device=DEV) / d ** 0.5).to(torch.bfloat16)
    for kind, b, gate in ((binding.MOE_ROUTE_DEEPSEEK, bias, None),
                          (binding.MOE_ROUTE_SOFTMAX_GROUPED, bias, wg),
                          (binding.MOE_ROUTE_SOFTMAX_GROUPED, None, None)):
        layer = binding.MoELayer(wr, b, ex, sh, K, 4, 2, True, 2.5, route_kind=kind,
                                 w_shared_gate=gate)
        for T in (1, 7, 130, 2100):
            x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
            y, inds, scores, logits = layer(x, want_intermediates=True)
            if kind == binding.MOE_ROUTE_DEEPSEEK:
                i2, s2 = binding.route_deepseek(logits, b, K, 4, 2, True, 2.5)
            else:
                i2, s2 = binding.route_softmax_grouped(logits, K, 4, 2, True, 2.5, bias=b)
            assert torch.equal(inds, i2) and torch.equal(scores, s2)
            _, offsets, perm, inv = binding.permute(inds, E)
            eo = binding.grouped_swiglu(x, offsets, perm, K, ex, sh)
            if gate is None:
                z = binding.combine(eo, scores, inv, eo[T * K:])
            else:
                z = binding.combine_gated(eo, scores, inv, eo[T * K:], binding.shared_gate(x, gate))
            assert torch.equal(y, z)
            assert bool(torch.isfinite(y.float()).all())
            assert torch.equal(y, layer(x))  # and with the copies of the intermediates left out
    torch.cuda.synchronize()
    binding.device_status()


def test_layer_captured_and_replayed():
    g = gen(22)
    d, I, E, K, T = 256, 128, 8, 2, 9
    ex, sh = make_experts(E, d, I, g), make_experts(1, d, I, g)
    wr = (torch.randn(E, d, generator=g, device=DEV) / d ** 0.5).to(torch.bfloat16)
    layer = binding.MoELayer(wr, None, ex, sh, K, 2, 1, False, 1.0,
                             route_kind=binding.MOE_ROUTE_SOFTMAX_GROUPED)
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    y = torch.empty_like(x)
    layer(x, y=y)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        layer(x, y=y)
    for _ in range(3):
        x.copy_(torch.randn(T, d, generator=g, device=DEV))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer(x))


def test_noalloc_with_scaled_experts():
    import ctypes
    g = gen(23)
    d, I, E, K, T = 256, 128, 8, 2, 11
    ex, sh = make_experts(E, d, I, g), make_experts(1, d, I, g)
    wr = (torch.randn(E, d, generator=g, device=DEV) / d ** 0.5).to(torch.bfloat16)
    bias = torch.zeros(E, device=DEV)
    layer = binding.MoELayer(wr, bias, ex, sh, K, 1, 1, True, 1.0)
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    want, y = layer(x), torch.empty_like(x)
    P = binding._ptr
    binding._check(binding.lib().moe_forward_noalloc(
        P(x), T, d, I, E, P(wr), P(bias), None, ctypes.byref(layer.params),
        ctypes.byref(layer.ew), ctypes.byref(layer.sw), P(y), None, None, None,
        binding._stream()))
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("M,N,K", [(300, 600, 400), (5, 300, 144), (100, 300, 2064), (400, 20000, 256)])
@pytest.mark.parametrize("sx,sw", [(-126, -20), (-126, -25), (-20, -126), (-100, -45), (-140, 20),
                                   (119, 10), (10, 119), (64, 64), (-149, -10)])
def test_scales_whose_product_is_no_normal_number(sx, sw, M, N, K):
    """Any fp32 scales: a sum of e4m3 products (2^-18 to 2^25) brings back into range what the
    product of its two scales alone leaves.  Beside the bound of check_matmul, each of the blocks'
    steps may lose half the smallest subnormal, 2^-150."""
    g = gen(M + sx)
    kb, nb = -(-K // 128), -(-N // 128)
    a, w = codes_of((M, K), g), codes_of((N, K), g)
    if sx + sw > 0:  # subnormal codes: sums below 2^-5, some of them 0
        a = (torch.randint(-7, 8, (M, K), generator=g, device=DEV) * 2.0 ** -9).to(F8)
        w = (torch.randint(-7, 8, (N, K), generator=g, device=DEV) * 2.0 ** -9).to(F8)
    a = a.float().mul_(torch.rand(M, 1, generator=g, device=DEV) < 0.9).to(F8)  # rows of zeros
    # the first k-block and every third row as scales usually are: lost and whole factors side by side
    sa = torch.full((M, kb), 2.0 ** sx, dtype=torch.float64, device=DEV)
    sb = torch.full((nb, kb), 2.0 ** sw, dtype=torch.float64, device=DEV)
    if sx + sw < 0:
        sa[::3], sb[:, 0] = 2.0 ** -60, 2.0 ** -70
        sa[M // 2, kb - 1] = 0.0
    sa *= 1 if sx < -126 else 1 + torch.rand(M, kb, generator=g, device=DEV) / 2
    sb *= 1 + torch.rand(nb, kb, generator=g, device=DEV) / 2
    sa, sb = sa.float(), sb.float()
    y = binding.matmul_blocks(a, sa, w, sb, out_dtype=torch.float32)
    torch.cuda.synchronize()
    binding.device_status()
    ref, tol = product64(a.double() * spread(sa, M, K, 1), w.double() * spread(sb, N, K, 128), kb)
    assert float(ref.abs().max()) < 2.0 ** 127
    check_within(y, ref, tol + (kb + 2) * 2.0 ** -149)


@pytest.mark.parametrize("T,E", [(3, 8), (40, 6), (600, 3)])
def test_experts_with_scales_whose_product_is_no_normal_number(T, E):
    """The down product's two scales together near 2^-147, its rows near 2^-129 (where bf16's own
    rounding is 2^-134)."""
    g = gen(T)
    d, I, K = 256, 128, 2
    ex = make_experts(E, d, I, g)
    for k, e in (("gate_s", -46), ("up_s", -52), ("down_s", -30)):
        ex[k] = (ex[k].double() * 2.0 ** e).float()
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    _, offsets, perm, _ = binding.permute(dispatch(T, E, K, g), E)
    y = binding.grouped_swiglu(x, offsets, perm, K, ex)
    torch.cuda.synchronize()
    off, tok = offsets.tolist(), perm.long() // K
    for e in range(E):
        if off[e + 1] > off[e]:
            at = slice(off[e], off[e + 1])
            ref, tol = expert_ref(x[tok[at]], ex, e)
            check_within(y[at], ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs() + 2.0 ** -134)


def test_calls_on_a_given_stream_allocate_there(monkeypatch):
    """With stream= every output and workspace is of that stream's memory (the current stream's may
    still be in use by work queued there), and the results equal those of the current stream."""
    g = gen(61)
    T, d, I, E, K = 40, 256, 128, 8, 2
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    ex, sh = make_experts(E, d, I, g), make_experts(1, d, I, g)
    wr = (torch.randn(E, d, generator=g, device=DEV) / d ** 0.5).to(torch.bfloat16)
    wg, bias = wr[0].contiguous(), torch.zeros(E, device=DEV)
    logits = binding.router_logits(x, wr)
    inds, scores = binding.route_softmax_grouped(logits, K, 2, 2, True, 1.0)
    _, offsets, perm, inv = binding.permute(inds, E)
    eo = binding.grouped_swiglu(x, offsets, perm, K, ex, sh)
    gate = binding.shared_gate(x, wg)
    ops = operands(40, 96, 256, 2)
    layer = binding.MoELayer(wr, None, ex, sh, K, 2, 2, True, 1.0, route_kind=binding.MOE_ROUTE_SOFTMAX_GROUPED)
    calls = {
        "quantize_blocks": lambda st: binding.quantize_blocks(x, stream=st),
        "matmul_blocks": lambda st: binding.matmul_blocks(*ops, stream=st),
        "route_softmax_grouped": lambda st: binding.route_softmax_grouped(logits, K, 2, 2, True, 1.0, stream=st),
        "route_softmax": lambda st: binding.route_softmax(logits, K, stream=st),
        "route_deepseek": lambda st: binding.route_deepseek(logits, bias, K, 2, 1, True, 1.0, stream=st),
        "router_logits": lambda st: binding.router_logits(x, wr, stream=st),
        "permute": lambda st: binding.permute(inds, E, stream=st),
        "grouped_swiglu": lambda st: binding.grouped_swiglu(x, offsets, perm, K, ex, sh, stream=st),
        "shared_gate": lambda st: binding.shared_gate(x, wg, stream=st),
        "combine": lambda st: binding.combine(eo, scores, inv, eo[T * K:], stream=st),
        "combine_gated": lambda st: binding.combine_gated(eo, scores, inv, eo[T * K:], gate, stream=st),
        "indexer_topk": lambda st: binding.indexer_topk(logits, 3, want_mask=True, stream=st),
        "layer": lambda st: layer(x, want_intermediates=True, stream=st),
    }
    want = {k: c(None) for k, c in calls.items()}
    layer.ws = None
    torch.cuda.synchronize()
    st, seen, empty = torch.cuda.Stream(), [], torch.empty

    def watched(*a, **kw):
        seen.append(torch.cuda.current_stream())
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", watched)
    got = {}
    for k, c in calls.items():
        seen.clear()
        got[k] = c(st)
        assert seen and all(s == st for s in seen), k
    monkeypatch.undo()
    torch.cuda.synchronize()
    for k in calls:
        a, b = (v if isinstance(v, tuple) else (v,) for v in (want[k], got[k]))
        assert len(a) == len(b)
        for u, v in zip(a, b):
            assert torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8)), k


def test_layer_keeps_its_workspace_for_the_streams_that_use_it():
    """A workspace used on a second stream is not handed out again when a later call replaces it,
    before that stream is done with it."""
    g = gen(62)
    d, I, E, K = 256, 128, 8, 2
    ex = make_experts(E, d, I, g)
    wr = (torch.randn(E, d, generator=g, device=DEV) / d ** 0.5).to(torch.bfloat16)
    layer = binding.MoELayer(wr, None, ex, None, K, 2, 2, True, 1.0,
                             route_kind=binding.MOE_ROUTE_SOFTMAX_GROUPED)
    x = torch.randn(64, d, generator=g, device=DEV).to(torch.bfloat16)
    big = torch.randn(4096, d, generator=g, device=DEV).to(torch.bfloat16)
    want = layer(x)
    torch.cuda.synchronize()
    old, size = layer.ws.data_ptr(), layer.ws.numel()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(200_000_000)  # some 0.1 s
        y = layer(x)
    layer(big)  # replaces the workspace while the call on st waits
    assert layer.ws.data_ptr() != old
    taken = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(4)]
    assert all(t.data_ptr() != old for t in taken)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("T,d,I,E,K,shared", [
    (64, 512, 1024, 40, 4, True), (1200, 640, 1024, 8, 4, True),   # tiles of 32 rows, of 128
    (2, 2048, 256, 16, 3, True), (200, 1408, 128, 2, 2, False)])   # several CTAs on a tile
def test_experts_write_an_output_off_a_32_byte_border(T, d, I, E, K, shared):
    """The call asks for 16 bytes: the same bits as on a whole border, and nothing around them."""
    import ctypes
    g = gen(T + d)
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    ex, sh = make_experts(E, d, I, g), make_experts(1, d, I, g) if shared else None
    _, offsets, perm, _ = binding.permute(dispatch(T, E, K, g), E)
    want = binding.grouped_swiglu(x, offsets, perm, K, ex, sh)
    buf = torch.full((want.numel() + 24,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[8:8 + want.numel()].view(want.shape)
    assert out.data_ptr() % 32 == 16
    need = binding.grouped_swiglu_workspace_bytes(T, d, I, E, K, shared)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    ew, sw = binding.expert_weights(ex), binding.expert_weights(sh)
    binding._check(binding.lib().moe_grouped_swiglu(
        binding._ptr(x), T, d, I, E, K, binding._ptr(offsets), binding._ptr(perm), ctypes.byref(ew),
        binding._ref(sw), binding._ptr(out), binding._ptr(ws), need, binding._stream()))
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert bool((buf[:8] == 7).all()) and bool((buf[8 + want.numel():] == 7).all())


@pytest.mark.parametrize("T,E,every", [(1, 64, 1), (64, 64, 4), (900, 64, 16), (128, 256, 24)])
def test_layer_at_a_checkpoints_size(T, E, every):
    """d = 7168, I = 2048, 8 of E experts and a shared one: the layer is its parts bit for bit, and
    every `every`-th expert that is hit, and the shared one, match 64 bits."""
    g = gen(T + E)
    d, I, K = 7168, 2048, 8
    ex, sh = {"bits": binding.MOE_BITS_E4M3}, make_experts(1, d, I, g)
    for k, (n, m) in (("gate", (I, d)), ("up", (I, d)), ("down", (d, I))):
        ex[k] = torch.empty(E, n, m, dtype=F8, device=DEV)
        for e in range(E):
            ex[k][e] = codes_of((n, m), g)
        ex[k + "_s"] = (torch.rand(E, n // 128, m // 128, generator=g, device=DEV) + 0.5) / (60 * m ** 0.5)
    wr = (torch.randn(E, d, generator=g, device=DEV) / d ** 0.5).to(torch.bfloat16)
    bias = 0.01 * torch.randn(E, generator=g, device=DEV)
    layer = binding.MoELayer(wr, bias, ex, sh, K, 8, 4, True, 2.5)
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    y, inds, scores, _ = layer(x, want_intermediates=True)
    _, offsets, perm, inv = binding.permute(inds, E)
    eo = binding.grouped_swiglu(x, offsets, perm, K, ex, sh)
    assert torch.equal(y, binding.combine(eo, scores, inv, eo[T * K:]))
    binding.device_status()
    off, tok = offsets.tolist(), perm.long() // K
    hit = [e for e in range(E) if off[e + 1] > off[e]]
    for e in hit[::every]:
        at = slice(off[e], off[e + 1])
        ref, tol = expert_ref(x[tok[at]], ex, e)
        check_within(eo[at], ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs())
    ref, tol = expert_ref(x, sh, 0)
    check_within(eo[T * K:], ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs())


@pytest.mark.parametrize("T,d,I,E,K,shared", [
    (64, 512, 1024, 40, 4, True), (1200, 640, 1024, 8, 4, True),   # tiles of 32 rows, of 128
    (2, 2048, 256, 16, 3, True), (200, 1408, 128, 2, 2, False)])   # several CTAs on a tile
def test_up_weights_whose_scale_and_the_rows_make_no_normal_number(T, d, I, E, K, shared):
    """u near 2^-130 from scales whose product is near 2^-147 (three bits left in fp32), in some
    blocks of some experts only: h and its codes, and the rows after the down product, as 64 bits
    have them."""
    g = gen(T + d + 1)
    x = (torch.randn(T, d, generator=g, device=DEV) * 2.0 ** -60).to(torch.bfloat16)
    sets = [make_experts(E, d, I, g)] + ([make_experts(1, d, I, g)] if shared else [])
    for ex in sets:
        for k, e in (("gate_s", 66), ("up_s", -70), ("down_s", 20)):
            ex[k] = (ex[k].double() * 2.0 ** e).float()
        ex["up_s"][:, :, ::3] *= 2.0 ** 8
        ex["up_s"][::3] *= 2.0 ** 20
    ex, sh = sets[0], sets[1] if shared else None
    _, offsets, perm, _ = binding.permute(dispatch(T, E, K, g), E)
    y = binding.grouped_swiglu(x, offsets, perm, K, ex, sh)
    torch.cuda.synchronize()
    binding.device_status()
    off, tok = offsets.tolist(), perm.long() // K
    for e in range(E):
        if off[e + 1] > off[e]:
            at = slice(off[e], off[e + 1])
            ref, tol = expert_ref(x[tok[at]], ex, e)
            assert 2.0 ** -126 < float(ref.abs().max()) < 1
            check_within(y[at], ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs() + 2.0 ** -134)
    if shared:
        ref, tol = expert_ref(x, sh, 0)
        check_within(y[T * K:], ref, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs() + 2.0 ** -134)
