"""Refusals of the block-scaled e4m3 calls and of the grouped softmax gate, on a machine without
a GPU: every check runs on the host before any CUDA call."""
import ctypes

import pytest
import torch

from deepseek_moe_layer_gb300 import binding

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails its host checks
BAD = binding.MOE_ERR_INVALID
F8 = torch.float8_e4m3fn


def _err():
    return binding.lib().moe_last_error().decode()


def _quant(x=FAKE, dtype=1, rows=4, n=256, ld=256, block_rows=1, codes=FAKE, scales=FAKE):
    return binding.lib().moe_quantize_blocks(x, dtype, rows, n, ld, block_rows, codes, scales, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(x=None), "NULL"), (dict(codes=None), "NULL"), (dict(scales=None), "NULL"),
    (dict(dtype=2), "dtype"), (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"),
    (dict(n=0), "n = 0"), (dict(n=24), "n = 24"), (dict(n=-16), "n = -16"),
    (dict(ld=248), "ld = 248"), (dict(ld=260), "ld = 260"), (dict(dtype=0, ld=258), "ld = 258"),
    (dict(block_rows=0), "block_rows"), (dict(block_rows=64), "block_rows"),
    (dict(x=ctypes.c_void_p(0x1008)), "aligned"), (dict(codes=ctypes.c_void_p(0x1008)), "aligned"),
    (dict(scales=ctypes.c_void_p(0x1002)), "aligned"),
    (dict(rows=(1 << 31) - 1, n=1 << 20, ld=1 << 20), "too many blocks"),
])
def test_quantize_refusals(kw, msg):
    assert _quant(**kw) == BAD
    assert msg in _err()


def _matmul(a=FAKE, sa=FAKE, M=4, lda=256, w=FAKE, sw=FAKE, N=8, K=256, dt=1, out=FAKE):
    return binding.lib().moe_matmul_blocks(a, sa, M, lda, w, sw, N, K, dt, out, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(a=None), "NULL"), (dict(sa=None), "NULL"), (dict(w=None), "NULL"),
    (dict(sw=None), "NULL"), (dict(out=None), "NULL"), (dict(M=0, w=None), "NULL"),
    (dict(M=-1), "M = -1"), (dict(M=1 << 31), "M = "), (dict(N=0), "N = 0"), (dict(K=0), "K = 0"),
    (dict(K=8, lda=16), "K = 8"), (dict(K=200, lda=256), "K = 200"), (dict(lda=240), "lda = 240"),
    (dict(lda=264), "lda = 264"), (dict(dt=3), "dtype"),
    (dict(a=ctypes.c_void_p(0x1004)), "aligned"), (dict(w=ctypes.c_void_p(0x1001)), "aligned"),
    (dict(out=ctypes.c_void_p(0x1001)), "aligned"),
    (dict(dt=0, out=ctypes.c_void_p(0x1002)), "aligned"),
    (dict(sa=ctypes.c_void_p(0x1002)), "aligned"),
    (dict(M=(1 << 31) - 1, N=(1 << 31) - 1), "too many tiles"),
])
def test_matmul_refusals(kw, msg):
    assert _matmul(**kw) == BAD
    assert msg in _err()


def test_empty_calls_do_nothing():
    assert _quant(rows=0, x=None, codes=None, scales=None) == binding.MOE_OK
    assert _matmul(M=0, a=None, sa=None, out=None) == binding.MOE_OK


def _grouped(E=16, K=2, G=4, tg=2, rows=3, logits=FAKE, inds=FAKE, scores=FAKE, dtype=0):
    p = binding.route_params(K, G, tg, True, 1.0)
    return binding.lib().moe_route_softmax_grouped(logits, dtype, rows, E, None, ctypes.byref(p),
                                                   inds, scores, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(logits=None), "NULL"), (dict(inds=None), "NULL"), (dict(scores=None), "NULL"),
    (dict(dtype=9), "dtype"), (dict(rows=-2), "rows"), (dict(E=0), "E = 0"),
    (dict(E=1025, G=1, tg=1), "E = 1025"), (dict(G=0), "n_group"), (dict(G=3), "not divisible"),
    (dict(E=66, G=33, tg=1), "n_group = 33"), (dict(tg=0), "topk_group"), (dict(tg=5), "topk_group"),
    (dict(K=0), "top_k"), (dict(K=9), "top_k = 9"), (dict(E=64, G=1, tg=1, K=33), "top_k = 33"),
])
def test_grouped_gate_refusals(kw, msg):
    assert _grouped(**kw) == BAD
    assert msg in _err()


def test_grouped_gate_empty_and_without_params():
    assert _grouped(rows=0, logits=None, inds=None, scores=None) == binding.MOE_OK
    assert binding.lib().moe_route_softmax_grouped(FAKE, 0, 3, 16, None, None, FAKE, FAKE,
                                                   None) == BAD


def _ew(bits=binding.MOE_BITS_E4M3, **kw):
    f = dict(gate=0x1000, up=0x1000, down=0x1000, gate_scale=0x1000, up_scale=0x1000,
             down_scale=0x1000)
    f.update(kw)
    return binding.ExpertWeights(bits, 0, f["gate"], f["up"], f["down"], f["gate_scale"], None,
                                 f["up_scale"], None, f["down_scale"], None)


def _swiglu(experts, shared=None, T=4, d=256, I=128, E=16, K=2, ws_bytes=1 << 30):
    return binding.lib().moe_grouped_swiglu(
        FAKE, T, d, I, E, K, FAKE, FAKE, ctypes.byref(experts),
        None if shared is None else ctypes.byref(shared), FAKE, ctypes.c_void_p(0x10000), ws_bytes,
        None)


@pytest.mark.parametrize("kw,msg", [
    (dict(gate=None), "NULL"), (dict(down_scale=None), "scale pointer is NULL"),
    (dict(up=0x1008), "16-byte aligned"), (dict(gate_scale=0x1002), "4-byte aligned"),
])
def test_scaled_expert_weight_refusals(kw, msg):
    assert _swiglu(_ew(**kw)) == BAD
    assert msg in _err()
    assert _swiglu(_ew(), shared=_ew(**kw)) == BAD
    assert "shared expert" in _err() and msg in _err()


def test_scaled_experts_need_a_scaled_shared_expert():
    bf16 = binding.ExpertWeights(16, 0, 0x1000, 0x1000, 0x1000, *([None] * 6))
    assert _swiglu(_ew(), shared=bf16) == BAD and "MOE_BITS_E4M3" in _err()
    assert _swiglu(bf16, shared=_ew()) == BAD and "bits = 264" in _err()


def test_scaled_experts_workspace_and_sizes():
    L = binding.lib()
    need = L.moe_grouped_swiglu_workspace_bytes(4, 256, 128, 16, 1, 1)
    R = 4 * 1 + 4  # slots: codes and fp32 scales of the rows and of h, the inverse dispatch
    al = lambda v: (v + 255) // 256 * 256  # noqa: E731
    scaled = al(R * 256) + al(R * 2 * 4) + al(R * 128) + al(R * 4) + al(4 * 1 * 4)
    assert need >= scaled
    assert _swiglu(_ew(), shared=_ew(), K=1, ws_bytes=scaled - 1) == BAD and "ws_bytes" in _err()
    assert _swiglu(_ew(), E=1024, d=1 << 22, I=128, T=1, K=1) == BAD and "too large" in _err()
    assert _swiglu(_ew(), d=200) == BAD and "d = 200" in _err()


def test_forward_takes_the_grouped_gate_without_a_bias():
    L = binding.lib()
    a = binding.LayerArgs()
    a.route_kind, a.x, a.T, a.d, a.I, a.E = binding.MOE_ROUTE_SOFTMAX_GROUPED, 0x1000, 4, 256, 128, 16
    a.w_router, a.y = 0x1000, 0x1000
    ew = _ew()
    a.experts = ctypes.pointer(ew)
    for K, G, tg, msg in ((9, 4, 2, "top_k = 9"), (2, 3, 1, "not divisible"), (2, 4, 0, "topk_group")):
        a.params = binding.route_params(K, G, tg, True, 1.0)
        assert L.moe_forward_ex(ctypes.byref(a), ctypes.c_void_p(0x10000), 1 << 30, None) == BAD
        assert msg in _err()
    a.params = binding.route_params(8, 4, 2, True, 1.0)
    rc = L.moe_forward_ex(ctypes.byref(a), ctypes.c_void_p(0x10000), 64, None)
    assert rc == BAD and "ws_bytes" in _err()


def test_binding_checks_types_and_shapes():
    x = torch.zeros(4, 256)
    with pytest.raises(TypeError):
        binding.quantize_blocks(x.half())
    with pytest.raises(ValueError):
        binding.quantize_blocks(x.t())
    with pytest.raises(ValueError):
        binding.quantize_blocks(x, codes=torch.zeros(4, 128).to(F8))
    with pytest.raises(TypeError):
        binding.quantize_blocks(x, scales=torch.zeros(4, 2, dtype=torch.bfloat16))
    a, w = torch.zeros(4, 256).to(F8), torch.zeros(130, 256).to(F8)
    sa, sw = torch.ones(4, 2), torch.ones(2, 2)
    with pytest.raises(TypeError):
        binding.matmul_blocks(x, sa, w, sw)
    with pytest.raises(ValueError):
        binding.matmul_blocks(a, sa[:, :1].contiguous(), w, sw)
    with pytest.raises(ValueError):
        binding.matmul_blocks(a, sa, w, sw[:1])
    with pytest.raises(ValueError):
        binding.matmul_blocks(a, sa, w[:, :128].contiguous(), sw)
    with pytest.raises(TypeError):
        binding.matmul_blocks(a, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        binding.route_softmax_grouped(x, 2, 4, 2, True, 1.0, bias=torch.zeros(4))
    # host memory never reaches the library
    for call in (lambda: binding.quantize_blocks(x), lambda: binding.matmul_blocks(a, sa, w, sw),
                 lambda: binding.route_softmax_grouped(x, 2, 4, 2, True, 1.0)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    e = {"bits": binding.MOE_BITS_E4M3, "gate": torch.zeros(2, 128, 256).to(F8),
         "up": torch.zeros(2, 128, 256).to(F8), "down": torch.zeros(2, 256, 128).to(F8),
         "gate_s": torch.ones(2, 1, 2), "up_s": torch.ones(2, 1, 2), "down_s": torch.ones(2, 2, 1)}
    assert binding.expert_weights(e).bits == binding.MOE_BITS_E4M3
    with pytest.raises(ValueError):
        binding.expert_weights({**e, "down_s": torch.ones(2, 1, 2)})
    with pytest.raises(TypeError):
        binding.expert_weights({**e, "up": torch.zeros(2, 128, 256)})


# The kernels count columns in 32 bits, rounded up to their tiles: the last sizes below 2^31 are
# refused (they would have been counted as negative, past every bound).
@pytest.mark.parametrize("n", [(1 << 31) - 16, (1 << 31) - 128, (1 << 31) - 496])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_refuses_sizes_that_round_up_past_32_bits(n, block_rows):
    assert _quant(rows=1, n=n, ld=n, block_rows=block_rows) == BAD
    assert f"n = {n}" in _err()


@pytest.mark.parametrize("kw", [dict(N=(1 << 31) - 1, K=16, lda=16), dict(N=(1 << 31) - 511, K=16, lda=16),
                                dict(K=(1 << 31) - 16, lda=(1 << 31) - 16, N=1),
                                dict(K=(1 << 31) - 496, lda=(1 << 31) - 496, N=1)])
def test_matmul_refuses_sizes_that_round_up_past_32_bits(kw):
    assert _matmul(M=1, **kw) == BAD
    assert ("K = " if kw["K"] > 16 else "N = ") in _err()


def _dict(E, d, I, device="cpu"):
    z = lambda *s: torch.zeros(*s, device=device).to(F8)  # noqa: E731
    one = lambda *s: torch.ones(*s, device=device)  # noqa: E731
    b = lambda n: -(-n // 128)  # noqa: E731
    return {"bits": binding.MOE_BITS_E4M3, "gate": z(E, I, d), "up": z(E, I, d), "down": z(E, d, I),
            "gate_s": one(E, b(I), b(d)), "up_s": one(E, b(I), b(d)), "down_s": one(E, b(d), b(I))}


def _other(w, key, E, d, I):
    """w with `key` and its scales of another shape."""
    o = _dict(E, d, I)
    return {**w, key: o[key], key + "_s": o[key + "_s"]}


GOOD = (4, 256, 128)  # E, d, I


@pytest.mark.parametrize("experts,shared,msg", [
    (_dict(3, 256, 128), None, "gate"),                                   # fewer than E experts
    (_dict(4, 384, 128), None, "gate"),                                   # another width than x
    (_other(_dict(*GOOD), "up", 4, 256, 256), None, "up"),                # up of another I
    (_other(_dict(*GOOD), "up", 2, 256, 128), None, "up"),
    (_other(_dict(*GOOD), "down", 4, 256, 256), None, "down"),
    (_other(_dict(*GOOD), "down", 3, 256, 128), None, "down"),
    (_dict(*GOOD), _dict(1, 256, 256), "gate"),                           # a shared expert of its own I
    (_dict(*GOOD), _other(_dict(1, 256, 128), "down", 1, 128, 128), "down"),
])
def test_experts_of_other_shapes_never_reach_the_library(experts, shared, msg):
    """Codes and scales agree with each other, but not with x, the dispatch or the other weights."""
    x = torch.zeros(5, 256, dtype=torch.bfloat16)
    offsets, perm = torch.zeros(5, dtype=torch.int32), torch.zeros(10, dtype=torch.int32)
    with pytest.raises(ValueError, match=msg):
        binding.grouped_swiglu(x, offsets, perm, 2, experts, shared, I=128)
    with pytest.raises(ValueError, match=msg):
        binding.MoELayer(torch.zeros(4, 256, dtype=torch.bfloat16), None, {**experts, "gate": experts["gate"]},
                         shared, 2, 1, 1, True, 1.0, route_kind=binding.MOE_ROUTE_SOFTMAX)


def test_shared_experts_may_leave_out_their_only_dimension():
    one = {k: v[0] if isinstance(v, torch.Tensor) else v for k, v in _dict(1, 256, 128).items()}
    for shared in (one, _dict(1, 256, 128)):
        with pytest.raises(ValueError, match="CUDA device"):
            binding.grouped_swiglu(torch.zeros(5, 256, dtype=torch.bfloat16),
                                   torch.zeros(5, dtype=torch.int32), torch.zeros(10, dtype=torch.int32),
                                   2, _dict(*GOOD), shared)


def test_e4m3_experts_check_the_dispatch_and_the_device():
    x = torch.zeros(5, 256, dtype=torch.bfloat16)
    offsets, perm = torch.zeros(5, dtype=torch.int32), torch.zeros(10, dtype=torch.int32)
    w = _dict(*GOOD)
    with pytest.raises(TypeError, match="offsets"):
        binding.grouped_swiglu(x, offsets.long(), perm, 2, w)
    with pytest.raises(TypeError, match="perm"):
        binding.grouped_swiglu(x, offsets, perm.long(), 2, w)
    with pytest.raises(ValueError, match="perm"):
        binding.grouped_swiglu(x, offsets, perm[:9].contiguous(), 2, w)
    with pytest.raises(ValueError, match="perm"):
        binding.grouped_swiglu(x, offsets, torch.zeros(20, dtype=torch.int32)[::2], 2, w)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.grouped_swiglu(x, offsets, perm, 2, w)
    meta = _dict(*GOOD, device="meta")
    with pytest.raises(ValueError, match="gate is on meta"):
        binding.grouped_swiglu(x, offsets, perm, 2, meta)
    with pytest.raises(ValueError, match="gate is on meta"):
        binding.MoELayer(torch.zeros(4, 256, dtype=torch.bfloat16), None, meta, None, 2, 1, 1, True, 1.0,
                         route_kind=binding.MOE_ROUTE_SOFTMAX)


def test_e4m3_layer_checks_its_rows():
    layer = binding.MoELayer(torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4), _dict(*GOOD), None,
                             2, 1, 1, True, 1.0)
    with pytest.raises(ValueError, match="x must be"):
        layer(torch.zeros(5, 384, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="y must be"):
        layer(torch.zeros(5, 256, dtype=torch.bfloat16), y=torch.zeros(4, 256, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA device"):
        layer(torch.zeros(5, 256, dtype=torch.bfloat16))


@pytest.mark.parametrize("shape", [(3,), (5,), (1, 4)])
def test_grouped_gate_of_a_layer_checks_its_bias(shape):
    """The gate reads E of them."""
    with pytest.raises(ValueError, match="bias"):
        binding.MoELayer(torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(shape), _dict(*GOOD), None,
                         2, 1, 1, True, 1.0, route_kind=binding.MOE_ROUTE_SOFTMAX_GROUPED)


def test_bf16_layer_with_one_expert_per_token_needs_what_it_always_needed():
    """The reported size covers e4m3 experts too, which with top_k = 1 and a shared expert can need
    more; a layer of bf16 experts takes its own size, and the fixed workspace its old batches."""
    L = binding.lib()
    T, d, I, E = 600, 7168, 128, 16
    al = lambda v: (v + 255) // 256 * 256  # noqa: E731
    fixed = [al(d // 512 * T * E * 4), *[al(T * 4)] * 2, al(E * 4), al((E + 1) * 4), *[al(T * 4)] * 2,
             al(2 * T * d * 2)]  # logits, choices and dispatch; the experts' outputs
    bf16 = sum(fixed) + al(T * d * 2) + al(2 * T * I * 2)  # gathered rows and h
    e4m3 = sum(fixed) + al(2 * T * d) + al(2 * T * d // 128 * 4) + al(2 * T * I) + al(2 * T * I // 128 * 4) + al(T * 4)
    assert bf16 < e4m3 == L.moe_forward_workspace_bytes(T, d, I, E, 1, 1)
    ew = binding.ExpertWeights(16, 0, 0x1000, 0x1000, 0x1000, *([None] * 6))
    p = binding.route_params(1, 1, 1, True, 1.0)
    f, ref = FAKE, ctypes.byref
    call = lambda w, n: L.moe_forward(f, T, d, I, E, f, f, None, ref(p), ref(w), ref(w), f, None, None,  # noqa: E731
                                      None, ctypes.c_void_p(0x10000), n, None)
    assert call(ew, 1000) == BAD and f"< {bf16} required" in _err()
    assert call(_ew(), 1000) == BAD and f"< {e4m3} required" in _err()
    # the largest batch whose bf16 workspace fits the fixed one: refused (if at all) for x's alignment
    size = 64 << 20
    T = next(t for t in range(3000, 0, -1) if L.moe_forward_workspace_bytes(t, d, I, E, 1, 1) <= size) + 4
    odd = ctypes.c_void_p(0x1008)
    args = (odd, T, d, I, E, f, f, None, ref(p))
    assert L.moe_forward_workspace_bytes(T, d, I, E, 1, 1) > size
    L.moe_forward_noalloc(*args, ref(ew), ref(ew), f, None, None, None, None)
    assert "bytes of workspace" not in _err()
    e = _ew()
    assert L.moe_forward_noalloc(*args, ref(e), ref(e), f, None, None, None, None) == BAD
    assert "bytes of workspace" in _err()
