"""The operators over a paged cache on a machine without a GPU: every argument check of
moe_cache_append, moe_indexer_scores and moe_latent_attention runs on the host before any CUDA call,
and the binding refuses tensors that do not fit before it reaches the library."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

from deepseek_moe_layer_gb300 import binding

FAKE = 0x10000  # never dereferenced: every call below fails its host checks
I31 = 1 << 31


def _rc(rc):
    return rc, binding.lib().moe_last_error().decode()


def _append(**kw):
    f = dict(x=FAKE, T=4, ldx=576, W=576, slots=FAKE, cache=FAKE, scales=None, rows=256,
             norm_weight=FAKE, norm_bias=None, norm_cols=512, eps=1e-6, positions=FAKE,
             inv_freq=FAKE, rope_cols=64, rope_at=512, interleaved=1, q=FAKE, q_out=FAKE, H=8,
             q_token=8 * 64, q_head=64, q_out_token=8 * 64, q_out_head=64)
    f.update(kw)
    return _rc(binding.lib().moe_cache_append(ctypes.byref(binding.AppendArgs(**f)), None))


@pytest.mark.parametrize("kw,msg", [
    (dict(x=None), "NULL"), (dict(slots=None), "NULL"), (dict(cache=None), "NULL"),
    (dict(norm_weight=None), "NULL"), (dict(positions=None), "NULL"), (dict(inv_freq=None), "NULL"),
    (dict(q_out=None), "NULL"),
    (dict(T=-1), "T = -1"), (dict(T=I31), "T = "),
    (dict(W=0), "W = 0"), (dict(W=12, ldx=16), "W = 12"), (dict(W=1032, ldx=1032), "W = 1032"),
    (dict(ldx=568), "ldx = 568"), (dict(ldx=580), "ldx = 580"),
    (dict(rows=-1), "rows = -1"),
    (dict(norm_cols=584), "norm_cols = 584"), (dict(norm_cols=12), "norm_cols = 12"),
    (dict(norm_cols=-8), "norm_cols = -8"), (dict(eps=-1.0), "eps"),
    (dict(rope_cols=24), "rope_cols = 24"), (dict(rope_cols=-16), "rope_cols = -16"),
    (dict(rope_at=520), "rope_at = 520"), (dict(rope_at=4), "rope_at = 4"),
    (dict(rope_at=-8), "rope_at = -8"),
    (dict(scales=FAKE), "multiple of 128"),
    (dict(rope_cols=0, rope_at=0), "q given without a rotation"),
    (dict(H=0), "H = 0"), (dict(H=1025), "H = 1025"),
    (dict(q_token=4), "strides"), (dict(q_head=4), "strides"), (dict(q_out_token=4), "strides"),
    (dict(q_out_head=4), "strides"),
    (dict(x=FAKE + 8), "16-byte"), (dict(cache=FAKE + 8), "16-byte"), (dict(q=FAKE + 8), "16-byte"),
    (dict(q_out=FAKE + 8), "16-byte"), (dict(slots=FAKE + 4), "aligned to"),
    (dict(positions=FAKE + 2), "aligned to"),
])
def test_append_refusals(kw, msg):
    rc, err = _append(**kw)
    assert rc == binding.MOE_ERR_INVALID and msg in err, err


@pytest.mark.parametrize("T,H,token,head,fits", [
    (4, 8, 512, 64, True), (4, 8, 8 * 576, 576, True), (4, 8, 64, 256, True), (1, 8, 0, 64, True),
    (4, 1, 64, 0, True), (1, 1, 0, 0, True), (4, 8, -512, -64, True),
    (4, 8, 0, 64, False), (4, 8, 512, 0, False), (4, 8, 504, 64, False), (4, 8, 512, 56, False),
    (4, 8, 64, 248, False), (4, 8, 512, 512, False), (4, 1, 56, 0, False), (1, 8, 0, 56, False),
    (4, 8, 1 << 62, (1 << 62) - 8, False), (4, 8, -(1 << 63), 64, True),
])
def test_append_query_rows_do_not_lie_on_each_other(T, H, token, head, fits):
    # (a call whose rows fit goes on to the next check: slots that are misaligned)
    rc, err = _append(T=T, H=H, q_out_token=token, q_out_head=head, slots=FAKE + 4)
    assert rc == binding.MOE_ERR_INVALID and ("aligned to" if fits else "overlap") in err, err


def test_append_nothing_to_do():
    assert _append(T=0, x=None, slots=None, q=None)[0] == binding.MOE_OK
    rc, err = _rc(binding.lib().moe_cache_append(None, None))
    assert rc == binding.MOE_ERR_INVALID and "args" in err


@pytest.mark.parametrize("f8", [False, True])
def test_append_to_a_cache_without_rows(f8):
    # its rows' address is NULL, as an empty tensor's is (the call goes on to the next check)
    kw = dict(W=512, ldx=512, rope_at=448, scales=FAKE) if f8 else {}
    rc, err = _append(cache=None, rows=0, slots=FAKE + 4, **kw)
    assert rc == binding.MOE_ERR_INVALID and "aligned to" in err, err


def _cache(**kw):
    f = dict(rows=FAKE, pages=16, page=64, table=FAKE, sequences=4, width=8)
    f.update(kw)
    return binding.PagedCache(**f)


PAGED = [
    (dict(page=0), "page = 0"), (dict(pages=-1), "pages = -1"), (dict(pages=I31), "pages = "),
    (dict(pages=I31 // 64), "2^31 rows"), (dict(width=-1), "width"),
    (dict(width=1 << 25), "positions"), (dict(sequences=-1), "sequences"),
    (dict(sequences=3), "without cu_tokens"), (dict(table=None), "NULL pointer in the cache"),
    (dict(rows=None), "NULL pointer in the cache"), (dict(table=FAKE + 2), "4-byte"),
    (dict(rows=FAKE + 8), "16-byte"),
]


def _scores(cache=None, q=FAKE, w=FAKE, T=4, H=64, ks=None, cu=None, lengths=FAKE, n=512, out=FAKE,
            ld=512, null=False):
    c = None if null else ctypes.byref(_cache(**(cache or {})))
    return _rc(binding.lib().moe_indexer_scores(q, w, T, H, c, ks, cu, lengths, n, out, ld, None))


@pytest.mark.parametrize("cache,msg", PAGED)
def test_scores_cache_refusals(cache, msg):
    rc, err = _scores(cache)
    assert rc == binding.MOE_ERR_INVALID and msg in err, err


@pytest.mark.parametrize("kw,msg", [
    (dict(null=True), "cache is NULL"), (dict(q=None), "NULL"), (dict(w=None), "NULL"),
    (dict(out=None), "NULL"), (dict(lengths=None), "NULL lengths"), (dict(T=-1), "T = -1"),
    (dict(T=I31), "T = "), (dict(H=0), "H = 0"), (dict(H=129), "H = 129"), (dict(n=-1), "n = -1"),
    (dict(n=I31 - 1, ld=I31), "n = "), (dict(ld=511), "ld = 511"), (dict(q=FAKE + 8), "16-byte"),
    (dict(w=FAKE + 2), "4-byte"), (dict(out=FAKE + 2), "4-byte"), (dict(ks=FAKE + 2), "4-byte"),
    (dict(cu=FAKE + 2), "4-byte"), (dict(lengths=FAKE + 2), "4-byte"),
    (dict(cu=FAKE, cache=dict(sequences=0)), "without a sequence"),
])
def test_scores_refusals(kw, msg):
    rc, err = _scores(**kw)
    assert rc == binding.MOE_ERR_INVALID and msg in err, err


@pytest.fixture(scope="module")
def list_bound(tmp_path_factory):
    d = tmp_path_factory.mktemp("list")
    header = os.path.join(os.path.dirname(binding.__file__), "csrc", "score_list.h")
    (d / "b.cc").write_text(f'#include "{header}"\nextern "C" long long bound(long long T, long long B, int tt, int gtok, '
                            "long long n, int keys) { return moe::score_list_bound(T, B, tt, gtok, n, keys); }\n")
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(d / "b.so"), str(d / "b.cc")], check=True)
    f = ctypes.CDLL(str(d / "b.so")).bound
    f.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_int]
    f.restype = ctypes.c_longlong
    return f


def _entries(new, tt, gtok, n):
    """The list's entries where every token sees all n positions: groups of tt tokens, cut at sequences' ends."""
    owner = [b for b, t in enumerate(new) for _ in range(t)]
    total = 0
    for u in range(0, len(owner), tt):
        group = owner[u:u + tt]
        total += sum(-(-group.count(b) // gtok) for b in set(group)) * -(-n // 128)
    return total


def test_scores_list_is_no_longer_than_its_bound(list_bound):
    # (CTAs that the grid lacks leave the device idle: 1, 2 and 1 tokens of three sequences are four parts)
    assert _entries([1, 2, 1], 2, 2, 4096) == list_bound(4, 3, 2, 2, 4096, 128) == 128
    r = random.Random(1)
    for _ in range(2000):
        new = [r.choice((0, 1, 1, 2, 5, r.randint(0, 70))) for _ in range(r.randint(1, 12))]
        T, tt, gtok, n = sum(new), r.randint(1, 32), r.choice((1, 2, 4, 8)), r.randint(1, 3000)
        if T:
            assert _entries(new, tt, gtok, n) <= list_bound(T, len(new), tt, gtok, n, 128), (new, tt, gtok, n)
            assert _entries([1] * T, 1, gtok, n) == list_bound(T, 0, 1, gtok, n, 128)
            assert _entries([T], tt, gtok, n) <= list_bound(T, 1, tt, gtok, n, 128) < \
                _entries([T], tt, gtok, n) + -(-n // 128) * -(-tt // gtok)


def test_scores_nothing_to_do():
    assert _scores(dict(sequences=0), T=0, q=None, w=None, out=None, lengths=None)[0] == binding.MOE_OK
    assert _scores(n=0, ld=0, out=None)[0] == binding.MOE_OK


def _attention(cache=None, q=FAKE, T=4, H=128, qt=128 * 576, qh=576, cu=None, lengths=FAKE, inds=None,
               k=0, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, null=False):
    c = None if null else ctypes.byref(_cache(**(cache or {})))
    return _rc(binding.lib().moe_latent_attention(q, T, H, qt, qh, c, cu, lengths, 0.1, inds, k, out,
                                                  lse, ws, ws_bytes, None))


@pytest.mark.parametrize("cache,msg", PAGED)
def test_attention_cache_refusals(cache, msg):
    rc, err = _attention(cache)
    assert rc == binding.MOE_ERR_INVALID and msg in err, err


@pytest.mark.parametrize("kw,msg", [
    (dict(null=True), "cache is NULL"), (dict(q=None), "NULL"), (dict(out=None), "NULL"),
    (dict(ws=None), "NULL"), (dict(lengths=None), "NULL lengths"), (dict(T=-1), "T = -1"),
    (dict(H=0), "H = 0"), (dict(H=129), "H = 129"), (dict(qt=4), "strides"), (dict(qh=4), "strides"),
    (dict(inds=FAKE, k=0), "k = 0"), (dict(q=FAKE + 8), "16-byte"), (dict(out=FAKE + 8), "16-byte"),
    (dict(inds=FAKE + 2, k=4), "4-byte"), (dict(lse=FAKE + 2), "4-byte"), (dict(ws=FAKE + 16), "256-byte"),
    (dict(ws_bytes=1024), "ws_bytes = 1024"),
])
def test_attention_refusals(kw, msg):
    rc, err = _attention(**kw)
    assert rc == binding.MOE_ERR_INVALID and msg in err, err


def test_attention_workspace():
    L = binding.lib()
    size = L.moe_latent_attention_workspace_bytes
    assert size(0, 100) == 0 and size(-1, 100) == 0 and size(1, -1) == 0
    assert 0 < size(1, 0) <= size(1, 4096) <= size(64, 4096) <= size(1 << 20, 1 << 20) < 64 << 20
    assert _attention(dict(sequences=0), T=0, q=None, out=None, ws=None, lengths=None,
                      ws_bytes=0)[0] == binding.MOE_OK


def test_valid_calls_without_gpu_fail_loudly():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for rc, err in (_append(), _scores(), _attention()):
        assert rc == binding.MOE_ERR_NODEVICE and err


# ---- the binding --------------------------------------------------------------------------------

BF, F8, F32, I32, I64 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32, torch.int64


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def _call_append(**kw):
    a = dict(x=z(3, 576), slots=z(3, dtype=I64), cache=z(2, 64, 576), norm_weight=z(512, dtype=F32),
             positions=z(3, dtype=I32), inv_freq=z(32, dtype=F32), rope_at=512, q=z(3, 8, 64))
    a.update(kw)
    return binding.cache_append(**a)


@pytest.mark.parametrize("kw,exc,msg", [
    (dict(x=z(3, 576, dtype=F32)), TypeError, "x: dtype"), (dict(x=z(3 * 576)), ValueError, "x must"),
    (dict(x=z(576, 3).t()), ValueError, "unit stride"),
    (dict(slots=z(3, dtype=I32)), TypeError, "slots"), (dict(slots=z(4, dtype=I64)), ValueError, "slots"),
    (dict(slots=[1, 2, 3]), TypeError, "slots"),
    (dict(cache=z(2, 64, 512)), ValueError, "cache"), (dict(cache=z(2, 64, 576, dtype=F8)), TypeError, "cache"),
    (dict(cache=z(2, 64, 1152)[..., ::2]), ValueError, "contiguous"),
    (dict(scales=z(2, 64, 4, dtype=F32)), TypeError, "cache"),
    (dict(norm_weight=z(512)), TypeError, "norm_weight"),
    (dict(norm_bias=z(511, dtype=F32)), ValueError, "norm_bias"),
    (dict(norm_weight=None, norm_bias=z(512, dtype=F32)), ValueError, "without norm_weight"),
    (dict(positions=None), ValueError, "without positions"), (dict(positions=z(3, dtype=I64)), TypeError, "positions"),
    (dict(inv_freq=z(32)), TypeError, "inv_freq"), (dict(inv_freq=None), ValueError, "q given without inv_freq"),
    (dict(q=z(3, 8, 32)), ValueError, "q must"), (dict(q=z(3, 8, 64, dtype=F32)), TypeError, "q: dtype"),
    (dict(q_out=z(3, 9, 64)), ValueError, "q_out must"), (dict(q=None, q_out=z(3, 8, 64)), ValueError, "without q"),
    (dict(), ValueError, "CUDA device"),
])
def test_binding_append(kw, exc, msg):
    with pytest.raises(exc, match=msg):
        _call_append(**kw)


def test_attention_over_no_selection(monkeypatch):
    # [T, 0] entries select nothing, which the library refuses; its address is 0, which means all positions
    monkeypatch.setattr(binding, "_raw_stream", lambda t, stream: 0)
    for T, ws in ((3, None), (90, None), (3, torch.zeros(1 << 26, dtype=torch.uint8))):
        with pytest.raises(binding.MoeError, match="k = 0"):
            binding.latent_attention(z(T, 16, 576), z(4, 64, 576), z(T, 2, dtype=I32), z(T, dtype=I32), 0.1,
                                     inds=z(T, 0, dtype=I32), ws=ws)
    for k in (0, 5):  # no tokens: nothing to do
        assert binding.latent_attention(z(0, 16, 576), z(4, 64, 576), z(0, 2, dtype=I32), z(0, dtype=I32), 0.1,
                                        inds=z(0, k, dtype=I32), ws=z(0, dtype=torch.uint8)).shape == (0, 16, 512)


def _call_scores(**kw):
    a = dict(q=z(3, 64, 128), weights=z(3, 64, dtype=F32), keys=z(4, 64, 128),
             block_table=z(3, 2, dtype=I32), lengths=z(3, dtype=I32), n=100)
    a.update(kw)
    return binding.indexer_scores(**a)


@pytest.mark.parametrize("kw,exc,msg", [
    (dict(q=z(3, 64, 64)), ValueError, "q must"), (dict(q=z(3, 64, 128, dtype=F8)), TypeError, "q: dtype"),
    (dict(q=z(3, 64, 256)[..., ::2]), ValueError, "q must be contiguous"),
    (dict(weights=z(3, 64)), TypeError, "weights"), (dict(weights=z(3, 63, dtype=F32)), ValueError, "weights"),
    (dict(keys=z(4, 64, 64)), ValueError, "keys"), (dict(keys=z(4, 64, 128, dtype=F8)), TypeError, "keys"),
    (dict(key_scales=z(4, 64, 1, dtype=F32)), TypeError, "q: dtype"),
    (dict(q=z(3, 64, 128, dtype=F8), keys=z(4, 64, 128, dtype=F8), key_scales=z(4, 63, 1, dtype=F32)), ValueError,
     "key_scales"),
    (dict(block_table=z(2, 2, dtype=I32)), ValueError, "cu_tokens is None"),
    (dict(block_table=z(6, dtype=I32)), ValueError, "block_table"), (dict(block_table=z(3, 2, dtype=I64)), TypeError, "block_table"),
    (dict(lengths=z(3, dtype=I64)), TypeError, "lengths"), (dict(lengths=z(2, dtype=I32)), ValueError, "lengths"),
    (dict(cu_tokens=z(3, dtype=I32)), ValueError, "cu_tokens"), (dict(cu_tokens=z(4, dtype=I64)), TypeError, "cu_tokens"),
    (dict(out=z(3, 100)), TypeError, "out"), (dict(out=z(3, 99, dtype=F32)), ValueError, "out"),
    (dict(out=z(100, 3, dtype=F32).t()), ValueError, "out"),
    (dict(), ValueError, "CUDA device"),
])
def test_binding_scores(kw, exc, msg):
    with pytest.raises(exc, match=msg):
        _call_scores(**kw)


def _call_attention(**kw):
    a = dict(q=z(3, 16, 576), cache=z(4, 64, 576), block_table=z(3, 2, dtype=I32),
             lengths=z(3, dtype=I32), scale=0.1)
    a.update(kw)
    return binding.latent_attention(**a)


@pytest.mark.parametrize("kw,exc,msg", [
    (dict(q=z(3, 16, 512)), ValueError, "q must"), (dict(q=z(3, 16, 576, dtype=F32)), TypeError, "q: dtype"),
    (dict(q=z(3, 16, 1152)[..., ::2]), ValueError, "unit stride"),
    (dict(cache=z(4, 64, 512)), ValueError, "cache"), (dict(cache=z(4, 64, 576, dtype=F32)), TypeError, "cache"),
    (dict(inds=z(2, 8, dtype=I32)), ValueError, "inds"), (dict(inds=z(3, 8, dtype=I64)), TypeError, "inds"),
    (dict(out=z(3, 16, 576)), ValueError, "out"), (dict(out=z(3, 16, 512, dtype=F32)), TypeError, "out"),
    (dict(ws=z(16)), TypeError, "ws"), (dict(lengths=z(4, dtype=I32)), ValueError, "lengths"),
    (dict(), ValueError, "CUDA device"),
])
def test_binding_attention(kw, exc, msg):
    with pytest.raises(exc, match=msg):
        _call_attention(**kw)


# ---- what the binding hands to the library --------------------------------------------------------

class _Recorder:
    """Stands in for the library: keeps each call's arguments and answers MOE_OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 1 << 20 if name.endswith("_bytes") else 0
        return call


@pytest.fixture
def calls(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(binding, "_lib", r)
    monkeypatch.setattr(binding, "_raw_stream", lambda t, stream: 0)
    return r.calls


def test_scores_of_an_empty_8_bit_cache_stay_8_bit(calls):
    # an empty tensor's address is 0, and without key_scales the library takes q for bf16: twice its bytes
    _call_scores(q=z(3, 64, 128, dtype=F8), keys=z(0, 64, 128, dtype=F8), key_scales=z(0, 64, 1, dtype=F32))
    _call_scores(q=z(3, 64, 128, dtype=F8), keys=z(4, 64, 128, dtype=F8), key_scales=z(4, 64, dtype=F32))
    _call_scores()
    scales = [args[5] for name, args in calls]
    assert scales[0] and scales[1] and scales[2] is None


@pytest.mark.parametrize("W", [8, 64, 120, 192, 576])
def test_append_8_bit_rows_are_whole_blocks(calls, W):
    # (below 128 columns the scales are an empty tensor, whose address is 0: a cache of bf16 rows to the library)
    with pytest.raises(ValueError, match="multiple of 128"):
        binding.cache_append(z(3, W), z(3, dtype=I64), z(2, 64, W, dtype=F8), scales=z(2, 64, W // 128, dtype=F32))
    assert not calls


@pytest.mark.parametrize("pages,f8", [(0, True), (2, True), (2, False)])
def test_append_says_which_type_its_cache_has(calls, pages, f8):
    binding.cache_append(z(3, 256), z(3, dtype=I64), z(pages, 64, 256, dtype=F8 if f8 else BF),
                         scales=z(pages, 64, 2, dtype=F32) if f8 else None)
    assert (calls[0][1][0]._obj.scales is not None) == f8


@pytest.mark.parametrize("T,k", [(3, 0), (90, 0), (3, 5), (3, None)])
def test_attention_says_whether_positions_are_selected(calls, T, k):
    binding.latent_attention(z(T, 16, 576), z(4, 64, 576), z(T, 2, dtype=I32), z(T, dtype=I32), 0.1,
                             inds=None if k is None else z(T, k, dtype=I32))
    chosen, n = calls[-1][1][9:11]
    assert bool(chosen) == (k is not None) and n == (k or 0)


def _meta(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta")


BIG = 1 << 32  # a multiple of it vanishes in 32 bits


@pytest.mark.parametrize("kw", [
    dict(n=BIG + 100, out=_meta(3, BIG + 100, dtype=F32)), dict(block_table=_meta(3, BIG + 2, dtype=I32)),
    dict(keys=_meta(0, BIG + 64, 128)),
])
def test_scores_sizes_beyond_32_bits(calls, kw):
    with pytest.raises(ValueError, match="32 bits"):
        _call_scores(**kw)
    assert not calls


@pytest.mark.parametrize("kw", [
    dict(inds=_meta(3, BIG + 5, dtype=I32)), dict(block_table=_meta(3, BIG + 2, dtype=I32)),
    dict(q=_meta(3, 1, 576).expand(3, BIG + 16, 576)), dict(cache=_meta(0, BIG + 64, 576)),
])
def test_attention_sizes_beyond_32_bits(calls, kw):
    with pytest.raises(ValueError, match="32 bits"):
        _call_attention(**kw)
    assert not calls


@pytest.mark.parametrize("kw", [
    dict(rope_at=BIG + 512), dict(rope_at=512 - BIG), dict(x=_meta(3, BIG + 576), cache=_meta(2, 64, BIG + 576)),
    dict(norm_weight=_meta(BIG + 512, dtype=F32)),
    dict(q=_meta(3, 1, 64).expand(3, BIG + 8, 64), q_out=_meta(3, 1, 64).expand(3, BIG + 8, 64)),
])
def test_append_sizes_beyond_32_bits(calls, kw):
    with pytest.raises(ValueError, match="32 bits"):
        _call_append(**kw)
    assert not calls
