"""Host-side checks of rotary positions, the KV cache and the attention of
drafted tokens that need no GPU: the oracle against worked values, the rotary
steps against their formula, and the refusals."""
import ctypes
import math

import numpy as np
import pytest

import quantized_weight_decode_gb300 as nqp
from cases import attention_products_bar
from oracle import cache as oc


@pytest.fixture(scope="session", autouse=True)
def built():
    nqp.build()
    return nqp.lib()


# ---------------------------------------------------------------- the oracle
def test_oracle_rotation_by_a_quarter_turn():
    steps = np.array([1 << 62], dtype=np.uint64)          # a quarter turn a position
    x = np.array([[[1.0, 2.0, 7.0]]])
    for inter in (False, True):
        assert np.allclose(oc.rope(x, [1], steps, inter), [[[-2, 1, 7]]], atol=1e-15)
        assert np.allclose(oc.rope(x, [2], steps, inter), [[[-1, -2, 7]]], atol=1e-15)
        assert np.allclose(oc.rope(x, [-1], steps, inter, factor=2.0), [[[4, -2, 7]]], atol=1e-15)
        assert np.allclose(oc.rope(x, [1], steps, inter, adjoint=True), [[[2, -1, 7]]], atol=1e-15)


def test_oracle_quantise_worked_example():
    x = np.zeros((1, 64), np.float32)
    x[0, :4] = [127.0, -127.0, 0.5, 1.5]
    c, s = oc.quantise(x, 8)
    assert s[0, 0] == 1.0 and c[0, :4].tolist() == [127, -127, 0, 2]       # half to even
    c, s = oc.quantise(x * np.float32(7 / 127), 4)
    assert abs(float(s[0, 0]) - 1.0) < 1e-3 and c[0, :2].tolist() == [7, -7]
    c, s = oc.quantise(np.zeros((1, 64)), 4)
    assert s[0, 0] == 0 and not c.any()


@pytest.mark.parametrize("bits", [4, 8])
def test_oracle_packing_round_trip(bits):
    lo = -(1 << (bits - 1))
    c = np.arange(lo, -lo, dtype=np.int16).astype(np.int8)
    c = np.tile(c, 64 * 4 // len(c) + 1)[:256].reshape(2, 128)
    raw = oc.pack_codes(c, bits)
    assert raw.shape == (2, 128 * bits // 8) and np.array_equal(oc.unpack_codes(raw, bits), c)


def test_oracle_attention_closed_forms():
    k = np.zeros((3, 1, 64))
    v = np.arange(3 * 64, dtype=np.float64).reshape(3, 1, 64)
    q = np.ones((2, 2, 64))
    seen = np.array([[1, 1, 1], [0, 0, 0]], bool)
    o, lse, spread, _ = oc.attention(q, k, v, 0.5, seen)
    assert np.allclose(o[0], v.mean(0)) and np.allclose(lse[0], math.log(3)) and np.allclose(spread[0], v.mean(0))
    assert not o[1].any() and np.all(np.isneginf(lse[1]))
    k[2] = 1000.0                                          # one key takes it all
    o, lse, *_ = oc.attention(q, k, v, 0.5, seen)
    assert np.allclose(o[0], v[2]) and np.allclose(lse[0], 32000.0)


# ---------------------------------------------------------------- rotary steps
@pytest.mark.parametrize("scaling,f,ctx", [("plain", 1.0, 0.0), ("linear", 4.0, 0.0), ("ntk", 8.0, 0.0),
                                           ("yarn", 4.0, 8192.0), ("yarn", 1.0, 4096.0)])
@pytest.mark.parametrize("r,base", [(64, 10000.0), (128, 1e6), (2, 10000.0), (256, 5e5)])
def test_rope_steps(scaling, f, ctx, r, base):
    if scaling == "ntk" and r < 4:
        pytest.skip("R / (R - 2)")
    steps, factor = nqp.rope_steps(r, base, scaling, f, ctx, device="cpu")
    freq, want = oc.rope_frequencies(r, base, scaling, f, ctx)
    got = steps.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    # both sides round a few times in 53 bits
    assert np.all(np.abs(got - freq / (2 * math.pi)) <= 2.0 ** -48 * freq + 2.0 ** -64)
    assert abs(factor - want) <= 1e-6


def test_rope_steps_refusals():
    bad = [dict(rotary_dim=0), dict(rotary_dim=63), dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, base=float("nan")),
           dict(rotary_dim=64, scaling="linear", scale_factor=0.5),
           dict(rotary_dim=64, scaling="ntk", scale_factor=float("inf")),
           dict(rotary_dim=64, scaling="yarn", scale_factor=2.0), dict(rotary_dim=2, scaling="ntk", scale_factor=2.0)]
    for kw in bad:
        with pytest.raises(nqp.NQError) as e:
            nqp.rope_steps(device="cpu", **kw)
        assert e.value.code == nqp.EINVAL, kw
    with pytest.raises(ValueError):
        nqp.rope_steps(64, scaling="other", device="cpu")
    buf, fac = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    for scaling in (-1, 4):
        assert nqp.lib().nq_rope_steps(64, 10000.0, scaling, 1.0, 0.0, buf, ctypes.addressof(fac)) == nqp.EINVAL
    assert nqp.lib().nq_rope_steps(64, 10000.0, 0, 1.0, 0.0, None, ctypes.addressof(fac)) == nqp.EINVAL


# ---------------------------------------------------------------- refusals (nothing is launched)
P = 4096          # an aligned address that no refused call touches


def _rope(**kw):
    a = dict(x=P, out=P, dtype=0, tokens=4, heads=2, dim=64, rot=64, xt=128, xh=64, ot=128, oh=64, pos=P, steps=P,
             layout=0, factor=1.0, adjoint=0)
    a.update(kw)
    return nqp.lib().nq_rope(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), nqp.EINVAL), (dict(tokens=1 << 31), nqp.EINVAL), (dict(heads=0), nqp.EINVAL),
    (dict(heads=65536), nqp.EINVAL), (dict(dim=0), nqp.EINVAL), (dict(dim=4097), nqp.EINVAL),
    (dict(rot=63), nqp.EINVAL), (dict(rot=66), nqp.EINVAL), (dict(rot=-2), nqp.EINVAL), (dict(dtype=2), nqp.EINVAL),
    (dict(layout=2), nqp.EINVAL), (dict(x=None), nqp.EINVAL), (dict(out=None), nqp.EINVAL), (dict(pos=None), nqp.EINVAL),
    (dict(steps=None), nqp.EINVAL), (dict(x=P + 4), nqp.EALIGN), (dict(out=P + 8), nqp.EALIGN),
    (dict(tokens=0, x=None), nqp.OK)])
def test_rope_refusals(kw, want):
    assert _rope(**kw) == want


def _cache(**kw):
    c = nqp._CacheStruct(P, P, P, P, 8, 2, 128, 8, 4)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(k_codes=None), nqp.EINVAL), (dict(v_scales=None), nqp.EINVAL), (dict(head_dim=96), nqp.EINVAL),
              (dict(k_bits=5), nqp.EINVAL), (dict(v_bits=16), nqp.EINVAL), (dict(kv_heads=0), nqp.EINVAL),
              (dict(pages=0), nqp.EINVAL), (dict(pages=(1 << 31) // 64), nqp.EINVAL), (dict(v_codes=P + 1), nqp.EALIGN)]


def _append(cache=None, **kw):
    a = dict(k=P, v=P, dtype=1, tokens=3, kt=256, kh=128, vt=256, vh=128, slots=P, q=P, qo=P, heads=4, qt=512, qh=128,
             ot=512, oh=128, pos=P, steps=P, rot=128, layout=0, factor=1.0)
    a.update(kw)
    cache = cache or _cache()          # held until the call returns: only its address is passed
    return nqp.lib().nq_cache_append(ctypes.addressof(cache), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), nqp.EINVAL), (dict(k=None), nqp.EINVAL), (dict(v=None), nqp.EINVAL), (dict(slots=None), nqp.EINVAL),
    (dict(q=None), nqp.EINVAL), (dict(qo=None), nqp.EINVAL), (dict(pos=None), nqp.EINVAL), (dict(rot=24), nqp.EINVAL),
    (dict(rot=144), nqp.EINVAL), (dict(layout=-1), nqp.EINVAL), (dict(dtype=5), nqp.EINVAL), (dict(heads=-1), nqp.EINVAL),
    (dict(k=P + 2), nqp.EALIGN), (dict(kt=257), nqp.EALIGN), (dict(vh=132), nqp.EALIGN), (dict(qh=4), nqp.EALIGN),
    (dict(oh=1), nqp.EALIGN), (dict(tokens=0, k=None), nqp.OK)])
def test_append_refusals(kw, want):
    assert _append(**kw) == want


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_refusals(kw, want):
    c = _cache(**kw)
    assert _append(c) == want
    assert nqp.lib().nq_cache_read(ctypes.addressof(c), P, 1, P, P, 0, None) == want
    assert _attention(c) == want
    assert nqp.lib().nq_cache_read(None, P, 1, P, P, 0, None) == nqp.EINVAL


def test_read_refusals():
    c = _cache()
    read = lambda *a: nqp.lib().nq_cache_read(ctypes.addressof(c), *a, None)  # noqa: E731
    assert read(P, -1, P, P, 0) == nqp.EINVAL and read(None, 1, P, P, 0) == nqp.EINVAL
    assert read(P, 1, None, P, 0) == nqp.EINVAL and read(P, 1, P, P, 7) == nqp.EINVAL
    assert read(P, 1, P + 8, P, 0) == nqp.EALIGN and read(None, 0, None, None, 0) == nqp.OK


def _attention(cache=None, **kw):
    a = dict(q=P, qt=512, qh=128, total=6, heads=4, table=P, stride=9, width=9, lengths=P, starts=P, tree=P, seqs=2,
             drafts=3, context=500, scale=0.1, out=P, lse=P, ws=P, bytes=0)
    a.update(kw)
    cache = cache or _cache()          # held until the call returns: only its address is passed
    return nqp.lib().nq_tree_attention(ctypes.addressof(cache), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(seqs=0), nqp.EINVAL), (dict(seqs=65536), nqp.EINVAL), (dict(drafts=0), nqp.EINVAL), (dict(drafts=65), nqp.EINVAL),
    (dict(heads=5), nqp.EINVAL), (dict(heads=1), nqp.EINVAL), (dict(total=-1), nqp.EINVAL), (dict(total=7), nqp.EINVAL),
    (dict(context=-1), nqp.EINVAL), (dict(width=-1), nqp.EINVAL), (dict(starts=None, total=5), nqp.EINVAL),
    (dict(q=None), nqp.EINVAL), (dict(table=None), nqp.EINVAL), (dict(lengths=None), nqp.EINVAL), (dict(out=None), nqp.EINVAL),
    (dict(q=P + 2), nqp.EALIGN), (dict(qt=516), nqp.EALIGN), (dict(out=P + 4), nqp.EALIGN), (dict(total=0, q=None), nqp.OK)])
def test_attention_refusals(kw, want):
    assert _attention(**kw) == want


def test_attention_workspace_refusals():
    n = ctypes.c_size_t()
    ws = nqp.lib().nq_tree_attention_workspace_bytes
    for a in [(0, 1, 1, 8, 8, 64, 100), (1, 65, 1, 8, 8, 64, 100), (1, 1, 1, 8, 3, 64, 100), (1, 1, 1, 8, 8, 80, 100),
              (1, 1, 2, 8, 8, 64, 100), (1, 1, 1, 8, 8, 64, -5)]:
        assert ws(*a, ctypes.byref(n)) == nqp.EINVAL, a
    assert ws(1, 1, 1, 8, 8, 64, 100, None) == nqp.EINVAL


def test_binding_refuses_wrong_tensors():
    import torch
    with pytest.raises(ValueError):
        nqp.KVCache(torch.zeros((2, 2, 64, 100), dtype=torch.uint8), torch.zeros((2, 2, 64, 2), dtype=torch.float16),
                    torch.zeros((2, 2, 64, 128), dtype=torch.uint8), torch.zeros((2, 2, 64, 2), dtype=torch.float16))
    c = nqp.KVCache.empty(2, 2, 128, device="cpu")
    k = torch.zeros((3, 2, 128))
    s = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        c.append(k, torch.zeros((3, 2, 64)), s)
    with pytest.raises(ValueError):
        c.append(k, k, s.long())
    with pytest.raises(ValueError):
        c.append(k, k, s, steps=torch.zeros(64, dtype=torch.int64))
    with pytest.raises(ValueError):
        c.append(k, k, s, q=torch.zeros((3, 4, 64)))
    with pytest.raises(TypeError):
        c.append(k.half(), k.half(), s)
    with pytest.raises(ValueError):
        c.read(s.long())
    with pytest.raises(ValueError):
        c.attention(k, torch.zeros((1, 4), dtype=torch.int32), s[:1])
    with pytest.raises(ValueError):
        nqp.rope(k, s, torch.zeros(32, dtype=torch.int64), out=k.double())
    with pytest.raises(ValueError):
        nqp.rope(k.transpose(1, 2), s, torch.zeros(32, dtype=torch.int64))


def test_attention_refuses_tables_whose_keys_pass_an_int():
    """Keys are counted in whole tiles of up to 128 in 32-bit integers: a table of
    2^31 - 64 keys would have passed them."""
    most = ((1 << 31) - 256) // 64
    assert most * 64 + 127 < 1 << 31 <= (most + 3) * 64 + 127
    for width in (most + 1, (1 << 31) // 64 - 1, (1 << 31) - 1):
        assert _attention(width=width, stride=width) == nqp.EINVAL


def test_binding_refuses_tensors_that_the_kernels_cannot_reach():
    """Host memory, or memory of another device than the cache's."""
    import torch
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x, steps = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(32, dtype=torch.int64)
    c = nqp.KVCache.empty(2, 2, 64, device="cpu")
    far = nqp.KVCache.empty(2, 2, 64, device="meta")
    calls = [lambda: nqp.rope(x, i(3), steps), lambda: nqp.rope(x.to("meta"), i(3), steps), lambda: c.append(x, x, i(3)),
             lambda: c.append(x, x, i(3), q=x, positions=i(3), steps=steps), lambda: far.append(x, x, i(3)),
             lambda: c.read(i(3)), lambda: c.attention(x, i(1, 1), i(1)), lambda: c.attention(x, i(1, 1).to("meta"), i(1))]
    for k, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k}")
    with pytest.raises(ValueError):
        nqp.KVCache(c.k_codes, c.k_scales, far.v_codes, far.v_scales)


@pytest.mark.parametrize("length", [60, 900])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_the_bars_of_the_attention_see_a_lost_half(length, dim):
    """Outputs that cancel, with the probabilities rounded in numpy: the formats of
    the kernels pass, one bf16 alone does not."""
    def bf16(x):
        b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
        return ((b + ((b >> 16 & 1) + 0x7FFF)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)
    rng = np.random.default_rng(17)
    hq, hkv, t = 10, 2, length + 2
    k, v = (oc.values(rng.integers(-128, 128, (t, hkv, dim)).astype(np.int8),
                      (rng.uniform(0.3, 2.0, (t, hkv, dim // 64)) / 127).astype(np.float16)) for _ in range(2))
    v[1::2] = -v[:-1:2]
    q = bf16(rng.standard_normal((2, hq, dim)) * 2.0 ** -4)
    seen = np.tril(np.ones((2, t), bool), length)
    fp16 = lambda x: x.astype(np.float16).astype(np.float64)  # noqa: E731
    hi_lo = lambda x: bf16(x) + bf16(x - bf16(x))  # noqa: E731
    for many, good in ((False, hi_lo), (True, fp16)):
        o, most, rms = attention_products_bar(many, q, k, v, dim ** -0.5, seen)
        for held, passes in ((good, True), (bf16, False)):
            got = np.zeros_like(o)
            for i in range(2):
                for h in range(hq):
                    x = np.where(seen[i], k[:, h // 5] @ q[i, h] * dim ** -0.5, -np.inf)
                    p = np.exp(x - x.max())
                    vv = fp16(v[:, h // 5]) if many else v[:, h // 5]
                    got[i, h] = held(p) @ vv / p.sum()
            err = np.abs(bf16(got) - o)
            assert (np.all(err <= most) and np.sqrt(np.mean(err ** 2)) <= rms) == passes, (many, passes)
