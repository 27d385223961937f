"""GPU checks of rotary positions and the quantised KV cache (written, read
back) against the fp64 oracle.

Bars.  Rotation: the angle (one int-to-fp32 conversion, one product, one
rounded constant: each half an ulp of at most pi) is off by at most 1.25 pi
2^-23, cosine and sine by 2 ulp more, the two products and the sum by 3 2^-24:
together below 1e-6 of factor (|a| + |b|); a bf16 result adds its rounding,
2^-8 of the value.  Codes and scales of unrotated inputs: exact.  Codes of
rotated keys: the value read back is within half a scale step (and what the
scale's FP16 rounding takes off the largest code) of the rotated key."""
import numpy as np
import pytest
import torch

import quantized_weight_decode_gb300 as nqp
import synth
from oracle import cache as oc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def built():
    nqp.build()
    nqp.lib()
    torch.cuda.set_device(0)
    assert nqp.last_device_error() == 0


def _steps(r, base=10000.0, scaling="plain", f=1.0, ctx=0.0):
    s, factor = nqp.rope_steps(r, base, scaling, f, ctx, device=DEV)
    return s, factor, s.cpu().numpy().view(np.uint64)


def _pair_bound(x, r, inter, factor):
    """1e-6 factor (|a| + |b|) of each rotated value, 0 for the others."""
    b = np.zeros_like(x)
    a = np.abs(x)
    if inter:
        s = a[..., 0:r:2] + a[..., 1:r:2]
        b[..., 0:r:2], b[..., 1:r:2] = s, s
    else:
        s = a[..., :r // 2] + a[..., r // 2:r]
        b[..., :r // 2], b[..., r // 2:r] = s, s
    return 1e-6 * factor * b


def _check_rope(x, y, pos, steps_np, r, inter, factor, adjoint):
    xs = x.double().cpu().numpy()
    want = oc.rope(xs, pos, steps_np, inter, factor, adjoint)
    tol = _pair_bound(xs, r, inter, factor)
    if y.dtype == torch.bfloat16:
        tol = tol * 1.01 + 2.0 ** -8 * np.abs(want)
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol + 1e-37), np.max(np.abs(got - want) - tol)
    assert torch.equal(x[..., r:], y[..., r:])             # what is not rotated passes


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,heads,dim,r", [
    (1, 1, 64, 64), (16, 48, 128, 128), (5, 3, 256, 64), (33, 7, 128, 32), (2, 1, 16, 16), (3, 5, 80, 48),
    (4, 3, 10, 6), (3, 2, 7, 4), (2, 3, 1, 0), (5, 2, 64, 0), (1, 2, 4096, 4096), (130, 2, 96, 24), (300, 1, 64, 64)])
def test_rope(tokens, heads, dim, r, dtype, inter):
    rng = synth.generator(0, 900, tokens, dim, r)
    x = torch.from_numpy(rng.standard_normal((tokens, heads, dim), dtype=np.float32)).to(DEV).to(dtype)
    pos = rng.integers(-5, 300000, tokens).astype(np.int32)
    pos[0] = (2 ** 31 - 1, -2 ** 31, 0)[tokens % 3]
    steps, factor, sn = _steps(r, scaling="yarn", f=4.0, ctx=8192.0) if r else (torch.zeros(0, dtype=torch.int64, device=DEV), 1.0, [])
    p = torch.from_numpy(pos).to(DEV)
    for adjoint in (False, True):
        y = nqp.rope(x, p, steps, layout=int(inter), factor=factor, adjoint=adjoint)
        if r:
            _check_rope(x, y, pos, sn, r, inter, factor, adjoint)
        else:
            assert torch.equal(x, y)
        z = x.clone()                                       # in place: the same bits
        assert nqp.rope(z, p, steps, out=z, layout=int(inter), factor=factor, adjoint=adjoint) is z
        assert torch.equal(y, z)
    assert nqp.last_device_error() == 0


def test_rope_strides_and_zero_tokens():
    steps, factor, sn = _steps(64)
    g = torch.Generator(device=DEV).manual_seed(5)
    rows = torch.randn((9, 20 * 64 + 3), device=DEV, generator=g)
    pos = torch.arange(100, 109, dtype=torch.int32, device=DEV)
    wide = torch.randn((9, 30, 64), device=DEV, generator=g)
    odd = rows[:, :20 * 64].unflatten(1, (20, 64))          # a token stride that is no multiple of 16 bytes
    swapped = torch.randn((6, 9, 64), device=DEV, generator=g).transpose(0, 1)
    for x in (wide[:, 4:24], odd, swapped, wide[:, :, :64][::2].contiguous()):
        n = x.shape[0]
        y = nqp.rope(x, pos[:n].contiguous(), steps)
        _check_rope(x, y, pos[:n].cpu().numpy(), sn, 64, False, 1.0, False)
        out = torch.full((n, x.shape[1] + 2, 64), 7.0, device=DEV)
        nqp.rope(x, pos[:n].contiguous(), steps, out=out[:, 1:-1])
        assert torch.equal(out[:, 1:-1], y) and bool((out[:, 0] == 7).all()) and bool((out[:, -1] == 7).all())
    assert nqp.rope(wide[:0], pos[:0], steps).shape == (0, 30, 64)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(inter):
    """The adjoint against the formula (<adjoint g, x> = <g, rope x>, and the
    oracle above) and against differences of the forward pass (a linear map:
    the difference quotient is exact up to rounding)."""
    steps, factor, _ = _steps(48, scaling="yarn", f=2.0, ctx=4096.0)
    gen = torch.Generator(device=DEV).manual_seed(9)
    x, g = (torch.randn((3, 2, 64), device=DEV, generator=gen) for _ in range(2))
    pos = torch.tensor([7, 123456, -3], dtype=torch.int32, device=DEV)
    gx = nqp.rope(g, pos, steps, layout=int(inter), factor=factor, adjoint=True)
    f = lambda v: float((nqp.rope(v, pos, steps, layout=int(inter), factor=factor).double() * g.double()).sum())  # noqa: E731
    assert abs(f(x) - float((gx.double() * x.double()).sum())) <= 1e-5 * float(g.norm() * x.norm())
    for t, h, i in [(0, 0, 0), (1, 1, 23), (1, 0, 24), (2, 1, 47), (0, 1, 63)]:
        d = torch.zeros_like(x)
        d[t, h, i] = 0.5
        assert abs(f(x + d) - f(x - d) - float(gx[t, h, i])) <= 4e-6 * float(g.norm() * x.norm())


def _make(pages, hkv, dim, kb, vb):
    c = nqp.KVCache.empty(pages, hkv, dim, kb, vb, DEV)
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xA5)
    for t in (c.k_scales, c.v_scales):
        t.fill_(float("nan"))
    return c


def _rows(t, slots):
    s = slots.long()
    return t[s // 64, :, s % 64].cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kb,vb", [(8, 8), (8, 4), (4, 8), (4, 4)])
@pytest.mark.parametrize("hkv,dim,tokens", [(1, 64, 1), (4, 128, 16), (2, 256, 70), (3, 64, 131), (16, 128, 7)])
def test_append_and_read_without_rotation(hkv, dim, tokens, kb, vb, dtype):
    gen = torch.Generator(device=DEV).manual_seed(tokens)
    pages = tokens // 64 + 3
    c = _make(pages, hkv, dim, kb, vb)
    k = torch.randn((tokens, hkv, dim), device=DEV, generator=gen).to(dtype)
    v = (torch.randn((tokens, hkv, dim), device=DEV, generator=gen) * 1e-3).to(dtype)
    k[..., 5] *= 30
    k[0, 0, :64] = 0                                        # a zero group
    v[-1, -1, -64:] = 1e-8                                  # a scale in FP16's subnormals, or 0
    slots = torch.randperm(pages * 64, device=DEV, generator=gen)[:tokens].to(torch.int32)
    before = [t.clone() for t in (c.k_codes, c.v_codes)]
    assert c.append(k, v, slots) is None
    rk, rv = c.read(slots, torch.float32)
    bk, bv = c.read(slots)
    for x, bits, codes, scales, got, half in ((k, kb, c.k_codes, c.k_scales, rk, bk), (v, vb, c.v_codes, c.v_scales, rv, bv)):
        want, ws = oc.quantise(x.float().cpu().numpy(), bits)
        assert np.array_equal(_rows(codes, slots), oc.pack_codes(want, bits))
        assert np.array_equal(_rows(scales, slots).view(np.uint16), ws.view(np.uint16))
        vals = oc.values(want, ws)
        assert np.array_equal(got.double().cpu().numpy(), vals)                     # exact in fp32
        assert torch.equal(half, got.to(torch.bfloat16))
    # nothing else was written
    other = torch.ones(pages * 64, dtype=torch.bool, device=DEV)
    other[slots.long()] = False
    rest = other.nonzero().flatten().to(torch.int32)
    for t, b in zip((c.k_codes, c.v_codes), before):
        assert np.array_equal(_rows(t, rest), _rows(b, rest))
    assert np.isnan(_rows(c.k_scales, rest)).all() and np.isnan(_rows(c.v_scales, rest)).all()
    assert nqp.last_device_error() == 0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,dim,r,tokens", [(40, 8, 128, 128, 16), (24, 4, 256, 64, 5), (1, 1, 64, 64, 300),
                                                 (6, 2, 128, 16, 65), (8, 8, 256, 256, 3), (5, 1, 64, 48, 1)])
def test_append_rotates_keys_and_queries(hq, hkv, dim, r, tokens, dtype, inter):
    gen = torch.Generator(device=DEV).manual_seed(r)
    c = _make(tokens // 64 + 2, hkv, dim, 8, 4)
    qkv = torch.randn((tokens, hq + 2 * hkv, dim), device=DEV, generator=gen).to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    slots = (torch.randperm(c.pages * 64, device=DEV, generator=gen)[:tokens]).to(torch.int32)
    steps, factor, sn = _steps(r, 1e6, "yarn", 4.0, 8192.0)
    pos = torch.arange(99990, 99990 + tokens, dtype=torch.int32, device=DEV)
    qo = c.append(k, v, slots, q=q, positions=pos, steps=steps, layout=int(inter), factor=factor)
    # the query as nq_rope rotates it (fp32 arithmetic, one rounding)
    ref = nqp.rope(q.float(), pos, steps, layout=int(inter), factor=factor)
    assert torch.equal(qo, ref.to(torch.bfloat16))
    _check_rope(q.float(), ref, pos.cpu().numpy(), sn, r, inter, factor, False)
    rk, rv = (t.double().cpu().numpy() for t in c.read(slots, torch.float32))
    kr = nqp.rope(k.float(), pos, steps, layout=int(inter), factor=factor).cpu().numpy()
    for got, x, bits, scales in ((rk, kr, 8, c.k_scales), (rv, v.float().cpu().numpy(), 4, c.v_scales)):
        want, ws = oc.quantise(x, bits)
        assert np.array_equal(got, oc.values(want, ws))
        step = np.repeat(_rows(scales, slots).astype(np.float64), 64, -1)
        assert np.all(np.abs(got - x) <= step * (0.5 + 2.0 ** -10 * (127 if bits == 8 else 7)))
    assert nqp.last_device_error() == 0


def test_append_strided_outputs_and_skipped_tokens():
    c = _make(3, 2, 64, 8, 8)
    gen = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn((6, h, 64), device=DEV, generator=gen) for h in (4, 2, 2))
    slots = torch.tensor([5, -1, 70, -7, 3, 191], dtype=torch.int32, device=DEV)
    buf = torch.full((6, 8, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    steps, factor, _ = _steps(64)
    pos = torch.arange(6, dtype=torch.int32, device=DEV)
    got = c.append(k, v, slots, q=q, q_out=buf[:, 2:6], positions=pos, steps=steps)
    assert got.data_ptr() == buf[:, 2:6].data_ptr()
    assert torch.equal(got, nqp.rope(q, pos, steps).to(torch.bfloat16))
    assert bool((buf[:, :2] == 9).all()) and bool((buf[:, 6:] == 9).all())
    assert int((~torch.isnan(c.k_scales)).sum()) == 4 * 2 and int((~torch.isnan(c.v_scales)).sum()) == 4 * 2
    rk, _ = c.read(slots, torch.float32)
    assert not bool(rk[1].any()) and not bool(rk[3].any())   # a negative slot reads as zeros
    # transposed inputs: the head stride larger than the token stride
    kt = torch.randn((2, 6, 64), device=DEV, generator=gen).transpose(0, 1)
    c.append(kt, v, slots)
    rk, _ = c.read(slots, torch.float32)
    want = oc.values(*oc.quantise(kt.cpu().numpy(), 8))
    assert np.array_equal(rk[[0, 2, 4, 5]].double().cpu().numpy(), want[[0, 2, 4, 5]])
    c.append(k[:0], v[:0], slots[:0])
    assert c.read(slots[:0])[0].shape == (0, 2, 64)
    assert nqp.last_device_error() == 0


def test_slots_beyond_the_cache_are_reported():
    c = _make(2, 1, 64, 8, 4)
    k = torch.ones((2, 1, 64), device=DEV)
    snap = [t.clone() for t in (c.k_codes, c.v_codes)]
    c.append(k, k, torch.tensor([128, 2 ** 31 - 1], dtype=torch.int32, device=DEV))
    assert nqp.last_device_error() == nqp.ERANGE and nqp.last_device_error() == 0
    assert torch.equal(c.k_codes, snap[0]) and torch.equal(c.v_codes, snap[1]) and bool(torch.isnan(c.k_scales).all())
    rk, rv = c.read(torch.tensor([128], dtype=torch.int32, device=DEV), torch.float32)
    assert not bool(rk.any()) and not bool(rv.any())
    assert nqp.last_device_error() == nqp.ERANGE


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_values_that_cannot_be_held_poison_their_group(bad):
    c = _make(1, 2, 128, 8, 4)
    k = torch.ones((3, 2, 128), device=DEV)
    v = torch.ones((3, 2, 128), device=DEV)
    k[1, 0, 70] = bad
    v[2, 1, 3] = bad
    slots = torch.arange(3, dtype=torch.int32, device=DEV)
    c.append(k, v, slots)
    assert nqp.last_device_error() == nqp.ERANGE
    rk, rv = c.read(slots, torch.float32)
    for got, (t, h, g) in ((rk, (1, 0, 1)), (rv, (2, 1, 0))):
        part = torch.zeros((3, 2, 2), dtype=torch.bool, device=DEV)
        part[t, h, g] = True
        part = part.repeat_interleave(64, -1)
        assert bool(torch.isnan(got[part]).all()) and bool(torch.isfinite(got[~part]).all())


def test_cache_beyond_four_gigabytes():
    """Rows whose byte offset passes 32 bits: the last pages of a large cache."""
    pages, hkv, dim = 36000, 8, 256                          # 4.7 GB of 8-bit codes
    c = nqp.KVCache.empty(pages, hkv, dim, 8, 4, DEV)
    assert c.k_codes.numel() > 2 ** 32
    gen = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn((4, hkv, dim), device=DEV, generator=gen)
    slots = torch.tensor([pages * 64 - 1, pages * 64 - 65, 64 * 20000 + 3, 0], dtype=torch.int32, device=DEV)
    c.append(k, -k, slots)
    rk, rv = (t.double().cpu().numpy() for t in c.read(slots, torch.float32))
    assert np.array_equal(rk, oc.values(*oc.quantise(k.cpu().numpy(), 8)))
    assert np.array_equal(rv, oc.values(*oc.quantise(-k.cpu().numpy(), 4)))
    assert int(c.k_codes.count_nonzero()) <= 4 * hkv * dim
    assert nqp.last_device_error() == 0


def test_on_another_stream():
    c = nqp.KVCache.empty(4, 2, 64, 8, 8, DEV)
    k = torch.randn((100, 2, 64), device=DEV)
    slots = torch.arange(100, dtype=torch.int32, device=DEV)
    steps, factor, _ = _steps(64)
    pos = torch.arange(100, dtype=torch.int32, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    a = torch.empty_like(k)
    nqp.rope(k, pos, steps, out=a, stream=st)
    c.append(k, k, slots, stream=st)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    c.read(slots, k_out=ko, v_out=vo, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(a, nqp.rope(k, pos, steps)) and torch.equal(ko, vo)
    assert np.array_equal(ko.double().cpu().numpy(), oc.values(*oc.quantise(k.cpu().numpy(), 8)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_outputs_on_sixteen_byte_boundaries(dtype):
    """Outputs that start 16 bytes into a 32-byte line."""
    c = nqp.KVCache.empty(2, 3, 64, 8, 4, DEV)
    k = torch.randn((70, 3, 64), device=DEV)
    slots = torch.arange(70, dtype=torch.int32, device=DEV)
    c.append(k, k, slots)
    want = c.read(slots, dtype)
    n, skip = 70 * 3 * 64, 16 // torch.empty(0, dtype=dtype).element_size()
    buf = torch.zeros((2, n + 2 * skip), dtype=dtype, device=DEV)
    ko, vo = (buf[i, skip:skip + n].view(70, 3, 64) for i in range(2))
    assert ko.data_ptr() % 32 == 16
    c.read(slots, k_out=ko, v_out=vo)
    assert torch.equal(ko, want[0]) and torch.equal(vo, want[1])
    assert not bool(buf[:, :skip].any()) and not bool(buf[:, skip + n:].any())
    # inputs and q_out too
    x = torch.zeros(2 * 70 * 3 * 64 + 2 * skip, dtype=dtype, device=DEV)
    kk = x[skip:skip + n].view(70, 3, 64)
    kk.copy_(k.to(dtype))
    c2 = nqp.KVCache.empty(2, 3, 64, 8, 4, DEV)
    q_out = torch.zeros(n + 8, dtype=torch.bfloat16, device=DEV)[8:].view(70, 3, 64)
    c2.append(kk, kk, slots, q=kk, q_out=q_out)
    assert torch.equal(q_out, kk.to(torch.bfloat16))
    c.append(k.to(dtype), k.to(dtype), slots)
    assert torch.equal(c2.k_codes, c.k_codes) and torch.equal(c2.v_codes, c.v_codes)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rope_in_a_graph_of_gradients(dtype, inter):
    """A result of a tensor that requires a gradient carries one: the adjoint's,
    bit for bit, for whatever layout the incoming gradient has, and its own
    gradient is the rotation again."""
    steps, factor, _ = _steps(48, scaling="yarn", f=2.0, ctx=4096.0)
    gen = torch.Generator(device=DEV).manual_seed(19)
    x, g = (torch.randn((5, 2, 64), device=DEV, generator=gen).to(dtype) for _ in range(2))
    pos = torch.tensor([7, 123456, -3, 0, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    kw = dict(layout=int(inter), factor=factor)
    want = nqp.rope(x, pos, steps, **kw)
    assert not want.requires_grad
    x.requires_grad_(True)
    for adjoint in (False, True):
        back = nqp.rope(g, pos, steps, adjoint=not adjoint, **kw)
        y = nqp.rope(x, pos, steps, adjoint=adjoint, **kw)
        assert y.requires_grad and (adjoint or torch.equal(y, want))
        gx, = torch.autograd.grad(y, x, g)
        assert gx.dtype == dtype and torch.equal(gx, back)
    y = nqp.rope(x, pos, steps, **kw)
    ones = nqp.rope(torch.ones_like(g), pos, steps, adjoint=True, **kw)
    assert torch.equal(torch.autograd.grad(y.sum(), x, retain_graph=True)[0], ones)      # one value, strides of 0
    wide = torch.zeros((5, 64, 2), dtype=dtype, device=DEV).transpose(1, 2)              # head_dim not contiguous
    wide.copy_(g)
    assert torch.equal(torch.autograd.grad(y, x, wide, retain_graph=True)[0], nqp.rope(g, pos, steps, adjoint=True, **kw))
    off = torch.zeros(5 * 2 * 64 + 1, dtype=dtype, device=DEV)[1:].view(5, 2, 64)        # off a 16-byte boundary
    off.copy_(g)
    assert torch.equal(torch.autograd.grad(y, x, off, retain_graph=True)[0], nqp.rope(g, pos, steps, adjoint=True, **kw))
    g.requires_grad_(True)
    gx, = torch.autograd.grad(y, x, g, create_graph=True)
    assert torch.equal(torch.autograd.grad(gx, g, x.detach())[0], want)
    with torch.no_grad():
        assert not nqp.rope(x, pos, steps, **kw).requires_grad
        z = x.detach().clone().requires_grad_(True)
        assert nqp.rope(z, pos, steps, out=z, **kw) is z and torch.equal(z, want)
    for out in (torch.empty_like(want), x):
        with pytest.raises(ValueError):
            nqp.rope(x, pos, steps, out=out, **kw)
    assert nqp.last_device_error() == 0
