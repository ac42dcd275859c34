"""GPU tests of rotary positions and of the paged cache against the formulas in 64 bits.

Tolerances.  A value stored in a type t is off by at most half a step,
h(t) = torch.finfo(t).eps / 2 relative (2^-8 bf16, 2^-24 fp32).  The rotation works in
fp32: two products and a sum of rounded cosines and sines (each within 2^-22 of its
value's scale 1), so before the store |y - y_exact| <= 2^-20 m (|x_a| + |x_b|).
Quantised codes are compared exactly: the same fp32 division and rounding to nearest
even on the host.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_attention_token_dsa_b200 import binding
    return binding


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def turned(x, pos, freq, offset, interleaved, sign, m):
    """The formula in 64 bits on the host; x [tokens, heads, dim] float64."""
    y = x.clone()
    r = 2 * len(freq)
    t = pos.double()[:, None, None] * freq.double()
    c, s = m * torch.cos(t), sign * m * torch.sin(t)
    i = torch.arange(len(freq))
    a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + i + r // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    bound = torch.zeros_like(x)
    bound[..., a] = bound[..., b] = abs(m) * (x[..., a].abs() + x[..., b].abs())
    return y, bound


def near(got, want, scale, dtype):
    half = torch.finfo(dtype).eps / 2
    err = (got.double().cpu() - want).abs()
    allowed = half * want.abs() * 1.001 + 2.0 ** -20 * scale
    assert bool((err <= allowed).all()), float((err - allowed).max())


# tokens, heads, dim, offset, rot: indexer and MLA shapes, one token, one head, odd sizes
# and parts that are not aligned to 16 bytes
SHAPES = [(1, 1, 128, 0, 64), (33, 64, 128, 0, 64), (5, 16, 576, 512, 64), (1000, 1, 128, 0, 128),
          (7, 3, 64, 0, 64), (3, 5, 50, 3, 20), (2, 2, 2, 0, 2), (9, 128, 192, 128, 64),
          (65, 1, 33, 1, 32), (2, 1, 1024, 512, 512), (1, 700, 72, 8, 48), (2, 90, 65536, 64, 64),
          (1, 65536, 64, 0, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(B, shape, dtype, interleaved):
    n, heads, dim, offset, rot = shape
    g = torch.Generator().manual_seed(sum(shape))
    x = torch.randn(n, heads, dim, generator=g).to(DT[dtype])
    pos = torch.randint(-5, 1 << 20, (n,), generator=g).to(torch.int32)
    freq = B.rope_frequencies(rot, scaling="yarn", factor=8.0)
    m = 1.2079
    for call, sign in ((B.rope, 1.0), (B.rope_backward, -1.0)):
        y = call(x.cuda(), pos.cuda(), freq, offset=offset, interleaved=interleaved, mscale=m)
        want, scale = turned(x.double(), pos, freq.cpu(), offset, interleaved, sign, m)
        near(y, want, scale, DT[dtype])
        keep = torch.ones(dim, dtype=torch.bool)
        keep[offset:offset + rot] = False
        assert torch.equal(y.cpu()[..., keep], x[..., keep])
        z = x.cuda()
        assert call(z, pos.cuda(), freq, offset=offset, interleaved=interleaved, mscale=m, out=z) is z
        assert torch.equal(z, y)


def test_rope_far_positions(B):
    """The last position of int32: the angle keeps its digits."""
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 123456789, 0], dtype=torch.int32)
    x = torch.ones(4, 2, 64)
    freq = B.rope_frequencies(64)
    y = B.rope(x.cuda(), pos.cuda(), freq)
    want, scale = turned(x.double(), pos, freq.cpu(), 0, False, 1.0, 1.0)
    near(y, want, scale, torch.float32)
    assert torch.equal(y[3].cpu(), x[3])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_cosines_and_sines(B, interleaved):
    """x = (1, 0) turned is (cos t, sin t): as the fp32 functions have them, which are off by at
    most one step, 2^-24 below 1, plus one rounding (2^-25).  Rounding the angle to 32 bits
    first adds up to pi 2^-25 (half a step of
    a fraction of a turn from 1/4 to 1/2 is 2^-26)."""
    g = torch.Generator().manual_seed(41)
    pos = torch.randint(0, 1 << 20, (4096,), generator=g).to(torch.int32)
    freq = B.rope_frequencies(64)
    x = torch.zeros(4096, 1, 64)
    first = slice(0, 64, 2) if interleaved else slice(0, 32)
    x[..., first] = 1.0
    want, _ = turned(x.double(), pos, freq.cpu(), 0, interleaved, 1.0, 1.0)
    y = B.rope(x.cuda(), pos.cuda(), freq, interleaved=interleaved).double().cpu()
    worst = float((y - want).abs().max())
    print("largest error:", worst, "=", worst * 2 ** 24, "steps")
    assert worst <= 1.55 * 2.0 ** -24
    # written to a cache as bf16: half a step of that, and the angle in 32 bits
    raw = torch.zeros(256, 16, 64, dtype=torch.bfloat16, device="cuda")
    B.cache_write(B.PagedCache(raw=raw), x[:, 0].cuda(), torch.arange(4096, device="cuda"), freq=freq,
                  pos=pos.cuda(), interleaved=interleaved)
    got = raw.view(4096, 64).double().cpu()
    assert bool(((got - want[:, 0]).abs() <= 2.0 ** -8 * want[:, 0].abs() * 1.001
                 + (1.55 + 3.1416 / 2) * 2.0 ** -24).all())


def test_rope_strides_and_surroundings(B):
    """A part of a wider buffer, heads before tokens, a broadcast input; what lies
    around the output stays as it was."""
    g = torch.Generator().manual_seed(3)
    freq = B.rope_frequencies(64)
    pos = torch.arange(6, dtype=torch.int32) * 1000
    wide = torch.randn(6, 4, 200, generator=g).bfloat16()
    for view in (lambda t: t[..., 40:168], lambda t: t[..., 41:169]):
        x = wide.cuda()
        out = torch.full((6, 4, 200), 7.0, dtype=torch.bfloat16, device="cuda")
        B.rope(view(x), pos.cuda(), freq, offset=32, out=view(out))
        want, scale = turned(view(wide).double(), pos, freq.cpu(), 32, False, 1.0, 1.0)
        near(view(out), want, scale, torch.bfloat16)
        around = torch.ones(200, dtype=torch.bool)
        view(around[None, None])[...] = False
        assert bool((out[..., around.cuda()] == 7.0).all())
    swapped = torch.randn(4, 6, 128, generator=g).cuda()
    y = B.rope(swapped.transpose(0, 1), pos.cuda(), freq, out=torch.empty_like(swapped).transpose(0, 1))
    want, scale = turned(swapped.transpose(0, 1).double().cpu(), pos, freq.cpu(), 0, False, 1.0, 1.0)
    near(y, want, scale, torch.float32)
    one = torch.randn(6, 1, 128, generator=g).cuda().expand(6, 4, 128)
    y = B.rope(one, pos.cuda(), freq)
    want, scale = turned(one.double().cpu(), pos, freq.cpu(), 0, False, 1.0, 1.0)
    near(y, want, scale, torch.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient_against_formula_and_differences(B, interleaved):
    """<dy, rope(x + e)> - <dy, rope(x - e)> over 2 e: rope is linear in x, so the
    difference quotient is exact up to the fp32 roundings of the two passes."""
    g = torch.Generator().manual_seed(4)
    n, heads, dim, offset, rot, m = 3, 2, 96, 32, 32, 1.37
    x, dy = torch.randn(n, heads, dim, generator=g), torch.randn(n, heads, dim, generator=g)
    pos = torch.tensor([1, 77, 4000], dtype=torch.int32)
    freq = B.rope_frequencies(rot)
    kw = dict(offset=offset, interleaved=interleaved, mscale=m)
    dx = B.rope_backward(dy.cuda(), pos.cuda(), freq, **kw).double().cpu()
    want, scale = turned(dy.double(), pos, freq.cpu(), offset, interleaved, -1.0, m)
    near(dx.float(), want, scale, torch.float32)
    for k in range(40):
        e = torch.zeros_like(x)
        at = tuple(int(torch.randint(0, s, (1,), generator=g)) for s in x.shape)
        e[at] = 1.0
        hi = B.rope((x + e).cuda(), pos.cuda(), freq, **kw).double().cpu()
        lo = B.rope((x - e).cuda(), pos.cuda(), freq, **kw).double().cpu()
        slope = float(((hi - lo) * dy.double()).sum() / 2)
        # x + e and x - e are rounded to fp32, then each output once: under 2^-18 here
        assert abs(slope - float(dx[at])) <= 2.0 ** -18 * (1 + float(dy.abs().sum()))


# ------------------------------------------------------------------- cache --

def e4m3(v):
    """Nearest e4m3 values of float64 v (finite), ties to even, saturating."""
    a = np.abs(v)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6)
    step = 2.0 ** (e - 3)
    return np.sign(v) * np.minimum(np.round(a / step) * step, 448.0)


def quantised(x, pow2):
    """x [rows, groups, 128] float32: (scale float32, code values), as documented."""
    amax = np.abs(x).max(-1)
    a = (amax / np.float32(448)).astype(np.float32)
    if pow2:
        m, e = np.frexp(amax)
        a = np.ldexp(np.float32(1), np.maximum(np.where(m > 0.875, e - 8, e - 9), -126))
    a = np.where(amax > 0, a, 1).astype(np.float32)
    return a, e4m3((x / a[..., None]).astype(np.float32).astype(np.float64))


FORMS = {"latent": (512, 64), "index": (128, 0), "bf16": (0, 576), "wide": (256, 200)}


def fresh(B, form, pages=6, page=16):
    """A cache inside wider blocks (a second layer beside it), filled with a mark."""
    dq, dr = FORMS[form]
    codes = scale = raw = None
    if dq:
        codes = torch.full((pages, 2, page, dq), 0x38, dtype=torch.uint8, device="cuda")
        codes = codes.view(torch.float8_e4m3fn)
        scale = torch.full((pages, 2, page, dq // 128), 3.0, device="cuda")
    if dr:
        raw = torch.full((pages, 2, page, dr), 5.0, dtype=torch.bfloat16, device="cuda")
    pick = lambda t: None if t is None else t[:, 1]  # noqa: E731
    return B.PagedCache(pick(codes), pick(scale), pick(raw)), (codes, scale, raw)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("n,stride", [(1, 0), (37, 0), (37, 3), (64, 8)])
def test_write_and_read_back(B, form, dtype, pow2, n, stride):
    dq, dr = FORMS[form]
    cache, whole = fresh(B, form)
    g = torch.Generator().manual_seed(n + stride + dq)
    x = (torch.randn(n, dq + dr + stride, generator=g) * torch.exp2(
        torch.randint(-12, 12, (n, 1), generator=g).float())).to(DT[dtype])
    if n > 5:
        x[-1] = 0.0                    # an all-zero row
        x[-2] = 448.0                  # on the border between two powers
        x[-3, ::2] = 449.5
    x = x[:, :dq + dr]
    order = torch.randperm(96, generator=g)[:n]
    slots = order.clone()
    skipped = min(n // 5, 7)
    slots[:skipped] = torch.tensor([-1, 96, -2 ** 40, 2 ** 40, 97, -96, 1 << 33])[:skipped]
    wide = torch.zeros(n, dq + dr + stride, dtype=DT[dtype], device="cuda")
    wide[:, :dq + dr] = x.cuda()
    B.cache_write(cache, wide[:, :dq + dr], slots.cuda(), pow2=pow2)
    live = slots[skipped:]
    xf = x[skipped:].float().numpy()
    untouched = torch.ones(96, dtype=torch.bool)
    untouched[live] = False
    if dq:
        codes = cache.codes.float().cpu().reshape(96, dq // 128, 128).numpy().astype(np.float64)
        scale = cache.scale.cpu().reshape(96, -1).numpy()
        a, want = quantised(xf[:, :dq].reshape(len(xf), -1, 128), pow2)
        assert np.array_equal(scale[live.numpy()], a)
        assert np.array_equal(codes[live.numpy()], want)
        assert np.all(codes[untouched.numpy()] == 1.0) and np.all(scale[untouched.numpy()] == 3.0)
        assert bool((whole[0].view(torch.uint8)[:, 0] == 0x38).all()) and bool((whole[1][:, 0] == 3.0).all())
        if pow2:
            assert np.array_equal(np.frexp(a)[0], np.full(a.shape, 0.5))
    if dr:
        raw = cache.raw.cpu().reshape(96, dr)
        assert torch.equal(raw[live], x[skipped:, dq:].to(torch.bfloat16))
        assert bool((raw[untouched] == 5.0).all()) and bool((whole[2][:, 0] == 5.0).all())

    # read back through a table that names the pages in no order, one of them twice
    table = torch.tensor([[5, 0, 3, 0], [1, 2, 4, 5]], dtype=torch.int32)
    rows = (table.long()[:, :, None] * 16 + torch.arange(16)).reshape(2, 64)
    for n_k, k_len in ((61, [61, 30]), (64, [0, 64]), (64, None), (1, [1, 1])):
        kl = None if k_len is None else torch.tensor(k_len, dtype=torch.int32).cuda()
        lens = [n_k, n_k] if k_len is None else [min(v, n_k) for v in k_len]
        for out_dtype in (torch.bfloat16, torch.float32):
            out = torch.full((2, n_k, dq + dr), 9.0, dtype=out_dtype, device="cuda")
            B.cache_read(cache, table.cuda(), n_k, kl, out=out)
            for b in range(2):
                parts = []
                r = rows[b, :lens[b]]
                if dq:
                    v = (codes[r.numpy()] * scale[r.numpy()][..., None].astype(np.float64)).reshape(len(r), dq)
                    parts.append(torch.from_numpy(v).float().to(out_dtype))
                if dr:
                    parts.append(raw[r].to(out_dtype))
                assert torch.equal(out[b, :lens[b]].cpu(), torch.cat(parts, 1))
                assert bool((out[b, lens[b]:] == 9.0).all())
        if not dr:
            c, s = B.cache_read_codes(cache, table.cuda(), n_k, kl)
            for b in range(2):
                r = rows[b, :lens[b]]
                assert np.array_equal(c[b, :lens[b]].float().cpu().numpy(), codes[r.numpy()].reshape(len(r), dq))
                assert np.array_equal(s[b, :lens[b]].cpu().numpy().reshape(len(r), dq // 128), scale[r.numpy()])
                assert bool((c[b, lens[b]:].view(torch.uint8) == 0).all()) and bool((s[b, lens[b]:] == 1).all())


def test_index_rows_equal_the_quantiser(B):
    """The index form holds exactly what dsa_quantize_e4m3 makes of the same rows."""
    x = torch.randn(50, 128, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    cache = B.PagedCache.empty(4, 16, 128, 0)
    B.cache_write(cache, x, torch.arange(50, device="cuda"))
    codes, scale = B.dsa_quantize_e4m3(x)
    assert torch.equal(cache.codes.view(torch.uint8).view(-1, 128)[:50], codes)
    assert torch.equal(cache.scale.view(-1)[:50], scale)


@pytest.mark.parametrize("pow2", [False, True])
def test_write_of_values_at_the_ends(B, pow2):
    """Largest and smallest magnitudes, infinities and NaN: a NaN stays one in its own
    place, an infinity reads back as one (power of two) and no other row changes."""
    x = torch.zeros(6, 128)
    x[0] = torch.linspace(-1, 1, 128) * 3.0e38
    x[1] = torch.linspace(-1, 1, 128) * 1e-35
    x[2, 5] = float("nan")
    x[2, 6] = 2.0
    x[3, 7] = float("inf")
    x[4] = 1.0
    x[5, 0] = 2.0 ** -140
    cache = B.PagedCache.empty(1, 16, 128, 0)
    B.cache_write(cache, x.cuda(), torch.arange(6, device="cuda"), pow2=pow2)
    y = B.cache_read(cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 6,
                     dtype=torch.float32)[0].cpu()
    amax = x[:2].abs().amax(1, keepdim=True)
    # e4m3 keeps 4 bits of a value over 2^-6 / 448 of the largest; below, steps of 2^-9 scales
    assert bool(((y[:2] - x[:2]).abs() <= x[:2].abs() * 2.0 ** -4 + amax * 2.0 ** -17).all())
    assert bool(torch.isnan(y[2, 5])) and float(y[2, 6]) == 2.0 and int(torch.isnan(y[2]).sum()) == 1
    if pow2:
        assert float(y[3, 7]) == float("inf") and int((y[3] != 0).sum()) == 1
    assert bool((y[4] == 1.0).all()) and bool(torch.isfinite(y[5]).all())


@pytest.mark.parametrize("pow2", [False, True])
def test_write_of_groups_whose_scale_would_be_zero(B, pow2):
    """amax / 448 rounds to 0 below 2^-141: the scale is then 1, so zeros stay zeros; the
    quantiser holds the same."""
    x = torch.zeros(4, 128)
    for r, power in enumerate((-149, -142, -141, -140)):
        x[r, 3], x[r, 7] = 2.0 ** power, -2.0 ** power
    cache = B.PagedCache.empty(1, 16, 128, 0)
    B.cache_write(cache, x.cuda(), torch.arange(4, device="cuda"), pow2=pow2)
    y = B.cache_read(cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 4,
                     dtype=torch.float32)[0].cpu()
    scale = cache.scale[0, :4, 0].cpu()
    assert bool((scale > 0).all())
    if pow2:                            # 2^-126 is the least: all of these are under its 2^-10
        assert bool((scale == 2.0 ** -126).all()) and bool((y == 0).all())
        return
    assert scale.tolist() == [1.0, 1.0, 2.0 ** -149, 2.0 ** -149]
    assert bool((y[:2] == 0).all()) and torch.equal(y[2], x[2])
    assert bool((y[3, [0, 1, 2, 4, 5, 6]] == 0).all()) and bool(torch.isfinite(y[3]).all())
    codes, sc = B.dsa_quantize_e4m3(x.cuda())
    assert torch.equal(codes.cpu(), cache.codes.view(torch.uint8)[0, :4].cpu())
    assert torch.equal(sc.cpu(), scale)


@pytest.mark.parametrize("form,offset,rot", [("latent", 512, 64), ("bf16", 512, 64), ("index", 0, 64),
                                             ("latent", 448, 128), ("wide", 248, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_write_rotated(B, form, offset, rot, interleaved):
    """The rotation inside the write equals the formula rounded once."""
    dq, dr = FORMS[form]
    cache, _ = fresh(B, form)
    g = torch.Generator().manual_seed(rot + offset)
    n, m = 29, 0.83
    x = torch.randn(n, dq + dr, generator=g).bfloat16()
    pos = torch.randint(0, 1 << 18, (n,), generator=g).to(torch.int32)
    freq = B.rope_frequencies(rot)
    slots = torch.randperm(96, generator=g)[:n]
    B.cache_write(cache, x.cuda(), slots.cuda(), pow2=True, freq=freq, pos=pos.cuda(), offset=offset,
                  interleaved=interleaved, mscale=m)
    want, scale = turned(x.double()[:, None], pos, freq.cpu(), offset, interleaved, 1.0, m)
    want, scale = want[:, 0], scale[:, 0]
    if dr:
        near(cache.raw.reshape(96, dr)[slots.cuda()], want[:, dq:], scale[:, dq:], torch.bfloat16)
    if dq:
        a = cache.scale.reshape(96, -1).cpu()[slots].repeat_interleave(128, 1)
        got = cache.codes.float().cpu().reshape(96, dq)[slots] * a
        # half a step of e4m3 (2^-4 relative, 2^-10 of the scale in its subnormal range)
        err = (got.double() - want[:, :dq]).abs()
        assert bool((err <= want[:, :dq].abs() * 2.0 ** -4 + a.double() * 2.0 ** -10
                     + 2.0 ** -20 * scale[:, :dq]).all())


def test_pages_outside_the_cache(B):
    """Table entries that name no page are not followed: their rows read as zeros, and
    entries behind the length are not looked at."""
    cache, _ = fresh(B, "latent")
    table = torch.tensor([[1, -1, 6, 2 ** 31 - 1], [0, -2 ** 31, -7, 99]], dtype=torch.int32).cuda()
    out = B.cache_read(cache, table, 64, torch.tensor([64, 16], dtype=torch.int32).cuda())
    assert bool((out[0, 16:] == 0).all()) and bool((out[1, 16:] == 0).all())
    assert bool((out[:, :16, 512:] == 5.0).all()) and bool((out[:, :16, :512] == 3.0).all())
    keys, _ = fresh(B, "index")
    c, s = B.cache_read_codes(keys, table, 64)
    assert bool((c.float()[0, 16:] == 0).all()) and bool((s[:, 16:] == 1.0).all())


def test_offsets_past_32_bits(B):
    """A page more than 2^31 elements from the start of its plane."""
    pages, page = 4200, 1024
    raw = torch.empty((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    cache = B.PagedCache(raw=raw)
    x = torch.randn(3, 576, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    slots = torch.tensor([pages * page - 1, pages * page - 500, 2], device="cuda")
    B.cache_write(cache, x, slots)
    assert torch.equal(raw[-1, -1], x[0]) and torch.equal(raw[0, 2], x[2])
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    out = B.cache_read(cache, table, page)
    assert torch.equal(out[0, page - 1], x[0]) and torch.equal(out[0, page - 500], x[1])


def test_reading_no_positions(B):
    """n_k = 0, with and without pages in the table: empty rows, nothing refused (an empty
    tensor has no address)."""
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for pages in (3, 0):
        table = torch.zeros(2, pages, dtype=torch.int32, device="cuda")
        for form in FORMS:
            cache, _ = fresh(B, form)
            width = sum(FORMS[form])
            for dtype in (torch.bfloat16, torch.float32):
                assert B.cache_read(cache, table, 0, lens, dtype=dtype).shape == (2, 0, width)
        cache, _ = fresh(B, "index")
        codes, scale = B.cache_read_codes(cache, table, 0, lens)
        assert codes.shape == (2, 0, 128) and scale.shape == (2, 0)
    torch.cuda.synchronize()


def test_streams_and_graphs(B):
    """Another stream, and a captured call replayed on new inputs."""
    g = torch.Generator().manual_seed(5)
    freq = B.rope_frequencies(64)
    x = torch.randn(16, 576, generator=g).bfloat16().cuda()
    pos = torch.arange(16, dtype=torch.int32).cuda()
    slots = torch.arange(16).cuda()
    table = torch.zeros(1, 1, dtype=torch.int32).cuda()

    def step(cache, stream=None):
        B.cache_write(cache, x, slots, pow2=True, freq=freq, pos=pos, offset=512, interleaved=True,
                      stream=stream)
        return B.cache_read(cache, table, 16, stream=stream)

    plain = step(B.PagedCache.empty(1, 16, 512, 64)).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = B.PagedCache.empty(1, 16, 512, 64)
    torch.cuda.synchronize()
    got = step(other, side)
    side.synchronize()
    assert torch.equal(got, plain)
    cache = B.PagedCache.empty(1, 16, 512, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache)
    new = torch.randn(16, 576, generator=g).bfloat16().cuda()
    x.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    captured = out.clone()
    assert torch.equal(captured, step(B.PagedCache.empty(1, 16, 512, 64)))
    assert not torch.equal(captured, plain)


def test_binding_refusals(B):
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    freq = B.rope_frequencies(64)
    for bad in (dict(x=x.half()), dict(pos=pos.long()), dict(freq=freq.float())):
        with pytest.raises(TypeError):
            B.rope(**{**dict(x=x, pos=pos, freq=freq), **bad})
    for bad in (dict(x=x[0]), dict(pos=pos[:3]), dict(x=x.transpose(1, 2)), dict(pos=pos.cpu()),
                dict(out=x[:2])):
        with pytest.raises(ValueError):
            B.rope(**{**dict(x=x, pos=pos, freq=freq), **bad})
    with pytest.raises(B.DsaError):
        B.rope(x, pos, freq, offset=80)
    with pytest.raises(B.DsaError):           # an output whose places coincide
        B.rope(x, pos, freq, out=x[:, :1].expand(4, 8, 128))
    cache = B.PagedCache.empty(2, 16, 512, 64)
    rows = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        B.cache_write(cache, rows, slots.int())
    for bad in (dict(x=rows[:, :512]), dict(slots=slots[:2]), dict(freq=freq), dict(pos=pos)):
        with pytest.raises(ValueError):
            B.cache_write(**{**dict(cache=cache, x=rows, slots=slots), **bad})
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(B.DsaError):
        B.cache_read(cache, table, 33)
    with pytest.raises(B.DsaError):
        B.cache_read_codes(cache, table, 16)
    with pytest.raises(ValueError):
        B.cache_read(cache, table, 16, k_len=pos)
    with pytest.raises(ValueError):
        B.PagedCache(cache.codes, cache.scale[:1], cache.raw)
    with pytest.raises(ValueError):
        B.PagedCache(cache.codes[:, ::2], cache.scale[:, ::2], cache.raw[:, ::2])
