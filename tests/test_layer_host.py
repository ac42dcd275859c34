"""Host-side checks of the cached-layer calls: frequency tables against the formula,
and every refusal before a launch.  CPU only; the fake pointers are never followed."""
import ctypes as C
import math

import pytest

FAKE = 0x10000


@pytest.fixture(scope="module")
def B():
    from sparse_attention_token_dsa_b200 import build
    build.build()
    from sparse_attention_token_dsa_b200 import binding
    return binding


# ------------------------------------------------------------- frequencies --

def test_plain_and_linear_frequencies(B):
    f = B.rope_frequencies(64, device="cpu")
    g = B.rope_frequencies(64, scaling="linear", factor=8.0, device="cpu")
    for i in range(32):
        want = 10000.0 ** (-2 * i / 64)
        assert abs(f[i].item() - want) <= 1e-15 * want
        assert abs(g[i].item() - want / 8) <= 1e-15 * want


@pytest.mark.parametrize("rot,base,factor,original", [(64, 10000.0, 40.0, 4096), (128, 5e5, 8.0, 8192),
                                                      (16, 10000.0, 2.0, 64), (2, 10000.0, 4.0, 4096)])
def test_yarn_frequencies(B, rot, base, factor, original):
    """Fast pairs (over 32 turns in the trained length) keep their frequency, slow ones
    (under one turn) are divided by the factor, those between are blended linearly."""
    f = B.rope_frequencies(rot, base, "yarn", factor, original, device="cpu").tolist()
    lo = math.floor(rot * math.log(original / (32 * 2 * math.pi)) / (2 * math.log(base)))
    hi = math.ceil(rot * math.log(original / (2 * math.pi)) / (2 * math.log(base)))
    lo, hi = max(lo, 0), min(hi, rot - 1)
    for i, got in enumerate(f):
        plain = base ** (-2 * i / rot)
        share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        want = plain / factor * share + plain * (1 - share)
        assert abs(got - want) <= 4e-15 * want
        turns = original * plain / (2 * math.pi)
        if i <= lo:
            assert got == plain
        if i >= hi:
            assert abs(got - plain / factor) <= 1e-15 * plain and turns < 32


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=514), dict(base=1.0),
                                dict(base=float("inf")), dict(scaling="linear", factor=0.0),
                                dict(scaling="yarn", factor=float("nan")),
                                dict(scaling="yarn", factor=2.0, original_len=0)])
def test_frequency_refusals(B, kw):
    args = dict(rot_dim=64)
    args.update(kw)
    with pytest.raises(B.DsaError):
        B.rope_frequencies(device="cpu", **args)


def test_frequency_scaling_name(B):
    with pytest.raises(ValueError):
        B.rope_frequencies(64, scaling="other", device="cpu")


# ------------------------------------------------------------------- rope --

def rope_problem(B, **kw):
    d = dict(n_tokens=4, heads=8, dim=128, offset=0, rot_dim=64, dtype=B.DSA_BF16, mscale=1.0,
             x_token_stride=1024, x_head_stride=128, out_token_stride=1024, out_head_stride=128,
             flags=0)
    d.update(kw)
    return B.DsaRopeProblem(**d)


def rope(B, p, x=FAKE, pos=FAKE, freq=FAKE, out=2 * FAKE):
    return B.lib.dsa_rope(None if p is None else C.byref(p), x, pos, freq, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_tokens=-1), -1), (dict(heads=0), -1), (dict(dim=0), -1), (dict(offset=-8), -1),
    (dict(rot_dim=0), -1), (dict(rot_dim=63), -2), (dict(rot_dim=514, dim=1024), -2),
    (dict(offset=72), -1), (dict(dtype=2), -2), (dict(dtype=9), -2), (dict(mscale=float("nan")), -1),
    (dict(mscale=float("inf")), -1), (dict(dim=65537), -2), (dict(heads=65537), -2),
    # an output whose places coincide
    (dict(out_head_stride=0), -1), (dict(out_token_stride=0), -1), (dict(out_head_stride=127), -1),
    (dict(out_token_stride=1023), -1), (dict(out_token_stride=-1024), -1),
    (dict(offset=2 ** 31 - 64), -1),
    # more units of a token than 32 bits count
    (dict(heads=65536, dim=65536, out_head_stride=65536, out_token_stride=1 << 33,
          x_head_stride=65535, x_token_stride=1 << 33), -2)])
def test_rope_problem_refusals(B, kw, status):
    assert rope(B, rope_problem(B, **kw)) == status


def test_rope_pointer_refusals(B):
    p = rope_problem(B)
    assert rope(B, None) == -1
    for name in ("x", "pos", "freq", "out"):
        assert rope(B, p, **{name: None}) == -1
    assert rope(B, p, x=FAKE + 1) == -1 and rope(B, p, out=FAKE + 1) == -1
    assert rope(B, p, pos=FAKE + 2) == -1 and rope(B, p, freq=FAKE + 4) == -1
    # in place needs the same strides
    assert rope(B, rope_problem(B, x_token_stride=2048), out=FAKE) == -1
    # no tokens: nothing to do, nothing looked at
    assert rope(B, rope_problem(B, n_tokens=0), x=None, pos=None, freq=None, out=None) == 0


# ------------------------------------------------------------------ cache --

def cache(B, **kw):
    d = dict(n_pages=4, page_size=64, dim_q=512, dim_raw=64, codes=FAKE, scale=FAKE, raw=FAKE,
             codes_page_stride=64 * 512, scale_page_stride=64 * 4, raw_page_stride=64 * 64)
    d.update(kw)
    return B.DsaCache(**d)


BAD_CACHES = [
    (dict(n_pages=0), -1), (dict(dim_q=-128), -1), (dict(dim_raw=-8), -1),
    (dict(dim_q=0, dim_raw=0, codes=None, scale=None, raw=None), -1), (dict(page_size=8), -2),
    (dict(page_size=48), -2), (dict(page_size=8192), -2), (dict(page_size=0), -2),
    (dict(dim_q=100), -2), (dict(dim_raw=60), -2), (dict(dim_q=8192), -2), (dict(codes=None), -1),
    (dict(scale=None), -1), (dict(raw=None), -1), (dict(codes=FAKE + 8), -1),
    (dict(scale=FAKE + 2), -1), (dict(raw=FAKE + 8), -1), (dict(codes_page_stride=64 * 512 + 8), -1),
    (dict(codes_page_stride=63 * 512), -1), (dict(scale_page_stride=64 * 4 - 1), -1),
    (dict(raw_page_stride=64 * 64 + 4), -1), (dict(raw_page_stride=0), -1),
    (dict(dim_q=0), -1), (dict(dim_raw=0), -1)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refusals(B, kw, status):
    c = cache(B, **kw)
    w = B.lib.dsa_cache_write(C.byref(c), FAKE, B.DSA_BF16, 576, 4, FAKE, None, None, None, 0, None)
    r = B.lib.dsa_cache_read(C.byref(c), FAKE, 1, 4, 100, None, FAKE, B.DSA_BF16, None)
    assert w == status and r == status


def test_cache_write_refusals(B):
    c = cache(B)

    def call(x=FAKE, dtype=1, stride=576, n=4, slots=FAKE, turn=None, pos=None, freq=None):
        return B.lib.dsa_cache_write(C.byref(c), x, dtype, stride, n, slots,
                                     None if turn is None else C.byref(turn), pos, freq, 0, None)

    assert B.lib.dsa_cache_write(None, FAKE, 1, 576, 4, FAKE, None, None, None, 0, None) == -1
    assert call(x=None) == -1 and call(slots=None) == -1 and call(n=-1) == -1
    assert call(stride=-1) == -1 and call(dtype=2) == -2 and call(x=FAKE + 1) == -1
    assert call(slots=FAKE + 4) == -1 and call(n=0, x=None, slots=None) == 0
    turn = rope_problem(B, offset=512, rot_dim=64)
    assert call(turn=turn) == -1 and call(turn=turn, pos=FAKE) == -1 and call(pos=FAKE) == -1
    for kw, status in [(dict(offset=516), -1), (dict(offset=508), -2), (dict(rot_dim=8), -2),
                       (dict(offset=520), -1), (dict(mscale=float("nan")), -1),
                       (dict(offset=-8), -1), (dict(offset=0, rot_dim=528), -2)]:
        t = rope_problem(B, **{**dict(offset=512, rot_dim=64), **kw})
        assert call(turn=t, pos=FAKE, freq=FAKE) == status, kw


def test_cache_read_refusals(B):
    c = cache(B)

    def call(table=FAKE, batch=1, pages=4, n_k=100, k_len=None, out=FAKE, dtype=1):
        return B.lib.dsa_cache_read(C.byref(c), table, batch, pages, n_k, k_len, out, dtype, None)

    assert call(table=None) == -1 and call(out=None) == -1 and call(batch=0) == -1
    assert call(n_k=-1) == -1 and call(n_k=257) == -1 and call(pages=1) == -1
    assert call(out=FAKE + 8) == -1 and call(dtype=2) == -2 and call(k_len=FAKE + 1) == -1
    assert call(table=FAKE + 2) == -1 and call(n_k=0) == 0
    codes = B.lib.dsa_cache_read_codes
    assert codes(C.byref(c), FAKE, 1, 4, 100, None, FAKE, FAKE, None) == -2      # dim_raw
    k = cache(B, dim_q=128, dim_raw=0, raw=None, raw_page_stride=0, codes_page_stride=64 * 128)
    assert codes(C.byref(k), FAKE, 1, 4, 100, None, FAKE, None, None) == -1
    latent = cache(B, dim_q=0, dim_raw=576, codes=None, scale=None, raw_page_stride=64 * 576)
    assert codes(C.byref(latent), FAKE, 1, 4, 100, None, FAKE, FAKE, None) == -1


def test_reading_no_positions(B):
    """n_k = 0: nothing to do and nothing looked at (an empty tensor has no address); what is
    wrong with the call otherwise is still refused."""
    index = cache(B, dim_q=128, dim_raw=0, raw=None, raw_page_stride=0, codes_page_stride=64 * 128)
    read, codes = B.lib.dsa_cache_read, B.lib.dsa_cache_read_codes
    for pages in (4, 0):
        for c in (cache(B), index):
            for dtype in (B.DSA_BF16, B.DSA_F32):
                assert read(C.byref(c), None, 2, pages, 0, None, None, dtype, None) == 0
        assert codes(C.byref(index), None, 2, pages, 0, None, None, None, None) == 0
    c = cache(B)
    assert read(C.byref(c), None, 0, 4, 0, None, None, B.DSA_BF16, None) == -1
    assert read(C.byref(c), None, 1, 4, 0, None, None, 2, None) == -2
    assert codes(C.byref(c), None, 1, 4, 0, None, None, None, None) == -2


def test_binding_refuses_host_tensors(B):
    import torch
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.rope(x, pos, B.rope_frequencies(64, device="cpu"))
    with pytest.raises(ValueError):
        B.PagedCache(raw=torch.zeros(2, 64, 576, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        B.PagedCache()
    with pytest.raises(TypeError):
        B.PagedCache(raw=[1, 2])


def test_arrivals_that_announce_shared_memory_release():
    """No run can show a missing release between two CTAs, so the source is read: relaxed
    arrivals on the pair's barriers announce TMEM alone, every other one goes through
    pair_publish (a release of shared memory), and pair_acquire stands between each wait of
    the matrix warps for such a barrier and the products."""
    import os
    import re
    from sparse_attention_token_dsa_b200 import build
    text = open(os.path.join(build.CSRC, "paged_mla.cuh")).read()
    relaxed = re.findall(r"mbar_arrive_cluster\((\w+)", text)
    assert sorted(relaxed) == ["o_empty", "s_empty"]
    assert sorted(re.findall(r"pair_publish\((\w+)", text)) == ["bar", "k_ready", "k_ready", "p_full",
                                                               "q_ready", "v_ready"]
    assert sorted(re.findall(r"ready\((\w+) \+ \w+ \* 8\);", text)) == ["k_ready", "v_ready"]   # codes
    waits = [m.start() for m in re.finditer(r"wait_(?:pair|seen)\((?:seen, )?&T->(?:q_ready|k_ready|p_full|v_ready)",
                                            text)]
    assert len(waits) == 4
    for at in waits:
        assert 0 < text.index("pair_acquire()", at) < text.index("pair_mma_bf16(", at)
    pair = open(os.path.join(build.CSRC, "pair.cuh")).read()
    publish = pair[pair.index("void pair_publish"):pair.index("void pair_acquire")]
    assert publish.index("fence.release.sync_restrict::shared::cta.cluster") < publish.index("mbar_arrive_cluster(")
