"""GPU tests of latent attention over the paged cache against the formula in 64 bits.

Tolerances.  A logit is scale times a sum of 576 products (exact in fp32) taken in 36 steps
of 16 terms: 52 additions, each off by at most one step 2^-23 of the sum of magnitudes, so
    d = 52 2^-23 scale max_s sum |q| |kv_s| + 2^-20 (1 + max |x|)
bounds a logit's error in the exponent (the second term: one rounding of x log2 e and the
exponential's own error).  So |lse - exact| <= d + 2^-22 |lse|.  An output weighs values with
weights rounded to bf16 (half a step, 2^-8 relative) over an unrounded denominator, and is
rounded once itself: |o - exact| <= (2^-8 + 3 d) sum_s w_s |v_s| + 2^-8 |o| (1 + 2^-7).
"""
import ctypes as C

import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_attention_token_dsa_b200 import binding
    return binding


class Problem:
    """A cache whose pages lie between those of another layer, in no order; rows that no
    sequence holds are NaN, table entries behind a length name no page."""

    def __init__(self, B, seed, k_lens, q_lens, n_q, heads, page, form, spread=1.0, room=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        batch = len(k_lens)
        per = [-(-n // page) for n in k_lens]
        width = max(max(per), 1) + room
        n_pages = sum(per) + 2
        order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
        self.table = torch.full((batch, width), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        nan = float("nan")
        rows = torch.full((n_pages, page, 576), nan, device="cuda")
        used = 0
        for b, n in enumerate(k_lens):
            pages = order[used:used + per[b]]
            used += per[b]
            self.table[b, :per[b]] = pages
            if per[b] < width:
                self.table[b, per[b]] = -5
            live = torch.full((per[b] * page, 576), nan, device="cuda")
            live[:n] = torch.randn(n, 576, device="cuda", generator=g)
            rows[pages.long()] = live.view(-1, page, 576)
        codes = scale = raw = None
        if form == "bf16":
            raw = torch.full((n_pages, 2, page, 576), nan, device="cuda", dtype=torch.bfloat16)
            raw[:, 1] = rows.bfloat16()
            self.rows = raw[:, 1].double()
            raw = raw[:, 1]
        else:
            codes = torch.full((n_pages, 3, page, 512), 0x7f, device="cuda", dtype=torch.uint8)
            codes = codes.view(torch.float8_e4m3fn)
            # scales differ from group to group
            power = torch.randint(-9, -5, (n_pages, page, 4), device="cuda", generator=g)
            sc = torch.exp2(power.float())
            if form == "anyscale":
                sc = sc * 1.2345
            q = (rows[..., :512].view(n_pages, page, 4, 128) / sc[..., None]).clamp(-448, 448)
            codes.view(torch.uint8)[:, 2] = q.view(n_pages, page, 512).to(torch.float8_e4m3fn).view(torch.uint8)
            scale = torch.full((n_pages, 2, page, 4), nan, device="cuda")
            scale[:, 0] = sc
            raw = torch.full((n_pages, 2, page, 64), nan, device="cuda", dtype=torch.bfloat16)
            raw[:, 1] = rows[..., 512:].bfloat16()
            codes, scale, raw = codes[:, 2], scale[:, 0], raw[:, 1]
            v = codes.float().view(n_pages, page, 4, 128) * scale[..., None]
            v = v.view(n_pages, page, 512)
            if form == "anyscale":      # entered in bf16, as documented
                v = v.bfloat16().float()
            self.rows = torch.cat((v, raw.float()), -1).double()
        self.cache = B.PagedCache(codes, scale, raw)
        self.q = (torch.randn(batch, n_q, heads, 576, device="cuda", generator=g) * spread).bfloat16()
        self.k_len = torch.tensor(k_lens, dtype=torch.int32, device="cuda")
        self.q_len = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device="cuda")
        self.k_lens, self.q_lens = k_lens, q_lens or [n_q] * batch
        self.n_q, self.heads, self.page = n_q, heads, page
        if q_lens:                      # queries of padding tokens
            for b, n in enumerate(q_lens):
                self.q[b, n:] = nan

    def run(self, B, **kw):
        batch = len(self.k_lens)
        out = torch.full((batch, self.n_q, self.heads, 512), 77.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((batch, self.n_q, self.heads), 77.0, device="cuda")
        kw = {**dict(out=out, out_lse=lse, flags=B.DSA_FLAG_CHECK), **kw}
        return B.paged_mla(self.q, self.cache, self.table, self.k_len, SCALE, self.q_len, **kw)

    def check(self, out, lse, tokens=None):
        worst = 0.0
        for b, (n, m) in enumerate(zip(self.k_lens, self.q_lens)):
            assert bool((out[b, m:] == 77.0).all()) and bool((lse[b, m:] == 77.0).all())
            pages = self.table[b, :-(-n // self.page)].long()
            kv = self.rows[pages].reshape(-1, 576)[:n]
            for t in (range(m) if tokens is None else [t for t in tokens if t < m]):
                seen = n - m + t + 1
                o, z = out[b, t].double(), lse[b, t].double()
                if seen <= 0:
                    assert bool((o == 0).all()) and bool((z == float("-inf")).all())
                    continue
                k, q = kv[:seen], self.q[b, t].double()
                x = SCALE * q @ k.T
                exact = torch.logsumexp(x, -1)
                w = torch.exp(x - exact[:, None])
                d = (52 * 2.0 ** -23 * SCALE * (q.abs() @ k.abs().T).amax(-1)
                     + 2.0 ** -20 * (1 + x.abs().amax(-1)))
                want, size = w @ k[:, :512], w @ k[:, :512].abs()
                bound = (2.0 ** -8 + 3 * d[:, None]) * size + 2.0 ** -8 * (1 + 2.0 ** -7) * want.abs()
                err = (o - want).abs()
                assert bool((err <= bound).all()), (b, t, float((err / bound).max()))
                assert bool(((z - exact).abs() <= d + 2.0 ** -22 * exact.abs()).all()), (b, t)
                worst = max(worst, float((err / bound).max()))
        return worst


CASES = [
    # k_lens, q_lens, n_q, heads, page: lengths of zero, one, around a tile and a page
    ([1], None, 1, 1, 64), ([0], None, 1, 16, 64), ([127, 128, 129, 0, 1], None, 1, 16, 64),
    ([64, 63, 65, 300], None, 1, 128, 16), ([1000], None, 1, 128, 64), ([5000], None, 1, 128, 16),
    ([700, 31], None, 1, 64, 32), ([900, 2], None, 1, 20, 128), ([900, 333], None, 1, 65, 256),
    ([4096, 17], None, 1, 7, 4096),
    # a few tokens, some of them before the first cached position
    ([129, 2, 4, 1000], None, 4, 16, 64), ([511, 513], None, 3, 100, 32), ([300], None, 2, 128, 64),
    # ragged tokens: none, one, all of them; a tile with rows of several tokens
    ([640, 5, 77, 0], [4, 0, 1, 4], 4, 32, 16), ([200, 260], [9, 3], 9, 33, 64),
    # prompt chunks: several row tiles, causal inside
    ([130], None, 130, 16, 64), ([400, 257], [150, 257], 257, 8, 32), ([300], None, 40, 128, 64),
    ([2000], None, 70, 24, 128)]


@pytest.mark.parametrize("case", CASES, ids=[str(c).replace(" ", "") for c in CASES])
@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_matches_formula(B, case, form):
    k_lens, q_lens, n_q, heads, page = case
    p = Problem(B, sum(k_lens) + n_q + heads, k_lens, q_lens, n_q, heads, page, form)
    out, lse = p.run(B)
    print("largest error / bound:", p.check(out, lse))
    again = p.run(B)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_scales_that_are_no_powers_of_two(B):
    p = Problem(B, 5, [700, 129], None, 2, 48, 64, "anyscale")
    p.check(*p.run(B))


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_many_sequences_and_room_in_the_table(B, form):
    """More sequences than clusters, lengths from 0 to some thousand, a table wider than
    any sequence."""
    g = torch.Generator().manual_seed(6)
    k_lens = torch.randint(0, 3001, (150,), generator=g).tolist()
    k_lens[3], k_lens[70] = 0, 1
    p = Problem(B, 6, k_lens, None, 1, 16, 64, form, room=40)
    p.check(*p.run(B))


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_padded_batch(B, form):
    """A batch padded to a long prompt: most row tiles are empty, rows of padding tokens
    stay as they were."""
    q_lens = [1, 300, 0, 7, 2, 512, 1]
    p = Problem(B, 18, [700, 300, 50, 3, 1500, 600, 1], q_lens, 512, 48, 32, form)
    out, lse = p.run(B)
    p.check(out, lse, tokens=[0, 1, 2, 6, 150, 299, 300, 511])


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_large_logits(B, form):
    """Logits of hundreds: the maximum is raised many times, weights vanish."""
    p = Problem(B, 7, [3000, 400], None, 2, 64, 64, form, spread=40.0)
    p.check(*p.run(B))


@pytest.mark.parametrize("heads,form", [(128, "bf16"), (128, "e4m3"), (16, "bf16")])
def test_long_sequence_beside_short_ones(B, heads, form):
    p = Problem(B, 8, [131072, 1, 5000, 20000], None, 1, heads, 64, form)
    p.check(*p.run(B))


@pytest.mark.parametrize("form,heads,n_q", [("bf16", 16, 1), ("e4m3", 16, 1), ("e4m3", 64, 3)])
def test_many_short_sequences_between_long_ones(B, form, heads, n_q):
    """Shares long enough for a pair's extra units, ends of shares among those of the short
    ones, pairs that begin and end with a share."""
    short = [0, 1, 127, 128, 129, 300, 64, 2] * 8
    k_lens = [90001] + short + [128 * 20] * 6 + [70000] + short[:11] + [17]
    q_lens = None if n_q == 1 else [1 + i % n_q for i in range(len(k_lens))]
    p = Problem(B, 23, k_lens, q_lens, n_q, heads, 64, form)
    p.check(*p.run(B))


def test_long_prompt_chunk_sampled(B):
    p = Problem(B, 9, [9000], None, 400, 128, 64, "bf16")
    out, lse = p.run(B)
    p.check(out, lse, tokens=[0, 1, 63, 200, 398, 399])


def test_closed_forms(B):
    """One position: its value, bit for bit.  q = 0: the mean of the values."""
    p = Problem(B, 10, [1, 96], None, 1, 128, 64, "bf16")
    out, lse = p.run(B)
    v = p.rows[p.table[0, 0].long(), 0, :512]
    assert torch.equal(out[0, 0].double(), v.expand(128, 512))
    p.q.zero_()
    out, lse = p.run(B)
    kv = p.rows[p.table[1, :2].long()].reshape(-1, 576)[:96, :512]
    assert bool(((out[1, 0].double() - kv.mean(0)).abs() <= 2.0 ** -8 * kv.mean(0).abs() + 1e-6).all())
    assert bool(((lse[1].double() - torch.log(torch.tensor(96.0).double())).abs() <= 1e-5).all())


@pytest.mark.parametrize("power", [-126, -20, 0, 7, 8, 40])
def test_every_code_and_scale_exactly(B, power):
    """One position whose row holds every finite e4m3 code, subnormals among them, with
    scales from the smallest to large ones: the output is its value, bit for bit (at 2^-126
    the nearest bf16 to it: bf16 ends at 2^-133, the smallest code's value is 2^-135)."""
    bits = torch.arange(256, dtype=torch.uint8)
    bits[0x7f], bits[0xff] = 0x7e, 0xfe
    codes = torch.zeros(1, 16, 512, dtype=torch.uint8)
    codes[0, 0] = torch.cat((bits, bits.flip(0)))
    codes = codes.cuda().view(torch.float8_e4m3fn)
    scale = torch.full((1, 16, 4), 2.0 ** power, device="cuda")
    cache = B.PagedCache(codes, scale, torch.zeros(1, 16, 64, dtype=torch.bfloat16, device="cuda"))
    q = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = B.paged_mla(q, cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                           torch.ones(1, dtype=torch.int32, device="cuda"), 1.0)
    want = (codes[0, 0].float() * 2.0 ** power).bfloat16().float()
    assert torch.equal(out[0, 0].float(), want.expand(16, 512)) and bool((lse == 0).all())


@pytest.mark.parametrize("form", ["bf16", "e4m3", "anyscale"])
@pytest.mark.parametrize("column", [0, 191, 511, 575])
def test_a_nan_stays_one(B, form, column):
    """A NaN in a cached row makes the outputs of the tokens that see it NaN, whatever the
    row's form (e4m3: the codes 0x7f and 0xff), and no other sequence's.  With codes and
    powers of two the tokens before it are right as well: only its logits are NaN."""
    p = Problem(B, 19, [700, 700, 140], None, 3, 16, 64, form)
    want = p.run(B)
    for at, code in ((5, 0x7f), (130, 0xff), (698, 0x7f)):
        page, row = p.table[1, at // 64].long(), at % 64
        bits = form != "bf16" and column < 512
        plane = p.cache.codes.view(torch.uint8) if bits else p.cache.raw
        at_column = column if bits or form == "bf16" else column - 512
        keep = plane[page, row, at_column].clone()
        plane[page, row, at_column] = code if bits else float("nan")
        out, lse = p.run(B)
        plane[page, row, at_column] = keep
        for b in (0, 2):
            assert torch.equal(out[b], want[0][b]) and torch.equal(lse[b], want[1][b])
        first = max(0, at - (700 - 3))
        assert bool(out[1, first:].isnan().all()) and bool(lse[1, first:].isnan().all())
        if form == "e4m3":
            assert torch.equal(out[1, :first], want[0][1, :first])
            assert torch.equal(lse[1, :first], want[1][1, :first])
    again = p.run(B)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_nan_codes_behind_the_length(B):
    """Rows of a sequence's last page behind its length hold NaN codes next to live rows."""
    p = Problem(B, 20, [70, 129, 300], None, 2, 48, 64, "e4m3")
    codes = p.cache.codes.view(torch.uint8)
    for b, n in enumerate(p.k_lens):
        page = p.table[b, (n - 1) // 64].long()
        codes[page, (n - 1) % 64 + 1:] = 0xff
    p.check(*p.run(B))


def test_no_position_is_lost_or_counted_twice(B):
    """q = 0: every weight is 1, and with one 1 in each row (column s // 32 mod 512) an output
    counts its positions exactly: n / total, a power of two here, so a slice of 32 positions
    that is lost or taken twice changes it by an eighth."""
    for form in ("bf16", "e4m3"):
        n, page = 131072, 64
        g = torch.Generator(device="cuda").manual_seed(24)
        table = torch.randperm(n // page, device="cuda", generator=g).to(torch.int32)[None]
        s = torch.arange(n, device="cuda")
        slot = table[0].long()[s // page] * page + s % page
        cache = B.PagedCache.empty(n // page, page, *((0, 576) if form == "bf16" else (512, 64)))
        one = 1.0 if form == "bf16" else 0x38
        plane = cache.raw if form == "bf16" else cache.codes.view(torch.uint8)
        plane.view(n, -1)[slot, s // 32 % 512] = one
        for heads, n_q in ((16, 1), (128, 1)):
            q = torch.zeros(1, n_q, heads, 576, dtype=torch.bfloat16, device="cuda")
            for length in (n, n // 2):
                k_len = torch.tensor([length], dtype=torch.int32, device="cuda")
                out, lse = B.paged_mla(q, cache, table, k_len, 1.0, flags=B.DSA_FLAG_CHECK)
                assert bool((out.float() == 1 / 512).all()), (form, heads, length)
                # log2 and the product with ln 2: under two steps of fp32, 2^-22
                exact = torch.log(torch.tensor(float(length)).double())
                assert bool(((lse.double().cpu() - exact).abs() <= 2.0 ** -22 * exact).all())


def test_no_lse_and_clamped_lengths(B):
    """out_lse is optional at the C entry; lengths outside their range are clamped."""
    p = Problem(B, 11, [128, 100], None, 2, 16, 64, "bf16")
    out, lse = p.run(B)
    prob = B.DsaPagedMlaProblem(2, 2, 16, 576, 512, 2, 64, SCALE, B.DSA_FLAG_CHECK)
    ws = torch.empty(B.paged_mla_workspace_size(2, 2, 16, 2, 64), dtype=torch.uint8, device="cuda")
    got = torch.empty_like(out)
    k_len = torch.tensor([2 ** 31 - 1, 100], dtype=torch.int32, device="cuda")
    q_len = torch.tensor([2 ** 31 - 1, 5], dtype=torch.int32, device="cuda")
    rc = B.lib.dsa_paged_mla(C.byref(prob), C.byref(p.cache.c), p.q.data_ptr(), p.table.data_ptr(),
                             k_len.data_ptr(), q_len.data_ptr(), got.data_ptr(), None, ws.data_ptr(),
                             ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(got, out)
    k_len[:] = -3
    q_len[:] = -1
    keep = got.clone()
    rc = B.lib.dsa_paged_mla(C.byref(prob), C.byref(p.cache.c), p.q.data_ptr(), p.table.data_ptr(),
                             k_len.data_ptr(), q_len.data_ptr(), got.data_ptr(), None, ws.data_ptr(),
                             ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(got, keep)


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_page_outside_the_cache_is_reported(B, form):
    """A table entry that names no page, inside a length: reported, not followed, and the
    next call on the same workspace is right."""
    p = Problem(B, 12, [300, 500], None, 1, 16, 64, form)
    ws = torch.empty(B.paged_mla_workspace_size(2, 1, 16, p.table.shape[1], 64), dtype=torch.uint8,
                     device="cuda")
    good = p.table.clone()
    for bad in (-1, p.cache.c.n_pages, 2 ** 31 - 1, -2 ** 31):
        p.table[1, 3] = bad
        with pytest.raises(B.DsaError) as e:
            p.run(B, workspace=ws)
        assert e.value.status == B.DSA_ERR_INVALID
        p.run(B, workspace=ws, flags=0)
        assert B.dsa_read_status(ws) == B.DSA_ERR_INVALID
    p.table.copy_(good)
    p.check(*p.run(B, workspace=ws))
    assert B.dsa_read_status(ws) == 0


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_expired_wait_returns_timeout_then_next_call_is_right(B, form):
    """DSA_FLAG_TEST_STALL: a loader of the first cluster stops after a tile and every wait
    lasts at most about a millisecond.  The call returns DSA_ERR_TIMEOUT within a fraction of a
    second, every role having drained its copies and products, and the next call on the same
    stream and workspace is right, as are tokens and rows around it."""
    import time
    p = Problem(B, 25, [74 * 128 * 3 + 5, 300], [1, 1], 2, 16, 64, form)
    ws = torch.empty(B.paged_mla_workspace_size(2, 2, 16, p.table.shape[1], 64), dtype=torch.uint8,
                     device="cuda")
    want = p.run(B, workspace=ws)
    p.check(*want)
    for _ in range(3):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        with pytest.raises(B.DsaError) as e:
            p.run(B, workspace=ws, flags=B.DSA_FLAG_CHECK | B.DSA_FLAG_TEST_STALL)
        took = time.perf_counter() - t0
        assert e.value.status == B.DSA_ERR_TIMEOUT
        assert took < 1.0, f"the failed call took {took:.3f} s"
        assert B.dsa_read_status(ws) == B.DSA_ERR_TIMEOUT
        got = p.run(B, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert B.dsa_read_status(ws) == B.DSA_OK


def test_equals_sparse_mla_over_every_position(B):
    """The selection of all positions gives the same attention (both within their bounds;
    sparse_mla's denominator sums rounded weights: 2^-8)."""
    p = Problem(B, 13, [777, 512], None, 1, 128, 64, "bf16")
    out, lse = p.run(B)
    kv = B.cache_read(p.cache, p.table, 777, p.k_len)
    idx = torch.arange(777, device="cuda", dtype=torch.int32).repeat(2, 1)
    idx[1, 512:] = -1
    ref, ref_lse = B.sparse_mla(p.q[:, 0].contiguous(), kv, idx, SCALE)
    size = torch.stack([kv[b, :n, :512].abs().float().mean() for b, n in enumerate([777, 512])])
    assert bool(((out[:, 0].float() - ref.float()).abs() <= 2.0 ** -5 * size[:, None, None]).all())
    assert bool(((lse[:, 0] - ref_lse).abs() <= 2.0 ** -7).all())


def test_offsets_past_32_bits(B):
    """Pages more than 2^32 bytes from the start of the plane."""
    n_pages, page = 4200, 1024
    raw = torch.empty((n_pages, page, 576), dtype=torch.bfloat16, device="cuda")
    p = Problem(B, 14, [1500], None, 1, 32, 1024, "bf16")
    raw[-1], raw[-2] = p.cache.raw[p.table[0, 0].long()], p.cache.raw[p.table[0, 1].long()]
    want = p.run(B)
    p.cache = B.PagedCache(raw=raw)
    p.table[0, 0], p.table[0, 1] = n_pages - 1, n_pages - 2
    got = p.run(B)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_streams_and_two_graphs(B):
    """Another stream; two captured graphs, each with its workspace, replayed together on
    lengths that have changed since the capture."""
    p = Problem(B, 15, [2000, 900], None, 1, 16, 64, "bf16", room=1)
    r = Problem(B, 16, [300, 3000, 5], None, 2, 128, 32, "e4m3", room=1)
    want = [p.run(B), r.run(B)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = B.paged_mla(p.q, p.cache, p.table, p.k_len, SCALE, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    graphs, outs, spaces = [], [], []   # a graph's workspace lives as long as the graph
    for x in (p, r):
        ws = torch.empty(B.paged_mla_workspace_size(len(x.k_lens), x.n_q, x.heads, x.table.shape[1],
                                                    x.page), dtype=torch.uint8, device="cuda")
        spaces.append(ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(x.run(B, workspace=ws, flags=0))
        graphs.append(g)
    p.k_len[0], p.k_lens[0] = 1500, 1500
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    p.check(*outs[0])
    assert torch.equal(outs[1][0], want[1][0]) and torch.equal(outs[1][1], want[1][1])


def test_refusals(B):
    p = Problem(B, 17, [100], None, 1, 16, 64, "bf16")

    def status(prob=None, cache=None, **kw):
        d = dict(batch=1, n_q=1, heads=16, dim_qk=576, dim_v=512, max_pages=2, page_size=64,
                 scale=SCALE, flags=0)
        d.update(prob or {})
        v = dict(q=0x1000, table=0x1000, k_len=0x1000, q_len=None, out=0x1000, lse=None, ws=0x1000,
                 nbytes=1 << 40)
        v.update(kw)
        c = p.cache.c if cache is None else cache
        return B.lib.dsa_paged_mla(C.byref(B.DsaPagedMlaProblem(**d)), C.byref(c), v["q"], v["table"],
                                   v["k_len"], v["q_len"], v["out"], v["lse"], v["ws"], v["nbytes"],
                                   None)

    for prob, want in [(dict(batch=0), -1), (dict(n_q=0), -1), (dict(heads=0), -1), (dict(heads=129), -2),
                       (dict(dim_qk=512), -2), (dict(dim_v=576), -2), (dict(max_pages=0), -1),
                       (dict(page_size=32), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
                       (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
                       (dict(max_pages=1 << 20), -2), (dict(batch=1 << 30), -2),
                       (dict(batch=1 << 20, n_q=1 << 12), -2)]:
        assert status(prob) == want, prob
    for kw in (dict(q=None), dict(table=None), dict(k_len=None), dict(out=None), dict(q=0x1008),
               dict(out=0x1008), dict(table=0x1002), dict(k_len=0x1002), dict(q_len=0x1001),
               dict(lse=0x1002), dict(ws=0x1008)):
        assert status(**kw) == -1, kw
    assert status(ws=None) == -3 and status(nbytes=1000) == -3
    keys = B.PagedCache.empty(2, 64, 128, 0)
    assert status(cache=keys.c) == -2
    assert status(cache=B.PagedCache.empty(2, 64, 512, 72).c) == -2
    with pytest.raises(ValueError):
        B.paged_mla(p.q[0], p.cache, p.table, p.k_len, SCALE)
    with pytest.raises(ValueError):
        B.paged_mla(p.q, p.cache, p.table, p.k_len[:0], SCALE)
    with pytest.raises(TypeError):
        B.paged_mla(p.q.half(), p.cache, p.table, p.k_len, SCALE)
    with pytest.raises(ValueError):
        B.paged_mla(p.q, p.cache, p.table, p.k_len, SCALE, out=torch.empty(1, device="cuda").bfloat16())
    with pytest.raises(B.DsaError):
        B.paged_mla(p.q, p.cache, p.table, p.k_len, SCALE,
                    workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
