"""A cached DSA layer put together from the library's calls, as a serving loop uses them:
rotary positions, the writes of a prompt and of single tokens, the indexer over the keys
read back, Sparse MLA over the rows read back, latent attention over the pages."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
PAGE = 64


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_attention_token_dsa_b200 import binding
    return binding


class Layer:
    """Pages of latent rows (e4m3 + bf16) and of indexer keys (e4m3), one block table."""

    def __init__(self, B, batch, most, seed):
        self.B = B
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        per = -(-most // PAGE)
        self.latent = B.PagedCache.empty(batch * per, PAGE, 512, 64)
        self.keys = B.PagedCache.empty(batch * per, PAGE, 128, 0)
        self.table = torch.randperm(batch * per, device="cuda", generator=g).to(torch.int32).view(batch, per)
        self.freq = B.rope_frequencies(64, scaling="yarn", factor=40.0)
        self.m = 0.1 * torch.log(torch.tensor(40.0)).item() + 1.0

    def slots(self, seq, pos):
        page = self.table[seq, (pos // PAGE).long()].long()
        return page * PAGE + pos.long() % PAGE

    def append(self, seq, pos, latent, key):
        """seq, pos [tokens] int32; latent [tokens, 576], key [tokens, 128] bf16."""
        B, slots = self.B, self.slots(seq.long(), pos)
        B.cache_write(self.latent, latent, slots, pow2=True, freq=self.freq, pos=pos, offset=512,
                      interleaved=True, mscale=self.m)
        turned = B.rope(key[:, None], pos, self.freq, offset=0, mscale=self.m)[:, 0]
        B.cache_write(self.keys, turned, slots)
        return turned


def rows(layer, b, n):
    """The cached latent rows of a sequence in 64 bits."""
    at = layer.slots(torch.full((n,), b, device="cuda"), torch.arange(n, device="cuda"))
    c = layer.latent
    v = c.codes.view(-1, 4, 128).float()[at] * c.scale.view(-1, 4)[at][..., None]
    return torch.cat((v.flatten(1), c.raw.view(-1, 64)[at].float()), 1).double()


def test_prompt_then_single_tokens(B):
    lens = [200, 77, 130]
    most = 330
    layer = Layer(B, 3, most, 21)
    g = layer.g
    latent = torch.randn(3, most, 576, device="cuda", generator=g).bfloat16()
    key = torch.randn(3, most, 128, device="cuda", generator=g).bfloat16()
    # the prompts, all sequences' tokens in one call
    seq = torch.cat([torch.full((n,), b, device="cuda") for b, n in enumerate(lens)]).to(torch.int32)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens]).to(torch.int32)
    turned = layer.append(seq, pos, latent[seq.long(), pos.long()], key[seq.long(), pos.long()])

    # the cache holds what the formula says: latent part quantised, rotated part rounded once
    angle = pos.double()[:, None] * layer.freq
    tail = latent[seq.long(), pos.long()][:, 512:].double().unflatten(1, (32, 2))
    want = torch.stack((tail[..., 0] * angle.cos() - tail[..., 1] * angle.sin(),
                        tail[..., 1] * angle.cos() + tail[..., 0] * angle.sin()), -1).flatten(1) * layer.m
    size = (tail.abs().sum(-1, keepdim=True) * layer.m).expand(-1, -1, 2).flatten(1)
    got = torch.cat([rows(layer, b, n) for b, n in enumerate(lens)])
    assert bool(((got[:, 512:] - want).abs() <= 2.0 ** -8 * want.abs() * 1.001 + 2.0 ** -20 * size).all())
    x = latent[seq.long(), pos.long()][:, :512].double()
    amax = x.view(-1, 4, 128).abs().amax(-1, keepdim=True).expand(-1, -1, 128).flatten(1)
    # half a step: 2^-4 of the value, or of the subnormal range (2^-10 scales, scale <= amax / 224)
    assert bool(((got[:, :512] - x).abs() <= x.abs() * 2.0 ** -4 + amax * 2.0 ** -17).all())

    # three steps of one token each
    for step in range(3):
        at = torch.tensor([n + step for n in lens], dtype=torch.int32, device="cuda")
        s = torch.arange(3, device="cuda", dtype=torch.int32)
        new = layer.append(s, at, latent[s.long(), at.long()], key[s.long(), at.long()])
        k_len = at + 1
        n_k = int(k_len.max())

        # the indexer over the keys read back equals the indexer over keys quantised in place
        q = torch.randn(3, 1, 64, 128, device="cuda", generator=g).bfloat16()
        q = B.rope(q[:, 0], at, layer.freq, mscale=layer.m)[:, None].contiguous()
        w = torch.randn(3, 1, 64, device="cuda", generator=g)
        codes, scale = B.cache_read_codes(layer.keys, layer.table, n_k, k_len)
        direct = torch.zeros(3, n_k, 128, device="cuda", dtype=torch.bfloat16)
        turned_all = B.rope(key[:, :n_k].reshape(-1, 1, 128), torch.arange(n_k, device="cuda").to(
            torch.int32).repeat(3), layer.freq, mscale=layer.m).view(3, n_k, 128)
        for b in range(3):
            direct[b, :k_len[b]] = turned_all[b, :k_len[b]]
        dc, ds = B.dsa_quantize_e4m3(direct)
        kw = dict(q_pos0=at, k_len=k_len, flags=B.DSA_FLAG_BY_POSITION | B.DSA_FLAG_CHECK)
        topk = 64
        idx, score = B.dsa_index(q, codes, w, topk, k_scale=scale, **kw)
        idx2, score2 = B.dsa_index(q, dc.view(torch.float8_e4m3fn), w, topk, k_scale=ds, **kw)
        assert torch.equal(idx, idx2) and torch.equal(score, score2)

        # Sparse MLA over every position = latent attention over the pages
        qm = torch.randn(3, 1, 16, 576, device="cuda", generator=g).bfloat16()
        qm = B.rope(qm[:, 0], at, layer.freq, offset=512, interleaved=True, mscale=layer.m)
        kv = B.cache_read(layer.latent, layer.table, n_k, k_len)
        every, _ = B.dsa_index(q, codes, w, 512, k_scale=scale, **kw)
        for b in range(3):
            n = int(k_len[b])
            assert torch.equal(every[b, 0, :n], torch.arange(n, device="cuda", dtype=torch.int32))
            assert bool((every[b, 0, n:] == -1).all())
        sparse, sparse_lse = B.sparse_mla(qm, kv, every[:, 0].contiguous(), SCALE)
        dense, dense_lse = B.paged_mla(qm[:, None].contiguous(), layer.latent, layer.table, k_len, SCALE,
                                       flags=B.DSA_FLAG_CHECK)
        for b in range(3):
            v = rows(layer, b, int(k_len[b]))
            xs = SCALE * qm[b].double() @ v.T
            p = torch.softmax(xs, -1)
            ref, size = p @ v[:, :512], p @ v[:, :512].abs()
            # weights in bf16, one rounding of the output, logits within 2^-11 (both kernels)
            bound = (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -7 * ref.abs()
            assert bool(((dense[b, 0].double() - ref).abs() <= bound).all())
            assert bool(((sparse[b].double() - ref).abs() <= bound + 2.0 ** -8 * size).all())
            z = torch.logsumexp(xs, -1)
            assert bool(((dense_lse[b, 0] - z).abs() <= 2.0 ** -10).all())
            assert bool(((sparse_lse[b] - z).abs() <= 2.0 ** -7).all())

        # attention over the indexer's own selection: those rows alone
        few, _ = B.sparse_mla(qm, kv, idx[:, 0].contiguous(), SCALE)
        for b in range(3):
            v = rows(layer, b, int(k_len[b]))[idx[b, 0][idx[b, 0] >= 0].long()]
            p = torch.softmax(SCALE * qm[b].double() @ v.T, -1)
            ref, size = p @ v[:, :512], p @ v[:, :512].abs()
            assert bool(((few[b].double() - ref).abs() <= 2.0 ** -6 * size + 2.0 ** -7 * ref.abs()).all())
    assert turned.shape == (sum(lens), 128) and new.shape == (3, 128)


def test_rows_written_one_by_one_equal_rows_written_at_once(B):
    a, b = Layer(B, 2, 150, 22), Layer(B, 2, 150, 22)
    g = a.g
    latent = torch.randn(300, 576, device="cuda", generator=g).bfloat16()
    key = torch.randn(300, 128, device="cuda", generator=g).bfloat16()
    seq = (torch.arange(300, device="cuda") % 2).to(torch.int32)
    pos = (torch.arange(300, device="cuda") // 2).to(torch.int32)
    a.append(seq, pos, latent, key)
    for t in torch.randperm(300).tolist():
        b.append(seq[t:t + 1], pos[t:t + 1], latent[t:t + 1], key[t:t + 1])
    for x, y in ((a.latent, b.latent), (a.keys, b.keys)):
        assert torch.equal(x.codes.view(torch.uint8), y.codes.view(torch.uint8))
        assert torch.equal(x.scale, y.scale)
    assert torch.equal(a.latent.raw, b.latent.raw)
