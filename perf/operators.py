"""Cases of the operators around a cached DSA layer: rotary positions, the write into
the paged cache, the read from it, and latent attention over its pages.

`own` false runs each operator as elementary torch operations in 32 bits (angles in
64); `own` true makes the framework's calls on the same state.
"""
import math

import torch

own = False

LATENT, ROPE = 512, 64          # a cached MLA row: latent part, rotated part
ROW = LATENT + ROPE
INDEX = 128                     # a cached indexer key
SCALE = 192 ** -0.5             # softmax scale of the MLA read


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the indexer's queries of one decode step: 32 sequences, 64 heads
        dict(name="rope step", op="rope", tokens=32, heads=64, dim=128, offset=0, rot=64,
             interleaved=False, dtype="bf16", inverse=False, factor=1.0),
        # the indexer's queries of an 8192-token prompt, positions scaled for long contexts
        dict(name="rope prompt", op="rope", tokens=8192, heads=64, dim=128, offset=0, rot=64,
             interleaved=False, dtype="bf16", inverse=False, factor=40.0),
        # the gradient of MLA queries of a training sequence (odd length), fp32
        dict(name="rope gradient", op="rope", tokens=2049, heads=64, dim=576, offset=512, rot=64,
             interleaved=True, dtype="f32", inverse=True, factor=40.0),
        # one decode step appends a latent row to each of 32 sequences, rotating its last part
        dict(name="write step", op="write", tokens=32, form="latent", page=64, dtype="bf16",
             rotate=True, scattered=True),
        # an 8K prompt's latent rows (odd length)
        dict(name="write prompt", op="write", tokens=8191, form="latent", page=64, dtype="bf16",
             rotate=True, scattered=False),
        # the indexer keys of a 128K prompt
        dict(name="write index keys", op="write", tokens=131072, form="index", page=64,
             dtype="bf16", rotate=False, scattered=False),
        # the latent rows of two long sequences, dequantised for Sparse MLA
        dict(name="read latent", op="read", batch=2, n_k=32768, form="latent", page=64,
             ragged=True),
        # the indexer keys of a decode batch, codes and scales for the indexer's scan
        dict(name="read index keys", op="read", batch=32, n_k=16384, form="index", page=64,
             ragged=True),
        # one token of a short conversation, 16 heads on this device
        dict(name="mla step short", op="mla", batch=1, n_q=1, heads=16, n_k=1000, form="bf16",
             page=64, ragged=False),
        # one token for each of 32 sequences of 128K
        dict(name="mla step 128K", op="mla", batch=32, n_q=1, heads=128, n_k=131072, form="bf16",
             page=64, ragged=False),
        # four tokens a sequence (three guessed ahead), ragged lengths, e4m3 rows
        dict(name="mla guess e4m3", op="mla", batch=24, n_q=4, heads=64, n_k=16001, form="e4m3",
             page=64, ragged=True),
        # a chunk of a prompt behind 8K cached positions
        dict(name="mla chunk", op="mla", batch=1, n_q=512, heads=128, n_k=8704, form="bf16",
             page=32, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "mla", "mla"])
    if op == "rope":
        dim, offset, rot = rng.choice([(128, 0, 64), (576, 512, 64), (64, 0, 64), (128, 0, 128)])
        heads = rng.choice([1, 5, 16, 32, 64, 128])
        most = 2049 * 64 * 576 // (heads * dim)
        return dict(op=op, tokens=_log(rng, 1, min(16384, most)), heads=heads, dim=dim,
                    offset=offset, rot=rot, interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f32"]), inverse=rng.random() < 0.5,
                    factor=rng.choice([1.0, 4.0, 40.0]))
    if op == "write":
        form = rng.choice(["latent", "index", "bf16"])
        return dict(op=op, tokens=_log(rng, 1, 131072 if form == "index" else 32768), form=form,
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "f32"]),
                    rotate=form != "index" and rng.random() < 0.5, scattered=rng.random() < 0.5)
    if op == "read":
        form = rng.choice(["latent", "index", "bf16"])
        batch = _log(rng, 1, 64)
        most = (524288 if form == "index" else 65536) // batch
        return dict(op=op, batch=batch, n_k=_log(rng, 1, most), form=form,
                    page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)
    n_q = rng.choice([1, 1, 1, 2, 3, 5, _log(rng, 2, 700)])
    heads = rng.choice([8, 16, 20, 32, 64, 128])
    batch = _log(rng, 1, 48 if n_q < 8 else 4)
    most = min(32 * 131072 // batch, 32 * 128 * 131072 // (batch * n_q * heads))
    return dict(op=op, batch=batch, n_q=n_q, heads=heads,
                n_k=_log(rng, max(1, n_q // 2), max(n_q, min(131072, most))),
                form=rng.choice(["bf16", "e4m3"]), page=rng.choice([16, 32, 64, 128]),
                ragged=rng.random() < 0.7)


# ----------------------------------------------------------------- inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _frequencies(rot, factor, base=10000.0, trained=4096, fast=32.0, slow=1.0):
    """Radians a position for each pair, the slow ones divided by `factor` (YaRN),
    and the factor on the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    freq = base ** (-2.0 * i / rot)
    if factor == 1.0:
        return freq.cuda(), 1.0

    def at(turns):
        return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return (freq / factor * ramp + freq * (1 - ramp)).cuda(), 0.1 * math.log(factor) + 1.0


def _widths(form):
    """(values held in e4m3, values held in bf16) of a cached row."""
    return {"latent": (LATENT, ROPE), "e4m3": (LATENT, ROPE), "index": (INDEX, 0),
            "bf16": (0, ROW)}[form]


def _pages(form, n_pages, page, g):
    """Planes of a cache that earlier tokens have filled."""
    dim_q, dim_raw = _widths(form)
    codes = scale = raw = None
    if dim_q:
        codes = torch.randn(n_pages, page, dim_q, device="cuda", generator=g, dtype=torch.bfloat16)
        codes = (codes * 128).clamp_(-448, 448).to(torch.float8_e4m3fn)
        scale = torch.randint(-8, -5, (n_pages, page, dim_q // 128), device="cuda", generator=g)
        scale = torch.exp2(scale.float())
    if dim_raw:
        raw = torch.randn(n_pages, page, dim_raw, device="cuda", generator=g, dtype=torch.bfloat16)
    return codes, scale, raw


def _sequences(batch, n_k, page, ragged, least, g):
    """Pages of each sequence in no order, and its cached length."""
    n = -(-n_k // page)
    table = torch.randperm(batch * n, device="cuda", generator=g).to(torch.int32).view(batch, n)
    k_len = torch.full((batch,), n_k, dtype=torch.int32, device="cuda")
    if ragged:
        k_len = torch.randint(min(least, n_k), n_k + 1, (batch,), device="cuda", generator=g)
        k_len = k_len.to(torch.int32)
        k_len[0] = n_k
    return table, k_len


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "rope":
        s["x"] = torch.randn(case["tokens"], case["heads"], case["dim"], device="cuda", generator=g,
                             dtype=_dtype(case["dtype"]))
        top = int(4096 * case["factor"])
        start = torch.randint(0, top, (1,), device="cuda", generator=g)
        s["pos"] = (start + torch.arange(case["tokens"], device="cuda")).to(torch.int32)
        s["freq"], s["mscale"] = _frequencies(case["rot"], case["factor"])
        s["out"] = torch.empty_like(s["x"])
    elif case["op"] == "write":
        dim_q, dim_raw = _widths(case["form"])
        n, page = case["tokens"], case["page"]
        n_pages = -(-n // page) + 8
        s["codes"], s["scale"], s["raw"] = _pages(case["form"], n_pages, page, g)
        s["x"] = torch.randn(n, dim_q + dim_raw, device="cuda", generator=g,
                             dtype=_dtype(case["dtype"]))
        if case["scattered"]:       # a step of many sequences: one row in each of many pages
            s["slots"] = torch.randperm(n_pages * page, device="cuda", generator=g)[:n].contiguous()
        else:                       # a prompt: whole pages, in no order
            rows = torch.randperm(n_pages, device="cuda", generator=g)[:, None] * page
            s["slots"] = (rows + torch.arange(page, device="cuda")).view(-1)[:n].contiguous()
        s["pos"] = torch.randint(0, 131072, (n,), device="cuda", generator=g).to(torch.int32)
        s["freq"], _ = _frequencies(ROPE, 40.0)
        s["offset"] = dim_q + dim_raw - ROPE
    elif case["op"] == "read":
        dim_q, dim_raw = _widths(case["form"])
        batch, n_k, page = case["batch"], case["n_k"], case["page"]
        s["table"], s["k_len"] = _sequences(batch, n_k, page, case["ragged"], 0, g)
        s["codes"], s["scale"], s["raw"] = _pages(case["form"], s["table"].numel(), page, g)
        if case["form"] == "index":
            s["out"] = (torch.zeros(batch, n_k, dim_q, device="cuda", dtype=torch.uint8)
                        .view(torch.float8_e4m3fn), torch.ones(batch, n_k, device="cuda"))
        else:
            s["out"] = torch.zeros(batch, n_k, dim_q + dim_raw, device="cuda", dtype=torch.bfloat16)
    else:
        batch, n_q, heads = case["batch"], case["n_q"], case["heads"]
        n_k, page = case["n_k"], case["page"]
        s["table"], s["k_len"] = _sequences(batch, n_k, page, case["ragged"], n_q, g)
        s["codes"], s["scale"], s["raw"] = _pages(case["form"], s["table"].numel(), page, g)
        s["q"] = torch.randn(batch, n_q, heads, ROW, device="cuda", generator=g,
                             dtype=torch.bfloat16)
        s["q_len"] = torch.full((batch,), n_q, dtype=torch.int32, device="cuda")
        if case["ragged"] and n_q > 1:
            s["q_len"] = torch.randint(1, n_q + 1, (batch,), device="cuda", generator=g)
            s["q_len"] = s["q_len"].to(torch.int32)
        # rows behind a sequence's last query stay as they are
        s["out"] = torch.zeros(batch, n_q, heads, LATENT, device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros(batch, n_q, heads, device="cuda")
        s["workspace"] = torch.empty(64 << 20, device="cuda", dtype=torch.uint8)
    return s


# ---------------------------------------------------- the framework's calls --

def _own(s):
    from sparse_attention_token_dsa_b200 import binding as dsa
    if s["op"] == "rope":
        call = dsa.rope_backward if s["inverse"] else dsa.rope
        return call(s["x"], s["pos"], s["freq"], offset=s["offset"], interleaved=s["interleaved"],
                    mscale=s["mscale"], out=s["out"])
    cache = dsa.PagedCache(s["codes"], s["scale"], s["raw"])
    if s["op"] == "write":
        turn = dict(freq=s["freq"], pos=s["pos"], offset=s["offset"], interleaved=True)
        dsa.cache_write(cache, s["x"], s["slots"], pow2=s["form"] != "index",
                        **(turn if s["rotate"] else {}))
        return s["codes"], s["scale"], s["raw"]
    if s["op"] == "read":
        if s["form"] == "index":
            return dsa.cache_read_codes(cache, s["table"], s["n_k"], k_len=s["k_len"], out=s["out"])
        return dsa.cache_read(cache, s["table"], s["n_k"], k_len=s["k_len"], out=s["out"])
    return dsa.paged_mla(s["q"], cache, s["table"], s["k_len"], SCALE, q_len=s["q_len"],
                         out=s["out"], out_lse=s["lse"], workspace=s["workspace"])


# ------------------------------------------------------------- plain forms --

def _turned(part, pos, freq, interleaved, inverse, mscale):
    """part [tokens, heads, rot] in 32 bits, turned by pos * freq."""
    angle = pos.double()[:, None, None] * freq
    cos, sin = (angle.cos() * mscale).float(), (angle.sin() * mscale).float()
    if inverse:
        sin = -sin
    half = part.shape[-1] // 2
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)


def _plain_rope(s):
    lo, hi = s["offset"], s["offset"] + s["rot"]
    y = s["x"].clone()
    y[..., lo:hi] = _turned(s["x"][..., lo:hi].float(), s["pos"], s["freq"], s["interleaved"],
                            s["inverse"], s["mscale"]).to(y.dtype)
    return y


def _plain_write(s):
    dim_q, dim_raw = _widths(s["form"])
    x = s["x"].float()
    if s["rotate"]:
        part = _turned(x[:, None, s["offset"]:], s["pos"], s["freq"], True, False, 1.0)[:, 0]
        x = torch.cat((x[:, :s["offset"]], part), 1)
    if dim_q:
        groups = x[:, :dim_q].view(-1, dim_q // 128, 128)
        amax = groups.abs().amax(-1)
        if s["form"] == "index":
            a = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        else:
            part, power = torch.frexp(amax)
            power = torch.where(part > 0.875, power - 8, power - 9)
            a = torch.ldexp(torch.ones_like(amax), power)
            a = torch.where(amax > 0, a, torch.ones_like(amax))
        codes = (groups / a[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["codes"].view(torch.uint8).view(-1, dim_q)[s["slots"]] = codes.view(torch.uint8).flatten(1)
        s["scale"].view(-1, dim_q // 128)[s["slots"]] = a
    if dim_raw:
        s["raw"].view(-1, dim_raw)[s["slots"]] = x[:, dim_q:].to(torch.bfloat16)
    return s["codes"], s["scale"], s["raw"]


def _rows(s, n_k):
    """The first n_k positions of each sequence as [batch, n_k, width], 32 bits."""
    table = s["table"].long()
    parts = []
    if s["codes"] is not None:
        v = s["codes"][table].float().unflatten(-1, (-1, 128)) * s["scale"][table][..., None]
        parts.append(v.flatten(-2))
    if s["raw"] is not None:
        parts.append(s["raw"][table].float())
    return torch.cat(parts, -1).flatten(1, 2)[:, :n_k]


def _plain_read(s):
    n_k, table = s["n_k"], s["table"].long()
    live = torch.arange(n_k, device="cuda") < s["k_len"][:, None]
    if s["form"] == "index":
        codes = s["codes"].view(torch.uint8)[table].flatten(1, 2)[:, :n_k]
        codes = torch.where(live[..., None], codes, s["out"][0].view(torch.uint8))
        scale = s["scale"][table].flatten(1)[:, :n_k]
        return codes.view(torch.float8_e4m3fn), torch.where(live, scale, s["out"][1])
    return torch.where(live[..., None], _rows(s, n_k).to(torch.bfloat16), s["out"])


def _plain_mla(s):
    batch, n_q, heads, _ = s["q"].shape
    n_k = s["n_k"]
    kv = _rows(s, n_k)
    x = (s["q"].float().flatten(1, 2) @ kv.transpose(1, 2)).view(batch, n_q, heads, n_k) * SCALE
    token = torch.arange(n_q, device="cuda")
    pos = (s["k_len"] - s["q_len"])[:, None] + token
    x = x.masked_fill((torch.arange(n_k, device="cuda") > pos[..., None])[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
    total = x.sum(-1, keepdim=True)
    out = (x.flatten(1, 2) @ kv[..., :LATENT]).view(batch, n_q, heads, LATENT)
    out = out / total.masked_fill(total == 0, 1.0)
    lse = (top + total.log())[..., 0]
    live = (token < s["q_len"][:, None])[..., None]
    return torch.where(live[..., None], out.to(torch.bfloat16), s["out"]), torch.where(live, lse, s["lse"])


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "write": _plain_write, "read": _plain_read,
            "mla": _plain_mla}[s["op"]](s)


# ------------------------------------------------------------------- work --

def _row_bytes(form):
    dim_q, dim_raw = _widths(form)
    return dim_q + dim_q // 128 * 4 + dim_raw * 2


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        size = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=2 * n * case["dim"] * size + 4 * case["tokens"], flops=3 * n * case["rot"])
    if case["op"] == "write":
        dim = sum(_widths(case["form"]))
        size = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=case["tokens"] * (dim * size + 8 + _row_bytes(case["form"])),
                    flops=3 * case["tokens"] * dim)
    share = 0.5 if case["ragged"] else 1.0      # ragged lengths fill about half
    rows = case["n_k"] * (1 + share * (case["batch"] - 1))
    if case["op"] == "read":
        dim_q, dim_raw = _widths(case["form"])
        out = dim_q + 4 if case["form"] == "index" else 2 * (dim_q + dim_raw)
        return dict(bytes=rows * (_row_bytes(case["form"]) + out), flops=rows * dim_q)
    n_q = case["n_q"] * (0.5 if case["ragged"] and case["n_q"] > 1 else 1.0)
    heads = case["heads"] * n_q
    seen = max(1.0, rows / case["batch"] - (n_q - 1) / 2) * case["batch"]   # causal
    return dict(bytes=rows * _row_bytes(case["form"])
                + case["batch"] * heads * (2 * ROW + 2 * LATENT + 4),
                flops=2 * heads * seen * (ROW + LATENT))


# ------------------------------------------------------- 64-bit definition --

def _e4m3(v):
    """Nearest e4m3 value of 64-bit v, ties to even, largest 448."""
    a = v.abs().clamp(min=2.0 ** -20)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_turn(x, pos, freq, interleaved, sign, mscale):
    """Each pair as a complex number times mscale e^(i sign pos freq)."""
    half = x.shape[-1] // 2
    pairs = x.unflatten(-1, (half, 2)) if interleaved else x.unflatten(-1, (2, half)).transpose(-1, -2)
    turn = torch.polar(torch.full_like(freq, mscale).expand(len(pos), half),
                       sign * pos.double()[:, None] * freq)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    return y.flatten(-2) if interleaved else y.transpose(-1, -2).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        y = s["x"].double()
        part = slice(case["offset"], case["offset"] + case["rot"])
        y[..., part] = _exact_turn(y[..., part], s["pos"], s["freq"], case["interleaved"],
                                   -1.0 if case["inverse"] else 1.0, s["mscale"])
        return y
    if case["op"] == "write":
        dim_q, dim_raw = _widths(case["form"])
        x = s["x"].double()
        if case["rotate"]:
            tail = x[:, None, s["offset"]:]
            x[:, s["offset"]:] = _exact_turn(tail, s["pos"], s["freq"], True, 1.0, 1.0)[:, 0]
        codes = scale = raw = None
        if dim_q:
            codes = s["codes"].double()
            scale = s["scale"].double()
            for j in range(dim_q // 128):
                v = x[:, 128 * j:128 * j + 128]
                amax = v.abs().amax(1)
                a = amax / 448
                if case["form"] != "index":
                    a = torch.exp2(torch.ceil(torch.log2(a)))
                else:
                    a = a.float().double()      # the scale is held in 32 bits
                a[amax == 0] = 1.0
                codes.view(-1, dim_q)[s["slots"], 128 * j:128 * j + 128] = _e4m3(v / a[:, None])
                scale.view(-1, dim_q // 128)[s["slots"], j] = a
        if dim_raw:
            raw = s["raw"].double()
            raw.view(-1, dim_raw)[s["slots"]] = x[:, dim_q:]
        return codes, scale, raw
    batch, page = case["batch"], case["page"]
    dim_q, dim_raw = _widths(case["form"])

    def sequence(b):
        """The cached rows of sequence b in 64 bits."""
        at = torch.arange(int(s["k_len"][b]), device="cuda")
        where, row = s["table"][b].long()[at // page], at % page
        v = torch.empty(len(at), dim_q + dim_raw, device="cuda", dtype=torch.float64)
        for j in range(dim_q // 128):
            cols = slice(128 * j, 128 * j + 128)
            v[:, cols] = s["codes"][where, row][:, cols].double() * s["scale"][where, row, j, None].double()
        if dim_raw:
            v[:, dim_q:] = s["raw"][where, row].double()
        return v, where, row

    if case["op"] == "read":
        if case["form"] == "index":
            codes, scale = s["out"][0].double(), s["out"][1].double()
            for b in range(batch):
                _, where, row = sequence(b)
                codes[b, :len(row)] = s["codes"][where, row].double()
                scale[b, :len(row)] = s["scale"][where, row, 0].double()
            return codes, scale
        out = s["out"].double()
        for b in range(batch):
            v = sequence(b)[0]
            out[b, :len(v)] = v
        return out
    if work(case)["flops"] > 4e12:
        return None
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(batch):
        v = sequence(b)[0]
        tokens = int(s["q_len"][b])
        for t in range(0, tokens, 64):          # 64 queries at a time
            q = s["q"][b, t:min(t + 64, tokens)].double()
            x = torch.einsum("thd,sd->ths", q, v) * SCALE
            last = len(v) - tokens + t + torch.arange(len(q), device="cuda")
            dead = torch.arange(len(v), device="cuda")[None] > last[:, None]
            x = torch.where(dead[:, None], torch.full_like(x, -math.inf), x)
            z = torch.logsumexp(x, -1)
            w = torch.where(dead[:, None], torch.zeros_like(x), torch.exp(x - z[..., None]))
            out[b, t:t + len(q)] = torch.einsum("ths,sd->thd", w, v[:, :LATENT])
            lse[b, t:t + len(q)] = z
    return out, lse
