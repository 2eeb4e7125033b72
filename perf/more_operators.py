"""Positions rotated into the latent-attention layers' queries and rows, and
their cache held in 4 bits, as cases to measure.

    rotate   rotary positions on the last 64 channels of every head's query
    append   the new tokens' rows, normalised and rotated, into the bf16 pages
    store4   the same into pages of 4-bit rows, and every row read back as bf16
             (what a prompt's expansion does with them)
    decode4  attention of one or a few new tokens over the 4-bit pages
    step4    a decode step: queries rotated, the new rows written, attention

A 4-bit row has 416 bytes: 256 of e2m1 codes (512 latent channels, the even one
of a pair in the low half), the 64 shared channels in bf16, and 32 e4m3 scales
(one for 16 channels); a channel stands for its code times its scale.

``run`` computes a case in elementary torch operations in 32 bits (angles in
64), or, where ``own`` is true, by the package's calls.
"""
import math

import torch

own = False

LATENT = 512                 # latent (value) width of a cached row
PE = 64                      # key part shared by the heads: the rotated one
ROW = LATENT + PE
NOPE = 128                   # expanded key width of a head, beside its rotated part
ROW4 = LATENT // 2 + 2 * PE + LATENT // 16
SCALE = (NOPE + PE) ** -0.5
EPS = 1e-6
BASE = 10000.0
BATCH = "512,1024,2048,4096,8192,16384,16384,17408"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step of 64 sequences: their absorbed queries' last part, 96 heads
        dict(name="rotate_step", op="rotate", n=64, lo=700, hi=1024, new=1, heads=96, width=ROW,
             dtype="bf16", interleaved=False, inverse=False),
        # the prompts of the ragged 8-sequence batch, queries of 192 channels, 96 heads
        dict(name="rotate_prompts", op="rotate", n=8, lens=BATCH, new=0, heads=96, width=NOPE + PE,
             dtype="bf16", interleaved=True, inverse=False),
        # one token for each of 64 running sequences: the write of a decode step
        dict(name="append_step", op="append", n=64, lo=700, hi=1024, new=1, page=64, interleaved=False),
        # the batch's prompts written at once
        dict(name="append_prompts", op="append", n=8, lens=BATCH, new=0, page=64, interleaved=True),
        # a few odd prompts kept in 4 bits and read back to be expanded, on short pages
        dict(name="store4_odd", op="store4", n=5, lens="1,77,333,1000,2049", new=0, page=16, norm=True,
             interleaved=False),
        # the batch's prompts, whose latents come normalised
        dict(name="store4_prompts", op="store4", n=8, lens=BATCH, new=0, page=64, norm=False, interleaved=True),
        # one user, a short context, the heads of one of several replicas: latency
        dict(name="decode4_single", op="decode4", n=1, lens="1000", new=1, heads=16, page=64),
        # a decode step of 64 sequences, all 96 heads
        dict(name="decode4_batch", op="decode4", n=64, lo=2000, hi=4096, new=1, heads=96, page=64),
        # few users with long documents: the split over the positions carries it
        dict(name="decode4_long", op="decode4", n=2, lens="131072,100001", new=1, heads=32, page=128),
        # a full serving batch, the largest cache
        dict(name="decode4_full", op="decode4", n=128, lo=8000, hi=8192, new=1, heads=64, page=64),
        # four drafted tokens a sequence, checked in one step, on short pages
        dict(name="decode4_drafts", op="decode4", n=24, lo=100, hi=2100, new=4, heads=16, page=16),
        # all that a layer's decode step does with its cache, 64 running sequences
        dict(name="step4", op="step4", n=64, lo=700, hi=1024, new=1, heads=16, page=64, interleaved=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "store4", "decode4", "decode4", "decode4", "step4"])
    if op == "rotate":
        heads = rng.choice([1, 8, 16, 32, 64, 96])
        n = _log(rng, 1, 64)
        hi = _log(rng, 2, 4_000_000 // (n * heads))
        return dict(op=op, n=n, lo=max(1, hi // rng.randint(1, 8)), hi=hi, new=rng.choice([0, 1, rng.randint(1, 64)]),
                    heads=heads, width=rng.choice([PE, NOPE + PE, ROW]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.25)
    if op in ("append", "store4"):
        n = _log(rng, 1, 64)
        hi = _log(rng, 2, 65536 // n)
        case = dict(op=op, n=n, lo=max(1, hi // rng.randint(1, 8)), hi=hi, new=0, page=rng.choice([16, 32, 64, 128]),
                    interleaved=rng.random() < 0.5)
        if op == "append":
            case["new"] = rng.choice([0, 1, rng.randint(1, 64)])
        else:
            case["norm"] = n * hi <= 4096
        return case
    heads = rng.choice([1, 8, 16, 24, 32, 48, 64, 96, 128])
    new = 1 if op == "step4" else rng.choice([1, 1, 1, rng.randint(2, 9)])
    n = _log(rng, 1, 128)
    most = min(131072, 500_000 // n, 64_000_000 // (n * new * heads))
    hi = _log(rng, 16, max(17, most))
    case = dict(op=op, n=n, lo=max(1, hi // rng.randint(1, 8)), hi=hi, new=new, heads=heads,
                page=rng.choice([16, 32, 64, 128]))
    if op == "step4":
        case["interleaved"] = rng.random() < 0.5
    return case


def _spread(n, lo, hi):
    """n lengths between lo and hi, both of them among n >= 2."""
    return [hi if i == 0 else lo if i == n - 1 else lo + (i * 7919 * 31) % (hi - lo + 1) for i in range(n)]


def _lengths(case):
    if "lens" in case:
        return [int(x) for x in case["lens"].split(",")]
    return _spread(case["n"], case["lo"], case["hi"])


def _news(case, lens):
    """New tokens of each sequence: all of them (0), one, or up to `new`, ragged."""
    if case["new"] == 0:
        return lens
    return [max(1, min(m, case["new"] - (i % 3 if case["new"] > 3 else 0))) for i, m in enumerate(lens)]


def _offsets(lens):
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    return cu


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).to(dev)

    op, lens = case["op"], _lengths(case)
    news = _news(case, lens)
    total = sum(news)
    freq = BASE ** (-torch.arange(0, PE, 2, dtype=torch.float64) / PE)
    s = {"op": op, "n": case["n"], "lens": ints(lens), "cu": ints(_offsets(news)), "max_new": max(news),
         "max_len": max(lens), "single": case["new"] == 1, "interleaved": case.get("interleaved", False),
         "freq": freq.to(dev),
         # the same in whole 2^-64ths of a turn a position
         "turns": (freq / (2 * math.pi) * 2.0 ** 64).to(torch.int64).to(dev)}
    if op == "rotate":
        dtype, W = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32, case["width"]
        s.update(q=normal(total, case["heads"], W, dtype=dtype), inverse=case["inverse"],
                 out=torch.empty((total, case["heads"], W), dtype=dtype, device=dev))
        return s
    # pages of a cache that has served other sequences before: handed out in no order
    page = case["page"]
    pages = [-(-m // page) for m in lens]
    P = sum(pages) + 3
    perm = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
    width = max(pages) + 1
    rows = torch.arange(width, device=dev)[None, :]
    first = torch.tensor(_offsets(pages)[:-1], device=dev)[:, None]
    count = torch.tensor(pages, device=dev)[:, None]
    s["table"] = torch.where(rows < count, perm[(first + rows).clamp(max=P - 1)], -1).to(torch.int32).contiguous()
    s["page"] = page
    if op == "append":
        s.update(cache=normal(P, page, ROW), x=normal(total, ROW) * 1.5, norm_w=1 + 0.1 * normal(LATENT, dtype=torch.float32))
        return s
    s["cache"] = torch.cat([_pack(normal(min(65536, P * page - a), ROW)) for a in range(0, P * page, 65536)]).view(P, page, ROW4)
    if op == "store4":
        s.update(x=normal(total, ROW), norm_w=1 + 0.1 * normal(LATENT, dtype=torch.float32) if case["norm"] else None,
                 out=torch.empty((total, ROW), dtype=torch.bfloat16, device=dev))
        return s
    H = case["heads"]
    s.update(q=normal(total, H, ROW), o=torch.empty((total, H, LATENT), dtype=torch.bfloat16, device=dev),
             lse=torch.empty((total, H), dtype=torch.float32, device=dev))
    if op == "step4":
        # the queries as they are projected, and their absorbed form, whose last part is to be written
        s.update(x=normal(total, ROW), raw=normal(total, H, NOPE + PE))
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _own(state)
    return {"rotate": _rotate, "append": _append, "store4": _store4, "decode4": _decode4, "step4": _step4}[state["op"]](state)


def _own(s):
    import kda_linear_attention_gb300 as kda
    op, cu = s["op"], None if s["single"] else s["cu"]
    if op == "rotate":
        return kda.latent_rotate(s["q"][..., -PE:], s["turns"], s["lens"], cu, out=s["out"][..., -PE:],
                                 interleaved=s["interleaved"], inverse=s["inverse"])
    if op == "append":
        return kda.latent_append_rotated(s["x"], s["cache"], s["table"], s["lens"], s["turns"], cu, norm_w=s["norm_w"],
                                         eps=EPS, interleaved=s["interleaved"])
    if op == "store4":
        kda.latent4_append(s["x"], s["cache"], s["table"], s["lens"], cu, norm_w=s["norm_w"], eps=EPS,
                           turns=s["turns"], interleaved=s["interleaved"])
        return kda.latent4_gather(s["cache"], s["table"], s["cu"], out=s["out"])
    if op == "step4":
        kda.latent_rotate(s["raw"][..., NOPE:], s["turns"], s["lens"], cu, out=s["q"][..., LATENT:],
                          interleaved=s["interleaved"])
        kda.latent4_append(s["x"], s["cache"], s["table"], s["lens"], cu, turns=s["turns"], interleaved=s["interleaved"])
    o, lse = kda.latent4_decode(s["q"], s["cache"], s["table"], s["lens"], cu, scale=SCALE, o=s["o"], lse=s["lse"])
    return (o, lse) if op == "decode4" else (o, lse, _parts(s["cache"]))


def _parts(cache):
    """The three parts of 4-bit rows: codes (two a number), shared channels, scales."""
    a, b = LATENT // 2, LATENT // 2 + 2 * PE
    return cache[..., :a], cache[..., a:b].view(torch.bfloat16), cache[..., b:].view(torch.float8_e4m3fn)


def _pack(x):
    """bf16 rows of 576 as 4-bit rows."""
    c = x[:, :LATENT].float().view(-1, LATENT // 16, 16)
    top = c.abs().amax(2)
    # a quotient by a tensor: by a number it is a product with its rounded inverse, which misses borders
    scale = (top / torch.full_like(top, 6)).clamp(max=448).to(torch.float8_e4m3fn)
    d = scale.float()[..., None]
    y = torch.where(d > 0, c / d, c * 0)
    a = y.abs()
    # the borders between 0, 1/2, 1, 3/2, 2, 3, 4, 6; the even code takes a border itself
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
            + 8 * torch.signbit(c)).to(torch.uint8).view(-1, LATENT // 2, 2)
    return torch.cat([code[..., 0] | code[..., 1] << 4, x[:, LATENT:].contiguous().view(torch.uint8),
                      scale.view(torch.uint8)], 1)


def _unpack(rows):
    """4-bit rows [..., 416] as fp32 [..., 576]."""
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=rows.device)
    value = torch.cat([mag, -mag])
    pair = torch.arange(256, device=rows.device)
    pair = torch.stack([value[pair & 15], value[pair >> 4]], 1)
    code, pe, scale = _parts(rows)
    c = pair[code.long()].view(rows.shape[:-1] + (LATENT // 16, 16)) * scale.float()[..., None]
    return torch.cat([c.flatten(-2), pe.float()], -1)


def _owner(cu, total):
    """The sequence of each packed token, and the token's place in it."""
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu.long(), t, right=True) - 1
    return b, t - cu.long()[b]


def _positions(s, total):
    cu = s["cu"].long()
    b, i = _owner(s["cu"], total)
    return b, s["lens"].long()[b] - (cu[b + 1] - cu[b]) + i


def _turn(s, x, pos, inverse=False):
    """x [T, ..., 64] in 32 bits, rotated by its tokens' positions."""
    angle = pos.double()[:, None] * s["freq"]
    c, d = angle.cos().float(), angle.sin().float()
    c, d = (v.view(v.shape[:1] + (1,) * (x.dim() - 2) + v.shape[1:]) for v in (c, -d if inverse else d))
    x = x.float()
    if s["interleaved"]:
        u, v = x[..., ::2], x[..., 1::2]
        return torch.stack([u * c - v * d, v * c + u * d], -1).flatten(-2)
    u, v = x[..., :PE // 2], x[..., PE // 2:]
    return torch.cat([u * c - v * d, v * c + u * d], -1)


def _rotate(s):
    x = s["q"][..., -PE:]
    return _turn(s, x, _positions(s, x.shape[0])[1], s["inverse"]).to(x.dtype)


def _rows(s):
    """The new tokens' bf16 rows, and where in the cache they go."""
    b, pos = _positions(s, s["x"].shape[0])
    at = s["table"].long()[b, pos // s["page"]] * s["page"] + pos % s["page"]
    x = s["x"].float()
    c = x[:, :LATENT]
    if s.get("norm_w") is not None:
        c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * s["norm_w"]
    return torch.cat([c, _turn(s, x[:, LATENT:], pos)], 1).to(torch.bfloat16), at


def _append(s):
    rows, at = _rows(s)
    s["cache"].view(-1, ROW)[at] = rows
    return s["cache"]


def _append4(s):
    rows, at = _rows(s)
    s["cache"].view(-1, ROW4)[at] = _pack(rows)


def _store4(s):
    _append4(s)
    b, pos = _owner(s["cu"], s["x"].shape[0])
    at = s["table"].long()[b, pos // s["page"]] * s["page"] + pos % s["page"]
    return _unpack(s["cache"].view(-1, ROW4)[at]).to(torch.bfloat16)


def _decode4(s):
    q, cu, L = s["q"], s["cu"].long(), s["lens"].long()
    n, H = s["n"], q.shape[1]
    pos = torch.arange(s["max_len"], device=q.device)
    page = s["table"].long()[:, pos // s["page"]].clamp(min=0)
    c = _unpack(s["cache"].view(-1, ROW4)[page * s["page"] + pos % s["page"]])           # [n, positions, 576]
    i = torch.arange(s["max_new"], device=q.device)
    new = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = q[at].float().reshape(n, -1, ROW)                                                # [n, tokens * heads, 576]
    p = torch.matmul(x, c.transpose(1, 2)).mul_(SCALE).view(n, s["max_new"], H, -1)
    seen = (L - new)[:, None] + i + 1
    p.masked_fill_((pos >= seen[:, :, None])[:, :, None, :], -math.inf)
    m = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p = p.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, -1, s["max_len"]), c[:, :, :LATENT]).view(n, s["max_new"], H, LATENT) / z
    b, k = _owner(s["cu"], q.shape[0])
    return o[b, k].to(torch.bfloat16), (m + z.log())[b, k, :, 0]


def _step4(s):
    x = s["raw"][..., NOPE:]
    s["q"][..., LATENT:] = _turn(s, x, _positions(s, x.shape[0])[1]).to(torch.bfloat16)
    _append4(s)
    return _decode4(s) + (_parts(s["cache"]),)


# ------------------------------------------------------------------ what it has to do
def work(case):
    op, lens = case["op"], _lengths(case)
    news = _news(case, lens)
    t = sum(news)
    if op == "rotate":
        rows = t * case["heads"]
        return {"bytes": rows * 2 * PE * (2 if case["dtype"] == "bf16" else 4), "flops": rows * 3 * PE}
    if op == "append":
        return {"bytes": t * 2 * 2 * ROW + 4 * LATENT, "flops": t * (4 * LATENT + 3 * PE)}
    if op == "store4":
        return {"bytes": t * 2 * (2 * ROW + ROW4), "flops": t * (5 * LATENT + 3 * PE)}
    H = case["heads"]
    pairs = sum(k * (m - k) + k * (k + 1) // 2 for m, k in zip(lens, news))
    d = {"bytes": sum(lens) * ROW4 + t * H * (2 * ROW + 2 * LATENT + 4), "flops": 2 * H * pairs * (ROW + LATENT)}
    if op == "step4":
        d["bytes"] += t * (2 * ROW + ROW4 + H * 2 * PE)
        d["flops"] += t * (3 * LATENT + 3 * PE * (H + 1))
    return d


# ------------------------------------------------------------------ the same in 64 bits, from the definitions
def _exact_turn(x, pos, interleaved, inverse=False):
    """One token's x [..., 64] (fp64) as complex numbers times e^{i angle}."""
    i = torch.arange(PE // 2, dtype=torch.float64, device=x.device)
    angle = pos.double()[:, None] * torch.exp(-2 * i / PE * math.log(BASE))
    angle = angle.view(angle.shape[:1] + (1,) * (x.dim() - 2) + angle.shape[1:])
    turn = torch.polar(torch.ones_like(angle), -angle if inverse else angle)
    if interleaved:
        y = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) * turn
        return torch.view_as_real(y).flatten(-2)
    y = torch.complex(x[..., :PE // 2].contiguous(), x[..., PE // 2:].contiguous()) * turn
    return torch.cat([y.real, y.imag], -1)


def _exact_e4m3(x):
    # steps by binary exponent, the subnormal numbers' first
    steps = torch.tensor([2.0 ** (e - 3) for e in range(-6, 9)], dtype=x.dtype, device=x.device)
    step = steps[(torch.frexp(x).exponent.long() + 5).clamp(0, 14)]
    return ((x / step).round() * step).clamp(max=448)


def _exact_codes(c):
    """fp64 latents [..., 512] (of bf16 values) as (values of the codes, scales)."""
    g = c.view(c.shape[:-1] + (LATENT // 16, 16))
    top = g.abs().amax(-1)
    scale = _exact_e4m3(top / torch.full_like(top, 6))
    y = g / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    y = torch.where((scale > 0)[..., None], y, torch.zeros_like(y))
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).to(y.dtype)
    return ((y / step).round() * step).clamp(-6, 6), scale


def _exact_value(rows):
    """4-bit rows [n, 416] as fp64 [n, 576]."""
    code, pe, scale = _parts(rows)
    nib = torch.stack([code % 16, code // 16], 2).view(len(rows), LATENT)
    sign, e, m = 1.0 - 2.0 * (nib // 8).double(), nib // 2 % 4, (nib % 2).double()
    v = sign * torch.where(e == 0, m / 2, (1 + m / 2) * torch.tensor([0.5, 1, 2, 4], device=e.device)[e.long()])
    return torch.cat([v * scale.double().repeat_interleave(16, 1), pe.double()], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, lens, f = case["op"], _lengths(case), torch.float64
    news, dev = _news(case, lens), s["lens"].device
    pos = torch.cat([torch.arange(m - k, m) for m, k in zip(lens, news)]).to(dev)
    if op == "rotate":
        out = torch.empty(s["out"].shape[:2] + (PE,), dtype=f, device=dev)
        for a in range(0, len(pos), 8192):
            out[a:a + 8192] = _exact_turn(s["q"][a:a + 8192, :, -PE:].to(f), pos[a:a + 8192], s["interleaved"], s["inverse"])
        return out
    page, table = case["page"], s["table"].cpu().tolist()
    flat = s["cache"].flatten(0, 1)

    def rows(b, start, stop):
        at = [table[b][p // page] * page + p % page for p in range(start, stop)]
        return torch.tensor(at, dtype=torch.long, device=dev)

    if op != "decode4":
        at = torch.cat([rows(b, m - k, m) for b, (m, k) in enumerate(zip(lens, news))])
        x = s["x"].to(f)
        if s.get("norm_w") is not None:
            norm = (x[:, :LATENT].pow(2).sum(1, keepdim=True) / LATENT + EPS).sqrt()
            x[:, :LATENT] *= s["norm_w"].to(f) / norm
        x[:, LATENT:] = _exact_turn(x[:, LATENT:], pos, s["interleaved"])
    if op == "append":
        want = flat.to(f)
        want[at] = x
        return want.view(s["cache"].shape)
    if op == "store4":
        value, scale = _exact_codes(x[:, :LATENT].to(torch.bfloat16).to(f))
        return torch.cat([(value * scale[..., None]).flatten(1), x[:, LATENT:]], 1)
    q = s["q"].to(f)
    cached = lambda b, m: _exact_value(flat[rows(b, 0, m)])  # noqa: E731
    state = None
    if op == "step4":
        q[..., LATENT:] = _exact_turn(s["raw"][..., NOPE:].to(f), pos, s["interleaved"]).to(torch.bfloat16).to(f)
        value, scale = _exact_codes(x[:, :LATENT])
        new = torch.cat([(value * scale[..., None]).flatten(1), x[:, LATENT:].to(torch.bfloat16).to(f)], 1)
        pe, d = (t.to(f) for t in _parts(flat)[1:])
        pe[at], d[at] = x[:, LATENT:], scale
        state = (None, pe.view(s["cache"].shape[:2] + (PE,)), d.view(s["cache"].shape[:2] + (LATENT // 16,)))
    o, lse, a = s["o"].to(f), s["lse"].to(f), 0
    for b, (m, k) in enumerate(zip(lens, news)):
        c = cached(b, m)
        if op == "step4":
            c[m - k:] = new[a:a + k]
        for i in range(k):
            past = c[:m - k + i + 1]
            w = q[a + i] @ past.T * SCALE
            lse[a + i] = torch.logsumexp(w, 1)
            o[a + i] = torch.softmax(w, 1) @ past[:, :LATENT]
        a += k
    return (o, lse) if state is None else (o, lse, state)
