"""The latent-attention operators, as cases to measure.

A latent-attention layer keeps one 576-wide row a token (a 512-wide latent
and a 64-wide key part that all heads share) in a paged cache.  Its serving
path is four calls:

    append   the new tokens' rows, normalised, into the cache's pages
    gather   the cached rows of each sequence, in order (to be expanded)
    decode   attention of one or a few new tokens over the pages, in latent
             space (queries and outputs absorbed into the latent)
    prefill  causal attention of many new tokens with expanded keys and values

``run`` computes a case in elementary torch operations in 32 bits, or, where
``own`` is true, by the package's calls.
"""
import math

import torch

own = False

LATENT = 512                 # latent (value) width of a cached row
PE = 64                      # key part shared by the heads
ROW = LATENT + PE
NOPE = 128                   # expanded key width of a head, beside its shared part
DV = 128                     # expanded value width of a head
SCALE = (NOPE + PE) ** -0.5
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token for each of 64 running sequences: the write of a decode step
        dict(name="append_step", op="append", n=64, lo=700, hi=1024, new=1, page=64),
        # the prompts of the ragged 8-sequence batch written at once
        dict(name="append_prompts", op="append", n=8, lens="512,1024,2048,4096,8192,16384,16384,17408", new=0, page=64),
        # a few odd contexts read back before a chunk of new tokens is attended to
        dict(name="gather_odd", op="gather", n=5, lens="1,77,333,1000,2049", page=16),
        # the contexts of the 8-sequence batch read back
        dict(name="gather_batch", op="gather", n=8, lens="512,1024,2048,4096,8192,16384,16384,17408", page=64),
        # one user, a short context, the heads of one of several replicas: latency
        dict(name="decode_single", op="decode", n=1, lens="1000", new=1, heads=16, page=64),
        # a decode step of 64 sequences, all 96 heads
        dict(name="decode_batch", op="decode", n=64, lo=2000, hi=4096, new=1, heads=96, page=64),
        # few users with long documents: the split over the positions carries it
        dict(name="decode_long", op="decode", n=2, lens="131072,100001", new=1, heads=32, page=128),
        # a full serving batch, the largest cache
        dict(name="decode_full", op="decode", n=128, lo=8000, hi=8192, new=1, heads=64, page=64),
        # four drafted tokens a sequence, checked in one step, on short pages
        dict(name="decode_drafts", op="decode", n=24, lo=100, hi=2100, new=4, heads=16, page=16),
        # short ragged prompts
        dict(name="prefill_short", op="prefill", n=4, lens="1,33,130,515", ctx=0, heads=16),
        # the 4K prompt at all 96 heads
        dict(name="prefill_4k", op="prefill", n=1, lens="4096", ctx=0, heads=96),
        # a chunk of new tokens behind a context that was prefilled before
        dict(name="prefill_chunk", op="prefill", n=2, lens="1024,1000", ctx=8192, heads=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "prefill", "prefill"])
    if op in ("append", "gather"):
        n = _log(rng, 1, 64)
        hi = _log(rng, 2, 65536 // n)
        case = dict(op=op, n=n, lo=max(1, hi // rng.randint(1, 8)), hi=hi, page=rng.choice([16, 32, 64, 128]))
        if op == "append":
            case["new"] = rng.choice([0, 1, rng.randint(1, 64)])
        return case
    if op == "decode":
        heads = rng.choice([1, 8, 16, 24, 32, 48, 64, 96, 128])
        new = rng.choice([1, 1, 1, rng.randint(2, 9)])
        n = _log(rng, 1, 128)
        most = min(131072, 500_000 // n, 64_000_000 // (n * new * heads))
        hi = _log(rng, 16, max(17, most))
        return dict(op=op, n=n, lo=max(1, hi // rng.randint(1, 8)), hi=hi, new=new, heads=heads,
                    page=rng.choice([16, 32, 64, 128]))
    heads = rng.choice([1, 4, 8, 16, 32, 64, 96])
    n = _log(rng, 1, 16)
    hi = _log(rng, 1, 4096)
    ctx = rng.choice([0, 0, _log(rng, 16, 4096)])
    while hi > 1 and n * heads * hi * (hi + ctx) > 1_500_000_000 or n > 1 and n * heads * (hi + ctx) > 1_000_000:
        hi = max(1, hi // 2)
        n = max(1, n // 2)
    return dict(op=op, n=n, lo=max(1, hi // rng.randint(1, 4)), hi=hi, ctx=ctx, heads=heads)


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

    lens = _lengths(case)
    s = {"op": case["op"], "n": case["n"]}
    if case["op"] == "prefill":
        ctx, H = case["ctx"], case["heads"]
        klens = [m + ctx for m in lens]
        s.update(cu=ints(_offsets(lens)), cu_k=ints(_offsets(klens)), max_q=max(lens), max_k=max(klens),
                 q=normal(sum(lens), H, NOPE + PE), kv=normal(sum(klens), H, NOPE + DV), k_pe=normal(sum(klens), PE),
                 o=torch.empty((sum(lens), H, DV), dtype=torch.bfloat16, device=dev),
                 lse=torch.empty((sum(lens), H), dtype=torch.float32, device=dev))
        return s
    # pages of a cache that has served other sequences before: handed out in no order
    page = case["page"]
    pages = [-(-m // page) for m in lens]
    spare = 3
    perm = torch.randperm(sum(pages) + spare, generator=gen, device=dev).to(torch.int32)
    width = max(pages) + 1
    rows = torch.arange(width, device=dev)[None, :]
    first = torch.tensor(_offsets(pages)[:-1], device=dev)[:, None]
    count = torch.tensor(pages, device=dev)[:, None]
    table = torch.where(rows < count, perm[(first + rows).clamp(max=perm.numel() - 1)], -1).to(torch.int32).contiguous()
    s.update(cache=normal(sum(pages) + spare, page, ROW), table=table, page=page, max_len=max(lens))
    if case["op"] == "gather":
        s.update(cu=ints(_offsets(lens)), out=torch.empty((sum(lens), ROW), dtype=torch.bfloat16, device=dev))
        return s
    news = _news(case, lens)
    s.update(lens=ints(lens), cu=ints(_offsets(news)), max_new=max(news), single=case["new"] == 1)
    if case["op"] == "append":
        s.update(kv=(normal(sum(news), ROW) * 1.5), norm_w=1 + 0.1 * normal(LATENT, dtype=torch.float32))
    else:
        s.update(q=normal(sum(news), case["heads"], ROW),
                 o=torch.empty((sum(news), case["heads"], LATENT), dtype=torch.bfloat16, device=dev),
                 lse=torch.empty((sum(news), case["heads"]), dtype=torch.float32, device=dev))
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _own(state)
    return {"append": _append, "gather": _gather, "decode": _decode, "prefill": _prefill}[state["op"]](state)


def _own(s):
    import kda_linear_attention_gb300 as kda
    if s["op"] == "append":
        return kda.latent_append(s["kv"], s["cache"], s["table"], s["lens"], None if s["single"] else s["cu"],
                                 norm_w=s["norm_w"], eps=EPS)
    if s["op"] == "gather":
        return kda.latent_gather(s["cache"], s["table"], s["cu"], out=s["out"])
    if s["op"] == "decode":
        return kda.latent_decode(s["q"], s["cache"], s["table"], s["lens"], None if s["single"] else s["cu"],
                                 scale=SCALE, o=s["o"], lse=s["lse"])
    return kda.latent_prefill(s["q"], s["kv"], s["k_pe"], s["cu"], s["cu_k"], scale=SCALE, o=s["o"], lse=s["lse"])


def _owner(cu, total):
    """The sequence of each packed token, and the token's place in it."""
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu.long(), t, right=True) - 1
    return b, t - cu.long()[b]


def _append(s):
    cu, cache = s["cu"].long(), s["cache"]
    b, i = _owner(s["cu"], s["kv"].shape[0])
    pos = s["lens"].long()[b] - (cu[b + 1] - cu[b]) + i
    row = s["table"].long()[b, pos // s["page"]] * s["page"] + pos % s["page"]
    x = s["kv"].float()
    c = x[:, :LATENT]
    c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * s["norm_w"]
    cache.view(-1, ROW)[row] = torch.cat([c, x[:, LATENT:]], 1).to(torch.bfloat16)
    return cache


def _gather(s):
    b, pos = _owner(s["cu"], s["out"].shape[0])
    row = s["table"].long()[b, pos // s["page"]] * s["page"] + pos % s["page"]
    return s["cache"].view(-1, ROW)[row]


def _decode(s):
    q, cu, L = s["q"], s["cu"].long(), s["lens"].long()
    n, H = s["n"], q.shape[1]
    pos = torch.arange(s["max_len"], device=q.device)
    page = s["table"].long()[:, pos // s["page"]].clamp(min=0)
    c = s["cache"].view(-1, ROW)[page * s["page"] + pos % s["page"]].float()             # [n, positions, 576]
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


def _prefill(s):
    q, cu, cu_k = s["q"], s["cu"].long(), s["cu_k"].long()
    n, H = s["n"], q.shape[1]
    i = torch.arange(s["max_q"], device=q.device)
    j = torch.arange(s["max_k"], device=q.device)
    x = q[(cu[:-1, None] + i).clamp(max=q.shape[0] - 1)].float().transpose(1, 2)         # [n, H, queries, 192]
    at = (cu_k[:-1, None] + j).clamp(max=s["kv"].shape[0] - 1)
    kv = s["kv"][at].float().transpose(1, 2)                                             # [n, H, keys, 256]
    pe = s["k_pe"][at].float()[:, None]                                                  # [n, 1, keys, 64]
    p = torch.matmul(x[..., :NOPE], kv[..., :NOPE].transpose(2, 3))
    p = p.add_(torch.matmul(x[..., NOPE:], pe.transpose(2, 3))).mul_(SCALE)
    nq, nk = cu[1:] - cu[:-1], cu_k[1:] - cu_k[:-1]
    seen = (nk - nq)[:, None] + i + 1
    p.masked_fill_((j >= seen[:, :, None])[:, None], -math.inf)
    m = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p = p.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[..., NOPE:]) / z
    b, k = _owner(s["cu"], q.shape[0])
    return o[b, :, k].to(torch.bfloat16), (m + z.log())[b, :, k, 0]


# ------------------------------------------------------------------ what it has to do
def work(case):
    lens = _lengths(case)
    if case["op"] == "prefill":
        H, ctx = case["heads"], case["ctx"]
        tq, tk = sum(lens), sum(lens) + ctx * len(lens)
        pairs = sum(m * ctx + m * (m + 1) // 2 for m in lens)
        return {"bytes": tq * H * (2 * (NOPE + PE + DV) + 4) + tk * (2 * H * (NOPE + DV) + 2 * PE),
                "flops": 2 * H * pairs * (NOPE + PE + DV)}
    if case["op"] == "gather":
        return {"bytes": 2 * sum(lens) * 2 * ROW, "flops": 0}
    news = _news(case, lens)
    if case["op"] == "append":
        return {"bytes": 2 * sum(news) * 2 * ROW + 4 * LATENT, "flops": 4 * LATENT * sum(news)}
    H = case["heads"]
    pairs = sum(k * (m - k) + k * (k + 1) // 2 for m, k in zip(lens, news))
    return {"bytes": sum(lens) * 2 * ROW + sum(news) * H * (2 * ROW + 2 * LATENT + 4),
            "flops": 2 * H * pairs * (ROW + LATENT)}


def exact(case, seed):
    s = prepare(case, seed)
    lens, f = _lengths(case), torch.float64
    if case["op"] == "prefill":
        H, ctx = case["heads"], case["ctx"]
        o, lse = s["o"].to(f), s["lse"].to(f)
        a = c = 0
        for m in lens:
            keys, pe = s["kv"][c:c + m + ctx], s["k_pe"][c:c + m + ctx].to(f)
            hidden = torch.ones((m, m + ctx), dtype=torch.bool, device=pe.device).triu(ctx + 1)
            for h in range(H):
                k = torch.cat([keys[:, h, :NOPE].to(f), pe], 1)
                w = (s["q"][a:a + m, h].to(f) @ k.T * SCALE).masked_fill_(hidden, -math.inf)
                lse[a:a + m, h] = torch.logsumexp(w, 1)
                o[a:a + m, h] = torch.softmax(w, 1) @ keys[:, h, NOPE:].to(f)
            a, c = a + m, c + m + ctx
        return o, lse
    page, flat = case["page"], s["cache"].view(-1, ROW)
    table = s["table"].cpu().tolist()

    def rows(b, start, stop):
        at = [table[b][p // page] * page + p % page for p in range(start, stop)]
        return torch.tensor(at, dtype=torch.long, device=flat.device)

    if case["op"] == "gather":
        return torch.cat([flat[rows(b, 0, m)] for b, m in enumerate(lens)]).to(f)
    news = _news(case, lens)
    if case["op"] == "append":
        want, a = flat.to(f), 0
        for b, (m, k) in enumerate(zip(lens, news)):
            x = s["kv"][a:a + k].to(f)
            norm = (x[:, :LATENT].pow(2).sum(1, keepdim=True) / LATENT + EPS).sqrt()
            x[:, :LATENT] *= s["norm_w"].to(f) / norm
            want[rows(b, m - k, m)] = x
            a += k
        return want.view(s["cache"].shape)
    o, lse, a = s["o"].to(f), s["lse"].to(f), 0
    for b, (m, k) in enumerate(zip(lens, news)):
        x = flat[rows(b, 0, m)].to(f)
        for i in range(k):
            past = x[:m - k + i + 1]
            w = s["q"][a + i].to(f) @ past.T * SCALE
            lse[a + i] = torch.logsumexp(w, 1)
            o[a + i] = torch.softmax(w, 1) @ past[:, :LATENT]
        a += k
    return o, lse
