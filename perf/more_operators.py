"""What is measured of the operators around a K/V cache held in 8 bits.

Four operators: attention of a drafted tree over paged e4m3 K/V with a scale
for each block of tokens and head, the commit of the accepted path into such a
cache, the append of prompts to it, and the pages' forking, freeing and
compaction.  Each case is one call (or, where it says so, the calls of one
step) on inputs made from a seed.  `own` False: the operator in elementary
torch operations; True: the library's kernels.
"""
from __future__ import annotations

import math

import torch

own = False

VOCAB = 151936
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
MOST = 448.0  # e4m3's largest value


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request's block of 16 nodes on a short context: the latency of one layer
        dict(name="attend8_1x16_ctx1000", op="attend", N=1, T=16, Hkv=8, g=4, D=128, ctx=1000, page=64, block=16,
             dtype="bf16", heads_first=False),
        # a batch of 32 requests, blocks of 16 nodes, ragged contexts up to 8000 tokens, small pages
        dict(name="attend8_32x16_ctx8000", op="attend", N=32, T=16, Hkv=8, g=4, D=128, ctx=8000, page=16, block=16,
             dtype="bf16", heads_first=False),
        # wide trees of 64 nodes, five query heads a K/V head, long contexts, head-major pages
        dict(name="attend8_8x64_ctx32000", op="attend", N=8, T=64, Hkv=8, g=5, D=128, ctx=32000, page=64, block=64,
             dtype="bf16", heads_first=True),
        # single-token decoding on long contexts, fp16
        dict(name="attend8_48x1_ctx24001", op="attend", N=48, T=1, Hkv=8, g=4, D=128, ctx=24001, page=32, block=32,
             dtype="fp16", heads_first=False),
        # a short piece of one prompt, onto a partly filled block
        dict(name="append_1x100", op="append", N=1, tokens=100, L=16, Hkv=8, D=128, page=64, block=32, dtype="bf16"),
        # a batch of ragged prompts, head width 64
        dict(name="append_8x2000", op="append", N=8, tokens=2000, L=16, Hkv=8, D=64, page=64, block=64, dtype="fp16"),
        # one request's accepted path into the caches of 16 layers
        dict(name="commit8_1x16", op="commit", N=1, T=16, L=16, Hkv=8, D=128, page=64, block=32, dtype="bf16"),
        # 32 requests with trees of 64 nodes
        dict(name="commit8_32x64", op="commit", N=32, T=64, L=16, Hkv=8, D=128, page=16, block=16, dtype="bf16"),
        # one request branches once: its last page is copied, the others are shared
        dict(name="fork_1", op="fork", rows=8, forks=1, ctx=1000, L=16, Hkv=8, D=128, page=64, block=64, pages=512),
        # a search step over 64 rows: 48 are freed and forked anew from the other 16
        dict(name="fork_48", op="fork", rows=64, forks=48, ctx=8000, L=16, Hkv=8, D=128, page=16, block=16, pages=8200),
        # a small pool with few holes
        dict(name="compact_200", op="compact", rows=8, pages=200, used=0.9, L=4, Hkv=8, D=128, page=64, block=32,
             shared=False),
        # half of a large pool is free, pages are shared by several rows
        dict(name="compact_8001", op="compact", rows=64, pages=8001, used=0.5, L=8, Hkv=8, D=128, page=16, block=16,
             shared=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _layout(rng):
    page = rng.choice([16, 32, 64, 128])
    return dict(Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=page,
                block=rng.choice([b for b in (16, 32, 64, 128) if b <= page]))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "commit", "fork", "compact"])
    while True:
        c = dict(op=op, **_layout(rng))
        if op == "attend":
            c.update(N=_log_int(rng, 1, 64), T=_log_int(rng, 1, 64), g=rng.choice([1, 2, 4, 5, 8]),
                     ctx=_log_int(rng, 1, 32000), dtype=rng.choice(["bf16", "fp16"]), heads_first=rng.random() < 0.5)
            if c["N"] * c["ctx"] * c["Hkv"] * c["D"] <= 48 * 24001 * 8 * 128 and \
                    c["N"] * c["ctx"] * c["Hkv"] * c["g"] * c["T"] * c["D"] <= 8 * 32000 * 40 * 64 * 128:
                return c
        elif op == "append":
            c.update(N=_log_int(rng, 1, 32), tokens=_log_int(rng, 1, 4000), L=_log_int(rng, 1, 16),
                     dtype=rng.choice(["bf16", "fp16"]))
            if c["N"] * c["tokens"] * c["L"] * c["Hkv"] * c["D"] <= 8 * 2000 * 16 * 8 * 64:
                return c
        elif op == "commit":
            c.update(N=_log_int(rng, 1, 32), T=_log_int(rng, 1, 64), L=_log_int(rng, 1, 16),
                     dtype=rng.choice(["bf16", "fp16"]))
            return c
        elif op == "fork":
            rows = _log_int(rng, 2, 64)
            c.update(rows=rows, forks=rng.randint(1, rows - 1), ctx=_log_int(rng, 1, 8000), L=_log_int(rng, 1, 16))
            c["pages"] = c["forks"] + rng.randint(0, 50) + (rows - c["forks"]) * -(-c["ctx"] // c["page"])
            if c["pages"] * c["page"] * c["Hkv"] * c["D"] * c["L"] <= 8200 * 16 * 8 * 128 * 16:
                return c
        else:
            c.update(rows=_log_int(rng, 1, 64), pages=_log_int(rng, 8, 8001), used=rng.uniform(0.1, 1.0),
                     L=_log_int(rng, 1, 8), shared=rng.random() < 0.5)
            if c["pages"] * c["page"] * c["Hkv"] * c["D"] * c["L"] <= 8001 * 16 * 8 * 128 * 8:
                return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) % (1 << 30)) + 29)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _empty(*shape, dtype=torch.int32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _cache(g, c, pages, layers=None, heads_first=False):
    """Payload e4m3 [pages, page, heads, D] (layers in front where given) and scales [pages, blocks, heads]: values
    of the order of one, with scales of 2^-8 to 2^-6 by block and head."""
    lead = () if layers is None else (layers,)
    inner = (c["Hkv"], c["page"], c["D"]) if heads_first else (c["page"], c["Hkv"], c["D"])
    x = torch.randn(*lead, pages, *inner, generator=g, device="cuda", dtype=torch.float16)
    x = x.mul_(110).clamp_(-MOST, MOST).to(E4M3)
    e = torch.randint(-8, -5, (*lead, pages, c["page"] // c["block"], c["Hkv"]), generator=g, device="cuda")
    return (x.transpose(-3, -2) if heads_first else x), torch.exp2(e.float())


def _tree(g, N, T):
    """Random trees: parents [N, T] (node 0 the root), and who is whose ancestor (or self), [N, T, T]."""
    pick = _rand(g, N, T)
    at = torch.arange(T, device="cuda")
    parents = torch.maximum((pick * at).long(), at - 4).clamp_(max=T - 1)  # one of the four nodes before it
    parents = torch.minimum(parents, (at - 1).clamp(min=0))
    anc = torch.eye(T, dtype=torch.bool, device="cuda").repeat(N, 1, 1)
    for t in range(1, T):
        anc[:, t] |= anc.gather(1, parents[:, t].view(N, 1, 1).expand(N, 1, T))[:, 0]
    parents[:, 0] = -1
    return parents.to(torch.int32), anc


def _bits(anc):
    N, T, _ = anc.shape
    W = -(-T // 32)
    pad = torch.zeros(N, T, W * 32, dtype=torch.int64, device="cuda")
    pad[..., :T] = anc
    words = (pad.view(N, T, W, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).contiguous()


_handles = {}


def _handle(N, T, g, width, c):
    """The plan a serving program keeps for a model: one handle a configuration."""
    import draft_correction_slot_gb300 as dc
    key = (N, T, g, width, c["Hkv"], c["D"], c["page"], c["block"], c["dtype"])
    if key not in _handles:
        _handles[key] = dc.dcoco_tree_create_quant(
            max_batch=N, max_tree=T, q_heads=c["Hkv"] * g, kv_heads=c["Hkv"], head_dim=c["D"], page_size=c["page"],
            max_pages=width, scale_tokens=c["block"], dtype=DT[c["dtype"]])
    return _handles[key]


def _pool(c, width):
    import draft_correction_slot_gb300 as dc
    key = (c["pages"], c["page"], width, c["rows"])
    if key not in _handles:
        _handles[key] = dc.dcoco_pages_create(num_pages=c["pages"], page_size=c["page"], max_pages=width,
                                              max_rows=c["rows"])
    return _handles[key]


def _prepare_attend(c, g):
    N, T, H, G, D, page, dt = c["N"], c["T"], c["Hkv"], c["g"], c["D"], c["page"], DT[c["dtype"]]
    # contexts between an eighth of the longest and the longest, one of them the longest
    ctx = (c["ctx"] * (0.125 + 0.875 * _rand(g, N))).long().clamp(min=1)
    ctx[0] = c["ctx"]
    width = -(-(c["ctx"] + T) // page)
    need = (ctx + T + page - 1) // page
    total = N * width
    table = torch.randperm(total, generator=g, device="cuda").view(N, width).to(torch.int32)
    table = torch.where(torch.arange(width, device="cuda") < need[:, None], table, torch.zeros_like(table))
    k, ks = _cache(g, c, total, heads_first=c["heads_first"])
    v, vs = _cache(g, c, total, heads_first=c["heads_first"])
    # q, k and v of the nodes leave one projection: views of one buffer, as a model has them
    qkv = _randn(g, N, T, (G + 2) * H, D).to(dt)
    _, anc = _tree(g, N, T)
    s = dict(c=c, q=qkv[:, :, :G * H], k_new=qkv[:, :, G * H:G * H + H], v_new=qkv[:, :, G * H + H:],
             k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, table=table, ctx=ctx.to(torch.int32), anc=anc,
             bits=_bits(anc), out=_empty(N, T, G * H, D, dtype=dt), lse=_empty(N, T, G * H, dtype=torch.float32))
    if own:
        s["handle"] = _handle(N, T, G, width, c)
    return s


def _prepare_append(c, g):
    N, page = c["N"], c["page"]
    # prompts between an eighth of the longest and the longest behind up to two pages of context
    count = (c["tokens"] * (0.125 + 0.875 * _rand(g, N))).long().clamp(min=1)
    count[0] = c["tokens"]
    first = torch.cat([count.new_zeros(1), count.cumsum(0)])
    total = int(first[-1])
    ctx = (2 * page * _rand(g, N)).to(torch.int32)
    width = -(-(2 * page + c["tokens"]) // page)
    table = torch.randperm(N * width, generator=g, device="cuda").view(N, width).to(torch.int32)
    k, ks = _cache(g, c, N * width, c["L"])
    v, vs = _cache(g, c, N * width, c["L"])
    new = [torch.randn(c["L"], total, c["Hkv"], c["D"], generator=g, device="cuda", dtype=DT[c["dtype"]]) for _ in "kv"]
    s = dict(c=c, k_new=new[0], v_new=new[1], k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, table=table, ctx=ctx,
             first=first.to(torch.int32), new_len=_empty(N))
    if own:
        s["handle"] = _handle(N, 1, 1, width, c)
    return s


def _prepare_commit(c, g):
    N, T, L, page = c["N"], c["T"], c["L"], c["page"]
    width = -(-(2 * page + T) // page)  # two pages of context at most, then the tree
    ctx = (2 * page * _rand(g, N)).to(torch.int32)
    table = torch.randperm(N * width, generator=g, device="cuda").view(N, width).to(torch.int32)
    k, ks = _cache(g, c, N * width, L)
    v, vs = _cache(g, c, N * width, L)
    new = [torch.randn(L, N, T, c["Hkv"], c["D"], generator=g, device="cuda", dtype=DT[c["dtype"]]) for _ in "kv"]
    parents, anc = _tree(g, N, T)
    tokens = torch.randint(0, VOCAB, (N, T), generator=g, device="cuda", dtype=torch.int32)
    # the target agrees with the last child of most nodes
    at = torch.arange(T, device="cuda")
    child = torch.where(parents[:, None, :] == at[:, None], at, -1).amax(2)
    agree = (child >= 0) & (_rand(g, N, T) < 0.8)
    other = torch.randint(0, VOCAB, (N, T), generator=g, device="cuda", dtype=torch.int32)
    sampled = torch.where(agree, tokens.gather(1, child.clamp(min=0)), other)
    s = dict(c=c, k_new=new[0], v_new=new[1], k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, table=table, ctx=ctx,
             parents=parents, anc=anc, tokens=tokens, sampled=sampled, path=_empty(N, T), accept_len=_empty(N),
             next_token=_empty(N), new_len=_empty(N))
    if own:
        s["handle"] = _handle(N, T, 1, width, c)
    return s


def _planes(s):
    import draft_correction_slot_gb300 as dc
    return dc.page_planes([s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")])


def _prepare_fork(c, g):
    rows, forks, page = c["rows"], c["forks"], c["page"]
    order = torch.randperm(rows, generator=g, device="cuda")
    dst, base = order[:forks], order[forks:]  # the rows forked into; the others hold sequences
    width = -(-c["ctx"] // page)
    lens = torch.zeros(rows, dtype=torch.int64, device="cuda")
    lens[base] = (c["ctx"] * (0.125 + 0.875 * _rand(g, rows - forks))).long().clamp(min=1)
    lens[base[0]] = c["ctx"]
    held = (lens + page - 1) // page
    have = torch.arange(width, device="cuda") < held[:, None]
    ids = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)
    at = have.view(-1).cumsum(0).view(rows, width) - 1
    table = torch.where(have, ids[at.clamp(min=0)], torch.zeros_like(at, dtype=torch.int32))
    refs = torch.zeros(c["pages"], dtype=torch.int32, device="cuda")
    refs[table[have].long()] = 1
    k, ks = _cache(g, c, c["pages"], c["L"])
    v, vs = _cache(g, c, c["pages"], c["L"])
    src = base[torch.randint(0, rows - forks, (forks,), generator=g, device="cuda")]
    s = dict(c=c, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, table=table, lens=lens.to(torch.int32),
             held=held.to(torch.int32), refs=refs, src=src.to(torch.int32), dst=dst.to(torch.int32))
    if own:
        s["handle"], s["planes"] = _pool(c, width), _planes(s)
    return s


def _prepare_compact(c, g):
    rows, pages, page = c["rows"], c["pages"], c["page"]
    count = max(1, int(c["used"] * pages))
    used = torch.randperm(pages, generator=g, device="cuda")[:count].to(torch.int32)
    # the pages in use dealt to the rows in turn; where pages are shared a row begins with the first row's pages
    width = -(-count // rows) * 2
    held = (count - torch.arange(rows, device="cuda") + rows - 1) // rows
    at = torch.arange(rows, device="cuda")[:, None] + rows * torch.arange(width, device="cuda")
    have = torch.arange(width, device="cuda") < held[:, None]
    table = torch.where(have, used[at.clamp(max=count - 1)], -1)
    if c["shared"]:
        table[1:, :width // 2] = torch.where(have[1:, :width // 2] & (_rand(g, rows - 1, 1) < 0.5), table[:1, :width // 2],
                                             table[1:, :width // 2])
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    own_pages = table[have].long()
    refs.index_add_(0, own_pages, torch.ones_like(own_pages, dtype=torch.int32))
    k, ks = _cache(g, c, pages, c["L"])
    v, vs = _cache(g, c, pages, c["L"])
    s = dict(c=c, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, table=table, held=held.to(torch.int32), refs=refs,
             table_out=table.clone(), refs_out=refs.clone(), live=_empty(1))
    if own:
        s["handle"], s["planes"] = _pool(c, width), _planes(s)
    return s


def prepare(case, seed):
    g = _gen(seed)
    return {"attend": _prepare_attend, "append": _prepare_append, "commit": _prepare_commit, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, g)


# ------------------------------------------------------------------ plain forms
def _values(payload, scale, table, block):
    """The values of the tokens of the table's pages, [N, tokens, heads, D], in fp32."""
    N = table.shape[0]
    x = payload.view(torch.uint8)[table].view(E4M3).float()
    x = x * scale[table].repeat_interleave(block, 2)[..., None]
    return x.reshape(N, -1, *x.shape[3:])


def _plain_attend(s):
    c = s["c"]
    N, T, H, G, D = c["N"], c["T"], c["Hkv"], c["g"], c["D"]
    table = s["table"].long()
    S = table.shape[1] * c["page"]
    seen = torch.arange(S, device="cuda") < s["ctx"][:, None]
    zero = torch.zeros((), device="cuda")
    k = torch.cat([_values(s["k_cache"], s["k_scale"], table, c["block"]), s["k_new"].float()], 1)
    v = torch.cat([_values(s["v_cache"], s["v_scale"], table, c["block"]), s["v_new"].float()], 1)
    v = torch.where(torch.cat([seen, torch.ones(N, T, dtype=torch.bool, device="cuda")], 1)[:, :, None, None], v, zero)
    mask = torch.cat([seen[:, None].expand(N, T, S), s["anc"]], 2)  # [N, T, S + T]
    q = s["q"].float().view(N, T, H, G, D).permute(0, 2, 3, 1, 4).reshape(N, H, G * T, D)
    a = (q @ k.permute(0, 2, 3, 1)).view(N, H, G, T, S + T) / math.sqrt(D)
    a = torch.where(mask[:, None, None], a, zero - math.inf)
    m = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(m == -math.inf, zero, m))
    total = p.sum(-1, keepdim=True)
    o = (p.view(N, H, G * T, S + T) @ v.permute(0, 2, 1, 3)).view(N, H, G, T, D) / torch.where(total == 0, zero + 1, total)
    out = o.permute(0, 3, 1, 2, 4).reshape(N, T, H * G, D).to(s["q"].dtype)
    lse = (m + torch.log(total)).view(N, H, G, T).permute(0, 3, 1, 2).reshape(N, T, H * G)
    return {"out": out, "lse": lse}


def _least_scale(most):
    """The least power of two with most <= 448 times it, within 2^-64 .. 2^64."""
    m, e = torch.frexp(most)  # most = m 2^e, m in [0.5, 1): 448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.exp2(torch.where(most > 0, e, -64).clamp(-64, 64).float())


def _plain_write(s, name, n, pos, rows):
    """K or V of tokens at positions `pos` of requests `n` [tokens], from rows [L, tokens, heads, D]."""
    c = s["c"]
    page, block = c["page"], c["block"]
    cache, scale = s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
    pg, slot = s["table"].long()[n, pos // page], pos % page
    blocks = scale.shape[2]
    at = pg * blocks + slot // block  # the tokens' blocks among all of the pool's
    flat = scale.reshape(scale.shape[0], -1, scale.shape[3])  # [L, pages * blocks, heads]
    x = rows.float()
    zero = torch.zeros_like(flat)
    most = zero.index_reduce(1, at, x.abs().amax(3), "amax")
    first = pos // block * block  # a block has old tokens where it begins before the context's end
    ctx = s["ctx"].long()[n]
    old = (ctx - first).clamp(min=0)  # of each token's block
    count = torch.zeros(flat.shape[1], dtype=torch.int64, device="cuda").scatter(0, at, old)
    hit = torch.zeros(flat.shape[1], dtype=torch.bool, device="cuda").index_fill(0, at, True)
    need = _least_scale(most)
    now = torch.where((count > 0)[:, None], torch.maximum(flat, need), need)
    now = torch.where(hit[:, None], now, flat)
    # old tokens of the blocks whose scale has changed
    which = torch.unique(at)
    p8 = cache.view(E4M3)[:, which // blocks].float().view(x.shape[0], -1, blocks, block, *cache.shape[3:])
    i = torch.arange(which.numel(), device="cuda")
    p8 = p8[:, i, which % blocks]  # [L, hit blocks, block, heads, D]
    ratio = (flat[:, which] / now[:, which])[:, :, None, :, None]
    again = torch.where(torch.arange(block, device="cuda")[:, None, None] < count[which][:, None, None, None], p8 * ratio, p8)
    t = (which % blocks * block)[:, None] + torch.arange(block, device="cuda")
    cache[:, (which // blocks)[:, None], t] = again.to(E4M3).view(torch.uint8)
    cache[:, pg, slot] = (x / now[:, at][..., None]).clamp(-MOST, MOST).to(E4M3).view(torch.uint8)
    scale.copy_(now.view_as(scale))


def _plain_append(s):
    c = s["c"]
    first, ctx = s["first"].long(), s["ctx"].long()
    t = torch.arange(s["k_new"].shape[1], device="cuda")
    n = torch.searchsorted(first, t, right=True) - 1
    pos = ctx[n] + t - first[n]
    _plain_write(s, "k", n, pos, s["k_new"])
    _plain_write(s, "v", n, pos, s["v_new"])
    return {"new_len": (ctx + first[1:] - first[:-1]).to(torch.int32), "k_cache": s["k_cache"], "v_cache": s["v_cache"],
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_commit(s):
    c = s["c"]
    N, T = c["N"], c["T"]
    tokens, parents = s["tokens"], s["parents"].long()
    up = parents.clamp(min=0)
    same = (parents[:, :, None] == parents[:, None]) & (tokens[:, :, None] == tokens[:, None])
    later = torch.tril(torch.ones(T, T, dtype=torch.bool, device="cuda"), -1)
    first = ~(same & later).any(2)  # no earlier sibling with the same token
    match = (tokens == s["sampled"].gather(1, up)) & first | (parents < 0)
    taken = (match[:, None] | ~s["anc"]).all(2)  # the node and all its ancestors agree
    count = taken.sum(1)
    rank = torch.cumsum(taken, 1) - 1
    node = torch.arange(T, device="cuda").expand(N, T)
    path = torch.sort(torch.where(taken, node, T), 1).values
    last = path.gather(1, (count - 1)[:, None])
    n, t = taken.nonzero(as_tuple=True)
    pos = s["ctx"].long()[n] + rank[n, t]
    _plain_write(s, "k", n, pos, s["k_new"][:, n, t])
    _plain_write(s, "v", n, pos, s["v_new"][:, n, t])
    return {"path": torch.where(path == T, -1, path).to(torch.int32), "accept_len": (count - 1).to(torch.int32),
            "next_token": s["sampled"].gather(1, last)[:, 0], "new_len": (s["ctx"] + count).to(torch.int32),
            "k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _move(s, src, dst):
    for name in ("k_cache", "v_cache"):
        x = s[name].view(torch.uint8)
        x[:, dst] = x[:, src]
    for name in ("k_scale", "v_scale"):
        s[name][:, dst] = s[name][:, src]


def _pool_state(s):
    return {k: s[k] for k in ("table", "held", "lens", "refs", "k_cache", "v_cache", "k_scale", "v_scale")}


def _plain_fork(s):
    c = s["c"]
    page, src, dst = c["page"], s["src"].long(), s["dst"].long()
    table, held, lens, refs = s["table"], s["held"], s["lens"], s["refs"]
    col = torch.arange(table.shape[1], device="cuda")
    # the rows forked into are freed first
    gone = table[dst][col < held[dst][:, None]].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    n = lens[src].long()
    full, part = n // page, n % page > 0
    fresh = (refs == 0).nonzero()[:, 0][:c["forks"]].to(torch.int32)
    fresh = fresh[(part.cumsum(0) - part.long()).clamp(max=fresh.numel() - 1)]
    theirs = table[src]
    shared = theirs[col < full[:, None]].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    _move(s, theirs.gather(1, full[:, None].clamp(max=table.shape[1] - 1))[:, 0][part].long(), fresh[part].long())
    refs[fresh[part].long()] = 1
    mine = torch.where(col < full[:, None], theirs, torch.where((col == full[:, None]) & part[:, None], fresh[:, None], table[dst]))
    table[dst] = mine
    held[dst] = (full + part).to(torch.int32)
    lens[dst] = n.to(torch.int32)
    return _pool_state(s)


def _plain_compact(s):
    used = s["refs"] > 0
    live = used.sum()
    at = torch.arange(used.numel(), device="cuda")
    holes, movers = (~used & (at < live)).nonzero()[:, 0], (used & (at >= live)).nonzero()[:, 0]
    new = at.to(torch.int32)
    new[movers] = holes.to(torch.int32)
    _move(s, movers, holes)
    refs = s["refs"].clone()
    refs[holes] = s["refs"][movers]
    s["refs_out"].copy_(torch.where(at < live, refs, torch.zeros_like(refs)))
    have = torch.arange(s["table"].shape[1], device="cuda") < s["held"][:, None]
    s["table_out"].copy_(torch.where(have, new[s["table"].long().clamp(min=0)], s["table_out"]))
    s["live"].copy_(live)
    return {k: s[k] for k in ("live", "table_out", "refs_out", "k_cache", "v_cache", "k_scale", "v_scale")}


# ------------------------------------------------------------------ the library's calls
def _own_attend(s):
    import draft_correction_slot_gb300 as dc
    dc.dcoco_tree_attention_quant(s["handle"], s["c"]["N"], s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                                  s["k_scale"], s["v_scale"], s["table"], s["ctx"], out=s["out"], lse=s["lse"],
                                  tree_mask=s["bits"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_append(s):
    import draft_correction_slot_gb300 as dc
    dc.dcoco_tree_append_quant(s["handle"], s["c"]["N"], s["first"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                               s["k_scale"], s["v_scale"], s["table"], s["ctx"], new_len=s["new_len"])
    return {k: s[k] for k in ("new_len", "k_cache", "v_cache", "k_scale", "v_scale")}


def _own_commit(s):
    import draft_correction_slot_gb300 as dc
    dc.dcoco_tree_commit_quant(s["handle"], s["c"]["N"], s["tokens"], s["parents"], s["sampled"], s["k_new"], s["v_new"],
                               s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["ctx"],
                               path=s["path"], accept_len=s["accept_len"], next_token=s["next_token"],
                               new_len=s["new_len"])
    return {k: s[k] for k in ("path", "accept_len", "next_token", "new_len", "k_cache", "v_cache", "k_scale", "v_scale")}


def _own_fork(s):
    import draft_correction_slot_gb300 as dc
    state = (s["table"], s["held"], s["lens"], s["refs"])
    dc.dcoco_pages_free(s["handle"], s["dst"], *state)
    dc.dcoco_pages_fork(s["handle"], s["planes"], s["src"], s["dst"], *state)
    return _pool_state(s)


def _own_compact(s):
    import draft_correction_slot_gb300 as dc
    dc.dcoco_pages_compact(s["handle"], s["planes"], s["table"], s["held"], s["refs"], page_table_out=s["table_out"],
                           refs_out=s["refs_out"], live=s["live"])
    return {k: s[k] for k in ("live", "table_out", "refs_out", "k_cache", "v_cache", "k_scale", "v_scale")}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append, "commit": _own_commit, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"attend": _plain_attend, "append": _plain_append, "commit": _plain_commit, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


# ------------------------------------------------------------------ work and exact values
def _page_bytes(c):
    """K, V and their scales of one page in all layers."""
    return 2 * c["L"] * c["Hkv"] * (c["page"] * c["D"] + 4 * c["page"] // c["block"])


def work(case):
    c = case
    if c["op"] == "attend":
        # contexts between an eighth of the longest and the longest: 9/16 of it in the mean, the first at its longest
        tokens = c["ctx"] * (1 + (c["N"] - 1) * 0.5625)
        row, nodes = c["Hkv"] * c["D"], c["N"] * c["T"]
        return {"bytes": 2 * tokens * (row + 4 * c["Hkv"] / c["block"]) + 4 * nodes * row * (1 + c["g"])
                + 4 * nodes * c["Hkv"] * c["g"], "flops": 4 * row * c["g"] * c["T"] * (tokens + nodes)}
    if c["op"] == "append":
        tokens = c["tokens"] * (1 + (c["N"] - 1) * 0.5625)
        return {"bytes": 2 * c["L"] * c["Hkv"] * tokens * (3 * c["D"] + 4 / c["block"]), "flops": 0}
    if c["op"] == "commit":
        path = min(c["T"], 3)  # the accepted path's usual length here, the anchor included
        return {"bytes": 2 * c["L"] * c["N"] * c["Hkv"] * (path * 3 * c["D"] + 8) + 16 * c["N"] * c["T"], "flops": 0}
    if c["op"] == "fork":
        copied = c["forks"] * (1 - 1 / c["page"])  # a length ends inside a page
        return {"bytes": 2 * copied * _page_bytes(c) + 16 * c["forks"] * -(-c["ctx"] * 0.5625 // c["page"])
                + 4 * c["pages"], "flops": 0}
    moved = c["pages"] * c["used"] * (1 - c["used"])
    return {"bytes": 2 * moved * _page_bytes(c) + 8 * c["pages"] * (1 + c["used"]), "flops": 0}


def _exact_write(s, got, name, layer_rows, n, positions):
    """One request's tokens, block by block: layer_rows [L, tokens, heads, D] in 64 bits."""
    c = s["c"]
    page, block, ctx = c["page"], c["block"], int(s["ctx"][n])
    lo = positions[0]
    while lo <= positions[-1]:
        hi = min(positions[-1] + 1, lo // block * block + block)
        b0 = lo // block * block
        pg, at = int(s["table"][n, b0 // page]), b0 % page
        x = layer_rows[:, lo - positions[0]:hi - positions[0]]
        need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 3)) / MOST)))
        was = got[name + "_scale"][:, pg, at // block].clone()
        now = torch.maximum(was, need) if b0 < ctx else need
        got[name + "_scale"][:, pg, at // block] = now
        cache = got[name + "_cache"]
        cache[:, pg, at:at + max(0, ctx - b0)] *= (was / now)[:, None, :, None]
        cache[:, pg, at + lo - b0:at + hi - b0] = x / now[:, None, :, None]
        lo = hi


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "attend":
        N, T, H, G, D, page, block = c["N"], c["T"], c["Hkv"], c["g"], c["D"], c["page"], c["block"]
        out = torch.zeros(N, T, H * G, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(N, T, H * G, dtype=torch.float64, device="cuda")
        for n in range(N):
            L = int(s["ctx"][n])
            pages = s["table"][n, :-(-L // page)].long()
            for h in range(H):
                old = []
                for name in ("k", "v"):
                    x = s[name + "_cache"][:, :, h].contiguous().view(torch.uint8)[pages].view(E4M3).double() \
                        if N * H < 16 else s[name + "_cache"].view(torch.uint8)[pages, :, h].view(E4M3).double()
                    y = s[name + "_scale"][pages, :, h].double()
                    x = x.view(len(pages), page // block, block, D) * y[:, :, None, None]
                    old.append(x.view(-1, D)[:L])
                k = torch.cat([old[0], s["k_new"][n, :, h].double()])
                v = torch.cat([old[1], s["v_new"][n, :, h].double()])
                a = torch.einsum("tgd,sd->gts", s["q"][n, :, h * G:(h + 1) * G].double(), k) * D ** -0.5
                a[:, :, L:].masked_fill_(~s["anc"][n], -math.inf)
                out[n, :, h * G:(h + 1) * G] = torch.einsum("gts,sd->tgd", torch.softmax(a, -1), v)
                lse[n, :, h * G:(h + 1) * G] = torch.logsumexp(a, -1).T
        return {"out": out, "lse": lse}
    if c["op"] in ("append", "commit"):
        got = {"path": None, "accept_len": None, "next_token": None, "new_len": None}
        got = {"new_len": None} if c["op"] == "append" else got
        for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
            got[name] = s[name].double()
        ctx = s["ctx"].tolist()
        if c["op"] == "append":
            first = s["first"].tolist()
            rows = [list(range(a, b)) for a, b in zip(first, first[1:])]
        else:  # the walk, node by node
            parents, tokens, sampled = (s[k].tolist() for k in ("parents", "tokens", "sampled"))
            rows = []
            for n in range(c["N"]):
                path, node = [], 0
                while node is not None:
                    path.append(node)
                    node = next((t for t in range(node + 1, c["T"]) if parents[n][t] == node
                                 and tokens[n][t] == sampled[n][node]), None)
                rows.append(path)
        if sum(len(r) for r in rows) / c["block"] + len(rows) > 2000:
            return None
        for n, r in enumerate(rows):
            for name in ("k", "v"):
                x = s[name + "_new"][:, r[0]:r[-1] + 1] if c["op"] == "append" else s[name + "_new"][:, n, r]
                _exact_write(s, got, name, x.double(), n, list(range(ctx[n], ctx[n] + len(r))))
        return got
    # pages: what is where, row by row on the host; the floating outputs are copies
    names = ("k_cache", "v_cache", "k_scale", "v_scale")
    refs, held, table, moves = s["refs"].tolist(), s["held"].tolist(), s["table"].tolist(), {}
    if c["op"] == "fork":
        lens = s["lens"].tolist()
        for a in s["src"].tolist():  # the rows forked into are empty here
            n, page = lens[a], c["page"]
            if n % page:
                fresh = next(p for p in range(c["pages"]) if refs[p] == 0)
                refs[fresh] = 1
                moves[fresh] = table[a][n // page]
        got = {k: None for k in ("table", "held", "lens", "refs")}
    else:
        live = sum(r > 0 for r in refs)
        holes = [p for p in range(live) if refs[p] == 0]
        moves = dict(zip(holes, [p for p in range(live, c["pages"]) if refs[p] > 0]))
        got = {k: None for k in ("live", "table_out", "refs_out")}
    for name in names:
        x = s[name].clone()
        for to, came in moves.items():
            x[:, to] = s[name][:, came]
        got[name] = x
    return got
