"""What is measured of the verification and distillation operators.

Four operators: attention of a drafted tree over a paged cache, sampling of the
target's tokens, the commit of the accepted path into the cache, and the
distillation loss of the drafter.  Each case is one call (or, where it says
so, the calls of one step) on inputs made from a seed.  `own` False: the
operator in elementary torch operations; True: the library's kernels.
"""
from __future__ import annotations

import math

import torch

own = False

VOCAB = 151936
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request's block of 16 nodes on a short context: the latency of one layer
        dict(name="attend_1x16_ctx1000", op="attend", N=1, T=16, Hkv=8, g=4, D=128, ctx=1000, page=64,
             dtype="bf16", heads_first=False),
        # a batch of 32 requests, blocks of 16 nodes, ragged contexts up to 8000 tokens, small pages
        dict(name="attend_32x16_ctx8000", op="attend", N=32, T=16, Hkv=8, g=4, D=128, ctx=8000, page=16,
             dtype="bf16", heads_first=False),
        # wide trees of 64 nodes, 40 query heads (five a K/V head), long contexts, head-major pages
        dict(name="attend_8x64_ctx32000", op="attend", N=8, T=64, Hkv=8, g=5, D=128, ctx=32000, page=64,
             dtype="fp16", heads_first=True),
        # single-token decode at head width 64 on long contexts
        dict(name="attend_24x1_ctx16001", op="attend", N=24, T=1, Hkv=8, g=4, D=64, ctx=16001, page=32,
             dtype="bf16", heads_first=False),
        # one request's 16 node logits, every row with parameters of its own
        dict(name="sample_16", op="sample", R=16, V=VOCAB, dtype="bf16", mode="mixed"),
        # 32 requests x 16 nodes, mixed parameters as a server meets them
        dict(name="sample_512", op="sample", R=512, V=VOCAB, dtype="bf16", mode="mixed"),
        # fp32 logits of an odd vocabulary, nucleus sampling alone
        dict(name="sample_200_fp32_top_p", op="sample", R=200, V=32001, dtype="fp32", mode="top_p"),
        # one request's accepted path into the caches of 16 layers
        dict(name="commit_1x16", op="commit", N=1, T=16, L=16, Hkv=8, D=128, page=64, dtype="bf16"),
        # 32 requests with trees of 64 nodes
        dict(name="commit_32x64", op="commit", N=32, T=64, L=16, Hkv=8, D=128, page=16, dtype="bf16"),
        # the draft slots of one request: loss and gradient in one step
        dict(name="distill_15_step", op="distill", R=15, V=VOCAB, K=16, dtype="bf16", call="step", full=False),
        # the draft slots of 32 requests, loss first and the gradient in a call of its own
        dict(name="distill_480_loss_grad", op="distill", R=480, V=VOCAB, K=64, dtype="bf16", call="both",
             full=True),
        # fp32 logits of an odd vocabulary, many rows, one step
        dict(name="distill_2000_fp32_step", op="distill", R=2000, V=32001, K=32, dtype="fp32", call="step",
             full=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "sample", "commit", "distill"])
    if op == "attend":
        while True:
            c = dict(op=op, N=_log_int(rng, 1, 48), T=_log_int(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8]),
                     g=rng.choice([1, 2, 4, 5, 8]), D=rng.choice([64, 128]), ctx=_log_int(rng, 1, 32000),
                     page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16"]),
                     heads_first=rng.random() < 0.5)
            if c["N"] * c["ctx"] * c["Hkv"] * c["D"] <= 8 * 32000 * 8 * 128 and \
                    c["N"] * c["ctx"] * c["Hkv"] * c["g"] * c["T"] * c["D"] <= 8 * 32000 * 40 * 64 * 128:
                return c
    if op == "sample":
        return dict(op=op, R=_log_int(rng, 1, 512), V=rng.choice([VOCAB, _log_int(rng, 1000, VOCAB)]),
                    dtype=rng.choice(["bf16", "fp32"]) if rng.random() < 0.5 else "bf16",
                    mode=rng.choice(["mixed", "top_p", "top_k", "min_p", "plain"]))
    if op == "commit":
        return dict(op=op, N=_log_int(rng, 1, 32), T=_log_int(rng, 1, 64), L=_log_int(rng, 1, 16),
                    Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=rng.choice([16, 32, 64]),
                    dtype=rng.choice(["bf16", "fp16"]))
    while True:
        c = dict(op=op, R=_log_int(rng, 1, 2000), V=rng.choice([VOCAB, _log_int(rng, 1000, VOCAB)]),
                 K=_log_int(rng, 1, 128), dtype=rng.choice(["bf16", "fp32"]),
                 call=rng.choice(["step", "both", "loss", "grad"]), full=rng.random() < 0.5)
        if c["R"] * c["V"] <= 480 * VOCAB:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) % (1 << 30)) + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _logits(g, R, V, dtype):
    """2 N(0,1) with 32 tokens a row raised by U(4, 12), in rows padded to 16 bytes."""
    stride = -(-V // 8) * 8
    x = 2 * _randn(g, R, stride)
    at = torch.randint(0, V, (R, 32), generator=g, device="cuda")
    x.scatter_add_(1, at, 4 + 8 * _rand(g, R, 32))
    return x.to(DT[dtype])[:, :V]


def _tree(g, N, T):
    """Random trees: parents [N, T] (node 0 the root), and who is whose ancestor (or self), [N, T, T]."""
    pick = _rand(g, N, T)
    at = torch.arange(T, device="cuda")
    parents = torch.maximum((pick * at).long(), at - 4).clamp_(max=T - 1)  # one of the four nodes before it
    parents = torch.minimum(parents, (at - 1).clamp(min=0))
    eye = torch.eye(T, dtype=torch.bool, device="cuda")
    anc = eye.repeat(N, 1, 1)
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


def _handle(N, T, Hkv, g, D, page, pages, dtype):
    """The plan a serving program keeps for a model: one handle a configuration."""
    import draft_correction_slot_gb300 as dc
    key = (N, T, Hkv, g, D, page, pages, dtype)
    if key not in _handles:
        _handles[key] = dc.dcoco_tree_create(max_batch=N, max_tree=T, q_heads=Hkv * g, kv_heads=Hkv, head_dim=D,
                                             page_size=page, max_pages=pages, dtype=DT[dtype])
    return _handles[key]


def _prepare_attend(c, g):
    N, T, H, G, D, page, dt = c["N"], c["T"], c["Hkv"], c["g"], c["D"], c["page"], DT[c["dtype"]]
    # contexts between an eighth of the longest and the longest, one of them the longest
    ctx = (c["ctx"] * (0.125 + 0.875 * _rand(g, N))).long().clamp(min=1)
    ctx[0] = c["ctx"]
    width = -(-(c["ctx"] + T) // page)
    need = (ctx + T + page - 1) // page
    total = N * width
    order = torch.randperm(total, generator=g, device="cuda")
    table = order.view(N, width).to(torch.int32)
    table = torch.where(torch.arange(width, device="cuda") < need[:, None], table, torch.zeros_like(table))
    shape = (total, H, page, D) if c["heads_first"] else (total, page, H, D)
    cache = [torch.randn(shape, generator=g, device="cuda", dtype=dt) for _ in range(2)]
    # q, k and v of the nodes leave one projection: views of one buffer, as a model has them
    qkv = _randn(g, N, T, (G + 2) * H, D).to(dt)
    parents, anc = _tree(g, N, T)
    s = dict(c=c, q=qkv[:, :, :G * H], k_new=qkv[:, :, G * H:G * H + H], v_new=qkv[:, :, G * H + H:],
             k_cache=cache[0], v_cache=cache[1], table=table, ctx=ctx.to(torch.int32), anc=anc, bits=_bits(anc),
             out=torch.empty(N, T, G * H, D, dtype=dt, device="cuda"),
             lse=torch.empty(N, T, G * H, dtype=torch.float32, device="cuda"))
    if c["heads_first"]:  # [pages, page, heads, D] views of head-major storage
        s["k_cache"], s["v_cache"] = (x.transpose(1, 2) for x in cache)
    if own:
        s["handle"] = _handle(N, T, H, G, D, page, width, c["dtype"])
    return s


def _prepare_sample(c, g):
    R, mode = c["R"], c["mode"]
    x = _logits(g, R, c["V"], c["dtype"])
    s = dict(c=c, logits=x, u=_rand(g, R), temperature=0.6 + 0.6 * _rand(g, R),
             top_k=None, top_p=None, min_p=None)
    some = torch.arange(R, device="cuda") % 4  # mixed: rows of four kinds
    if mode in ("mixed", "top_k"):
        k = torch.randint(1, 101, (R,), generator=g, device="cuda")
        s["top_k"] = (torch.where(some == 1, k, 0) if mode == "mixed" else k).to(torch.int32)
    if mode in ("mixed", "top_p"):
        p = 0.7 + 0.28 * _rand(g, R)
        s["top_p"] = torch.where(some >= 2, p, torch.ones_like(p)) if mode == "mixed" else p
    if mode in ("mixed", "min_p"):
        p = 0.01 + 0.19 * _rand(g, R)
        s["min_p"] = torch.where(some == 3, p, torch.zeros_like(p)) if mode == "mixed" else p
    s["tokens"] = torch.empty(R, dtype=torch.int32, device="cuda")
    s["logprob"] = torch.empty(R, dtype=torch.float32, device="cuda")
    return s


def _prepare_commit(c, g):
    N, T, L, H, D, page, dt = c["N"], c["T"], c["L"], c["Hkv"], c["D"], c["page"], DT[c["dtype"]]
    width = -(-(2 * page + T) // page)  # two pages of context at most, then the tree
    ctx = (2 * page * _rand(g, N)).to(torch.int32)
    table = torch.randperm(N * width, generator=g, device="cuda").view(N, width).to(torch.int32)
    cache = [torch.randn(L, N * width, page, H, D, generator=g, device="cuda", dtype=dt) for _ in range(2)]
    new = [torch.randn(L, N, T, H, D, generator=g, device="cuda", dtype=dt) for _ in range(2)]
    parents, anc = _tree(g, N, T)
    tokens = torch.randint(0, VOCAB, (N, T), generator=g, device="cuda", dtype=torch.int32)
    sampled = torch.randint(0, VOCAB, (N, T), generator=g, device="cuda", dtype=torch.int32)
    # the target agrees with one child of most nodes: the last writer among the children of a node
    agree = _rand(g, N, T) < 0.8
    up = torch.where(agree & (parents >= 0), parents, T).long()
    wide = torch.cat([sampled, sampled[:, :1]], 1)
    sampled = wide.scatter(1, up, tokens)[:, :T].contiguous()
    s = dict(c=c, k_new=new[0], v_new=new[1], k_cache=cache[0], v_cache=cache[1], table=table, ctx=ctx,
             parents=parents, anc=anc, tokens=tokens, sampled=sampled)
    for name, shape in (("path", (N, T)), ("accept_len", (N,)), ("next_token", (N,)), ("new_len", (N,))):
        s[name] = torch.empty(shape, dtype=torch.int32, device="cuda")
    if own:
        s["handle"] = _handle(N, T, H, 1, D, page, width, c["dtype"])
    return s


def _prepare_distill(c, g):
    R, V, K = c["R"], c["V"], c["K"]
    x = _logits(g, R, V, c["dtype"])
    # the teacher's top logits: most of them where the student's are large, all tokens different
    mix = x.float() + 3 * _randn(g, R, V)
    top = mix.topk(K, dim=1)
    s = dict(c=c, logits=x, ids=top.indices.to(torch.int32).contiguous(),
             teacher=top.values.contiguous(), temperature=1.0 if R % 2 else 2.0,
             grad_loss=_rand(g, R) / R, teacher_lse=None)
    if c["full"]:
        s["teacher_lse"] = (mix / s["temperature"]).logsumexp(1)
    s["loss"] = torch.empty(R, dtype=torch.float32, device="cuda")
    s["lse"] = torch.empty(R, dtype=torch.float32, device="cuda")
    stride = x.stride(0)
    s["grad"] = torch.zeros(R, stride, dtype=x.dtype, device="cuda")[:, :V]
    if c["call"] == "grad":  # what the loss call before it left
        s["lse"].copy_((x.float() / s["temperature"]).logsumexp(1))
    return s


def prepare(case, seed):
    g = _gen(seed)
    return {"attend": _prepare_attend, "sample": _prepare_sample, "commit": _prepare_commit,
            "distill": _prepare_distill}[case["op"]](case, g)


# ------------------------------------------------------------------ plain forms
def _plain_attend(s):
    c = s["c"]
    N, T, H, G, D = c["N"], c["T"], c["Hkv"], c["g"], c["D"]
    table = s["table"].long()
    S = table.shape[1] * c["page"]
    seen = torch.arange(S, device="cuda") < s["ctx"][:, None]
    zero = torch.zeros((), device="cuda")
    k = torch.cat([s["k_cache"][table].reshape(N, S, H, D).float(), s["k_new"].float()], 1)
    v = torch.cat([s["v_cache"][table].reshape(N, S, H, D).float(), s["v_new"].float()], 1)
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


def _plain_sample(s):
    x = s["logits"].double()
    R, V = x.shape
    t = s["temperature"].double()[:, None]
    top, at = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    z = (top.double() - top[:, :1].double()) / t
    w = torch.exp(z)
    keep = torch.ones(R, V, dtype=torch.bool, device="cuda")
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (torch.arange(V, device="cuda") < k) | (k <= 0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        kept = w * keep
        before = torch.cumsum(kept, 1) - kept
        keep &= (before < p * kept.sum(1, keepdim=True)) | (p >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    kept = torch.zeros_like(w).scatter_(1, at, w * keep)  # back in vocabulary order
    cum = torch.cumsum(kept, 1)
    total = cum[:, -1:]
    tok = ((cum <= s["u"].double()[:, None] * total) | (kept == 0)).to(torch.uint8).argmin(1)
    z_tok = (x.gather(1, tok[:, None]) - top[:, :1].double()) / t
    return {"tokens": tok.to(torch.int32), "logprob": (z_tok - torch.log(total))[:, 0].float()}


def _plain_commit(s):
    c = s["c"]
    N, T, page = c["N"], c["T"], c["page"]
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
    pg, slot = s["table"].long()[n, pos // page], pos % page
    s["k_cache"][:, pg, slot] = s["k_new"][:, n, t]
    s["v_cache"][:, pg, slot] = s["v_new"][:, n, t]
    return {"path": torch.where(path == T, -1, path).to(torch.int32), "accept_len": (count - 1).to(torch.int32),
            "next_token": s["sampled"].gather(1, last)[:, 0], "new_len": (s["ctx"] + count).to(torch.int32),
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_distill(s):
    c, T = s["c"], s["temperature"]
    ids = s["ids"].long()
    z = s["logits"].float() / T
    m = z.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    t = s["teacher"] / T
    if s["teacher_lse"] is None:
        tm = t.amax(1, keepdim=True)
        t_lse = tm + torch.log(torch.exp(t - tm).sum(1, keepdim=True))
    else:
        t_lse = s["teacher_lse"][:, None]
    p = torch.exp(t - t_lse)
    got = {}
    if c["call"] != "grad":
        got["loss"] = T * T * (p * (t - t_lse - z.gather(1, ids) + lse)).sum(1)
        got["lse"] = lse[:, 0]
    if c["call"] != "loss":
        grad = torch.exp(z - lse) * p.sum(1, keepdim=True)
        grad.scatter_add_(1, ids, -p)
        got["grad"] = (grad * (s["grad_loss"][:, None] * T)).to(s["logits"].dtype)
    return got


# ------------------------------------------------------------------ the library's calls
def _own_attend(s):
    import draft_correction_slot_gb300 as dc
    dc.dcoco_tree_attention(s["handle"], s["c"]["N"], s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                            s["table"], s["ctx"], out=s["out"], lse=s["lse"], tree_mask=s["bits"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_sample(s):
    import draft_correction_slot_gb300 as dc
    dc.dcoco_sample(s["logits"], s["u"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"],
                    top_p=s["top_p"], min_p=s["min_p"], logprob=s["logprob"])
    return {"tokens": s["tokens"], "logprob": s["logprob"]}


def _own_commit(s):
    import draft_correction_slot_gb300 as dc
    dc.dcoco_tree_commit(s["handle"], s["c"]["N"], s["tokens"], s["parents"], s["sampled"], s["k_new"], s["v_new"],
                         s["k_cache"], s["v_cache"], s["table"], s["ctx"], path=s["path"],
                         accept_len=s["accept_len"], next_token=s["next_token"], new_len=s["new_len"])
    return {k: s[k] for k in ("path", "accept_len", "next_token", "new_len", "k_cache", "v_cache")}


def _own_distill(s):
    import draft_correction_slot_gb300 as dc
    call = s["c"]["call"]
    kw = dict(teacher_lse=s["teacher_lse"], temperature=s["temperature"])
    if call == "step":
        dc.dcoco_distill_step(s["logits"], s["ids"], s["teacher"], s["grad_loss"], loss=s["loss"], lse=s["lse"],
                              grad=s["grad"], **kw)
    if call in ("both", "loss"):
        dc.dcoco_distill_loss(s["logits"], s["ids"], s["teacher"], loss=s["loss"], lse=s["lse"], **kw)
    if call in ("both", "grad"):
        dc.dcoco_distill_grad(s["logits"], s["ids"], s["teacher"], s["lse"], s["grad_loss"], grad=s["grad"], **kw)
    names = {"loss": ("loss", "lse"), "grad": ("grad",)}.get(call, ("loss", "lse", "grad"))
    return {k: s[k] for k in names}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"attend": _own_attend, "sample": _own_sample, "commit": _own_commit, "distill": _own_distill}[op](state)
    return {"attend": _plain_attend, "sample": _plain_sample, "commit": _plain_commit,
            "distill": _plain_distill}[op](state)


# ------------------------------------------------------------------ work and exact values
def work(case):
    c = case
    if c["op"] == "attend":
        # contexts between an eighth of the longest and the longest: 9/16 of it in the mean, the first at its longest
        tokens = c["ctx"] * (1 + (c["N"] - 1) * 0.5625)
        row, e = c["Hkv"] * c["D"], 2
        nodes = c["N"] * c["T"]
        return {"bytes": 2 * e * row * (tokens + nodes) + 2 * e * nodes * row * c["g"] + 4 * nodes * c["Hkv"] * c["g"],
                "flops": 4 * row * c["g"] * c["T"] * (tokens + nodes)}
    if c["op"] == "sample":
        return {"bytes": c["R"] * (c["V"] * SIZE[c["dtype"]] + 28), "flops": 4 * c["R"] * c["V"]}
    if c["op"] == "commit":
        path = min(c["T"], 4)  # the accepted path's usual length here, the anchor included
        return {"bytes": 2 * 2 * 2 * c["L"] * c["N"] * path * c["Hkv"] * c["D"] + 16 * c["N"] * c["T"], "flops": 0}
    passes = {"loss": 1, "grad": 2, "step": 2, "both": 3}[c["call"]]
    return {"bytes": c["R"] * (passes * c["V"] * SIZE[c["dtype"]] + 8 * c["K"] + 16), "flops": 5 * c["R"] * c["V"]}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "attend":
        N, T, H, G, D = c["N"], c["T"], c["Hkv"], c["g"], c["D"]
        out = torch.zeros(N, T, H * G, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(N, T, H * G, dtype=torch.float64, device="cuda")
        for n in range(N):
            L = int(s["ctx"][n])
            pages = s["table"][n, :-(-L // c["page"])].long()
            for h in range(H):
                k = torch.cat([s["k_cache"][pages, :, h].reshape(-1, D)[:L], s["k_new"][n, :, h]]).double()
                v = torch.cat([s["v_cache"][pages, :, h].reshape(-1, D)[:L], s["v_new"][n, :, h]]).double()
                a = torch.einsum("tgd,sd->gts", s["q"][n, :, h * G:(h + 1) * G].double(), k) * D ** -0.5
                a[:, :, L:].masked_fill_(~s["anc"][n], -math.inf)
                out[n, :, h * G:(h + 1) * G] = torch.einsum("gts,sd->tgd", torch.softmax(a, -1), v)
                lse[n, :, h * G:(h + 1) * G] = torch.logsumexp(a, -1).T
        return {"out": out, "lse": lse}
    if c["op"] == "sample":
        R, V = s["logits"].shape
        lp = torch.zeros(R, dtype=torch.float64, device="cuda")
        for r in range(R):
            p = torch.softmax(s["logits"][r].double() / s["temperature"][r].double(), 0)
            by = torch.argsort(s["logits"][r].float(), descending=True, stable=True)
            if s["top_k"] is not None and int(s["top_k"][r]) > 0:
                by = by[: int(s["top_k"][r])]
            if s["top_p"] is not None and float(s["top_p"][r]) < 1:
                mass = torch.cumsum(p[by], 0)
                mass = torch.cat([mass.new_zeros(1), mass])
                by = by[: int((mass[:-1] < s["top_p"][r].double() * mass[-1]).sum())]
            if s["min_p"] is not None:
                by = by[p[by] >= s["min_p"][r].double() * p.max()]
            kept = torch.zeros_like(p)
            kept[by] = p[by]
            cum = torch.cumsum(kept, 0)
            tok = int(torch.searchsorted(cum, s["u"][r].double() * cum[-1], right=True))
            lp[r] = torch.log(p[tok] / kept.sum())
        return {"tokens": None, "logprob": lp}
    if c["op"] == "distill":
        T, R = s["temperature"], c["R"]
        got = {"loss": None, "lse": None, "grad": None}
        ids, rows = s["ids"].long(), torch.arange(R, device="cuda")
        t = s["teacher"].double() / T
        logp = t - (t.logsumexp(1) if s["teacher_lse"] is None else s["teacher_lse"].double())[:, None]
        logq = torch.log_softmax(s["logits"].double() / T, 1)
        if c["call"] != "grad":
            got["loss"] = T ** 2 * (logp.exp() * (logp - torch.gather(logq, 1, ids))).sum(1)
            got["lse"] = torch.logsumexp(s["logits"].double() / T, 1)
        if c["call"] != "loss":
            d = logq.exp_() * logp.exp().sum(1, keepdim=True)
            d.index_put_((rows[:, None].expand_as(ids), ids), -logp.exp(), accumulate=True)
            got["grad"] = d * (T * s["grad_loss"].double()[:, None])
        names = {"loss": ("loss", "lse"), "grad": ("grad",)}.get(c["call"], ("loss", "lse", "grad"))
        return {k: got[k] for k in names}
    # commit: the walk, node by node on the host, and its copies
    parents, tokens, sampled, ctx, table = (s[k].tolist() for k in ("parents", "tokens", "sampled", "ctx", "table"))
    got = {"path": None, "accept_len": None, "next_token": None, "new_len": None,
           "k_cache": s["k_cache"].clone(), "v_cache": s["v_cache"].clone()}
    for n in range(c["N"]):
        node, pos = 0, ctx[n]
        while node is not None:
            pg, slot = table[n][pos // c["page"]], pos % c["page"]
            got["k_cache"][:, pg, slot] = s["k_new"][:, n, node]
            got["v_cache"][:, pg, slot] = s["v_new"][:, n, node]
            pos += 1
            node = next((t for t in range(node + 1, c["T"]) if parents[n][t] == node
                         and tokens[n][t] == sampled[n][node]), None)
    return got
