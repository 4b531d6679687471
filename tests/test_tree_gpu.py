"""Tree attention, tree commit, sampling and distillation on the GPU against
64-bit references.  Tolerances count roundings: half a step of the 16-bit type
for each attention weight and for the output, fp32 sums elsewhere."""
import math

import numpy as np
import pytest

import tree_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import draft_correction_slot_gb300 as dc
    return torch, dc


def f64(x):
    return x.detach().double().cpu().numpy()


# ------------------------------------------------------------------ attention
class Attn:
    """A problem with random trees; unseen cache slots, pages and nodes hold NaN and infinities."""

    def __init__(self, torch, seed, ctx, T, Hkv, g, D, page, dtype, heads_first=False, tree_len=None, mask="tree",
                 poison=True, extra_pages=3):
        rng = np.random.default_rng(seed)
        self.torch, self.N, self.T, self.H, self.g, self.D, self.page, self.dtype = torch, len(ctx), T, Hkv, g, D, page, dtype
        N = self.N
        self.max_pages = max(1, -(-max(ctx) // page)) + 1
        used = [-(-c // page) for c in ctx]
        self.pages = sum(used) + extra_pages
        order = rng.permutation(self.pages)
        table = np.full((N, self.max_pages), -7, np.int32)  # unused entries are not page numbers
        at = 0
        for n in range(N):
            table[n, :used[n]] = order[at:at + used[n]]
            at += used[n]
        shape = (self.pages, Hkv, page, D) if heads_first else (self.pages, page, Hkv, D)
        bad = torch.tensor([math.nan, math.inf, -math.inf])
        caches = []
        for _ in range(2):
            x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
            if heads_first:
                x = x.transpose(1, 2)
            if poison:
                seen = torch.zeros(self.pages, page, dtype=torch.bool)
                for n in range(N):
                    pos = np.arange(ctx[n])
                    seen[torch.from_numpy(table[n, pos // page].astype(np.int64)), torch.from_numpy(pos % page)] = True
                x[~seen] = bad[torch.from_numpy(rng.integers(0, 3, (int((~seen).sum()), Hkv, D)))]
            if heads_first:
                caches.append(x.transpose(1, 2).contiguous().to(dtype).cuda().transpose(1, 2))
            else:
                caches.append(x.to(dtype).cuda())
        self.k_cache, self.v_cache = caches
        qkv = torch.from_numpy(rng.standard_normal((N, T, (g + 2) * Hkv, D)).astype(np.float32))
        self.len = np.full(N, T) if tree_len is None else np.asarray(tree_len)
        if poison:
            for n in range(N):
                qkv[n, self.len[n]:] = math.nan
        qkv = qkv.to(dtype).cuda()
        hq = g * Hkv
        self.q, self.k_new, self.v_new = qkv[:, :, :hq], qkv[:, :, hq:hq + Hkv], qkv[:, :, hq + Hkv:]
        par = np.full((N, T), -1, np.int32)
        for t in range(1, T):
            par[:, t] = rng.integers(max(0, t - 4), t, N)
        self.sees = np.zeros((N, T, T), bool)
        for n in range(N):
            for t in range(T):
                if mask == "causal":
                    self.sees[n, t, :t + 1] = True
                elif mask == "random":
                    self.sees[n, t] = rng.random(T) < 0.4
                elif mask == "none":
                    pass
                else:
                    self.sees[n, t, t] = True
                    if par[n, t] >= 0:
                        self.sees[n, t] |= self.sees[n, par[n, t]]
        self.mask = None
        if mask != "causal":
            W = -(-T // 32)
            bits = np.zeros((N, T, W * 32), np.uint64)
            bits[:, :, :T] = self.sees
            words = (bits.reshape(N, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
            self.mask = torch.from_numpy(words.view(np.int32)).cuda()
        self.ctx, self.table = np.asarray(ctx), table
        self.t_ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.t_table = torch.from_numpy(table).cuda()
        self.t_len = None if tree_len is None else torch.tensor(tree_len, dtype=torch.int32, device="cuda")

    def verifier(self, dc, **kw):
        return dc.TreeVerifier(self.H * self.g, self.H, self.D, self.page, self.max_pages,
                               **{**dict(max_batch=self.N, max_tree=self.T, dtype=self.dtype), **kw})

    def run(self, v, **kw):
        return v.attention(self.q, self.k_new, self.v_new, self.k_cache, self.v_cache, self.t_table, self.t_ctx,
                           tree_mask=self.mask, tree_len=self.t_len, **kw)

    def check(self, out, lse, scale=None, rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        ref, rl, mag, reach, flat = tree_ref.attention(
            f64(self.q), f64(self.k_new), f64(self.v_new), f64(self.k_cache), f64(self.v_cache), self.table, self.ctx,
            self.sees, self.len, scale)
        eps = self.torch.finfo(self.dtype).eps / 2
        err_s = (self.D + 8) * 2.0 ** -24 * reach[..., None]  # a score's fp32 sum
        tiny = 2.0 ** -25 * flat if self.dtype == self.torch.float16 else 0  # fp16 weights lose what is below 2^-25
        tol = (eps + 2 * err_s + 2.0 ** -20) * mag + eps * np.abs(ref) + tiny + 2.0 ** -24
        got, gl = f64(out), f64(lse)
        assert np.isfinite(got).all()
        worst = (np.abs(got - ref) / tol).max()
        assert worst <= 1, worst
        empty = np.isneginf(rl)
        assert (np.isneginf(gl) == empty).all() and (got[empty] == 0).all()
        live = ~empty
        assert (np.abs(gl[live] - rl[live]) <= (2 * err_s[..., 0] + 2.0 ** -20 + 2.0 ** -23 * np.abs(rl, where=live, out=np.zeros_like(rl)))[live]).all()


SHAPES = [
    # ctx, T, Hkv, g, D, page
    ([0], 1, 1, 1, 64, 16),
    ([1], 1, 2, 4, 128, 16),
    ([0, 1, 15, 16, 17], 3, 1, 3, 64, 16),
    ([127, 128, 129, 255, 256], 1, 2, 4, 128, 64),
    ([257, 5, 700], 16, 2, 4, 128, 16),
    ([64, 333], 7, 3, 5, 64, 32),
    ([1000], 33, 1, 8, 128, 128),
    ([300, 0], 64, 2, 5, 128, 64),
    ([130], 65, 1, 2, 64, 1024),
    ([77, 513], 130, 1, 1, 128, 16),
    ([200], 256, 1, 2, 64, 32),
    ([90], 5, 1, 71, 64, 32),
    ([129], 2, 1, 128, 128, 256),
    ([2500, 3], 4, 2, 2, 128, 64),
    ([40, 1999, 640, 0, 1280, 128, 127], 2, 4, 4, 64, 64),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention_shapes(env, i, dtype):
    torch, dc = env
    ctx, T, H, g, D, page = SHAPES[i]
    a = Attn(torch, 10 + i, ctx, T, H, g, D, page, getattr(torch, dtype), heads_first=i % 2 == 1)
    v = a.verifier(dc)
    for _ in range(2):  # twice: counters and workspaces are ready for the next call
        out, lse = a.run(v)
        a.check(out, lse)
    assert v.status() == dc.DCOCO_OK


@pytest.mark.parametrize("T,H,g,D,page", [(1, 4, 4, 64, 32), (3, 4, 5, 128, 16), (16, 4, 2, 64, 16), (12, 4, 5, 128, 64),
                                          (30, 4, 4, 128, 64), (70, 3, 4, 64, 128)])
def test_attention_more_units_than_blocks(env, T, H, g, D, page):
    """Each block takes several units, of one tile and of many, with empty ones between."""
    torch, dc = env
    rng = np.random.default_rng(T)
    ctx = [int(rng.choice([0, 1, 100, 128, 400, 900, 2500, 4500])) for _ in range(70)]
    a = Attn(torch, T, ctx, T, H, g, D, page, torch.bfloat16, tree_len=[int(rng.choice([0, 1, T, T])) for _ in ctx])
    v = a.verifier(dc)
    out, lse = a.run(v)
    assert v.status() == dc.DCOCO_OK
    again, lse2 = a.run(v)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    heads = H * g
    for n in rng.choice(70, 12, replace=False):  # the 64-bit reference of every request would take minutes
        b = Attn.__new__(Attn)
        b.__dict__.update(a.__dict__)
        one = slice(n, n + 1)
        b.q, b.k_new, b.v_new = a.q[one], a.k_new[one], a.v_new[one]
        b.table, b.ctx, b.sees, b.len = a.table[one], a.ctx[one], a.sees[one], a.len[one]
        b.check(out[one], lse[one])
    dead = torch.tensor([[t >= a.len[n] for t in range(T)] for n in range(70)], device="cuda")
    assert (out[dead] == 0).all() and int(torch.isneginf(lse[dead]).sum()) == int(dead.sum()) * heads


@pytest.mark.parametrize("mask", ["causal", "random", "none"])
@pytest.mark.parametrize("ctx", [[0, 0, 0], [37, 128, 1]])
@pytest.mark.parametrize("T", [1, 9, 40, 129])
def test_attention_masks_and_lengths(env, mask, ctx, T):
    """Empty rows (no context, nothing seen), and trees shorter than the call's nodes."""
    torch, dc = env
    a = Attn(torch, T, ctx, T, 2, 2, 64, 32, torch.bfloat16, tree_len=[0, (T + 1) // 2, T], mask=mask)
    v = a.verifier(dc)
    out, lse = a.run(v, scale=0.3)
    a.check(out, lse, scale=0.3)
    assert v.status() == dc.DCOCO_OK


def test_attention_unseen_nodes_hold_nan(env):
    """Infinities and NaN in the K/V of a node reach the nodes that see it, and no others."""
    torch, dc = env
    a = Attn(torch, 3, [150, 20], 24, 2, 4, 128, 16, torch.bfloat16, poison=False)
    v = a.verifier(dc)
    clean, _ = a.run(v)
    for j, value in ((5, math.nan), (11, math.inf), (17, -math.inf)):
        a.v_new[:, j] = value
        a.k_new[:, j] = math.nan
    out, _ = a.run(v)
    hit = torch.from_numpy(a.sees[:, :, [5, 11, 17]].any(-1)).cuda()
    assert torch.equal(out[~hit], clean[~hit])
    assert int(torch.isfinite(out[hit].float()).sum()) == 0
    a.k_new[:, [5, 11, 17]] = 0
    out, _ = a.run(v)
    assert torch.equal(out[~hit], clean[~hit])
    assert int(torch.isfinite(out[hit].float()).sum()) == 0


def test_attention_large_scores(env):
    """Scores of hundreds, rising and falling along the context: the running maximum moves a lot."""
    torch, dc = env
    for dtype in (torch.bfloat16, torch.float16):
        a = Attn(torch, 8, [1500, 900], 6, 1, 4, 128, 64, dtype)
        ramp = torch.linspace(0.1, 6, 1500).cuda()
        for n in range(2):
            pos = torch.arange(a.ctx[n], device="cuda")
            at = a.t_table[n].long()[pos // 64]
            a.k_cache[at, pos % 64] *= (ramp[pos] if n == 0 else ramp[-1] - ramp[pos]).to(dtype)[:, None, None]
        v = a.verifier(dc)
        a.check(*a.run(v, scale=1.0), scale=1.0)


def test_attention_batch_and_stream(env):
    """A request's outputs are the same bits alone, in a batch, and on another stream."""
    torch, dc = env
    a = Attn(torch, 21, [3000, 10, 700, 128, 1025], 8, 2, 4, 128, 32, torch.bfloat16)
    v = a.verifier(dc)
    out, lse = a.run(v)
    for n in range(a.N):
        o, l = v.attention(a.q[n:n + 1], a.k_new[n:n + 1], a.v_new[n:n + 1], a.k_cache, a.v_cache, a.t_table[n:n + 1],
                           a.t_ctx[n:n + 1], tree_mask=a.mask[n:n + 1])
        assert torch.equal(o[0], out[n]) and torch.equal(l[0], lse[n])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, l = a.run(v)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, out) and torch.equal(l, lse)
    g = torch.cuda.CUDAGraph()
    o.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        dc.dcoco_tree_attention(v.handle, a.N, a.q, a.k_new, a.v_new, a.k_cache, a.v_cache, a.t_table, a.t_ctx, out=o,
                                lse=l, tree_mask=a.mask)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)


def test_attention_shared_mask(env):
    torch, dc = env
    a = Attn(torch, 31, [30, 31, 200], 12, 1, 4, 64, 16, torch.float16)
    a.sees[:] = a.sees[0]
    a.mask = a.mask[:1].contiguous()
    a.check(*a.run(a.verifier(dc)))


def test_attention_far_pages(env):
    """A pool of more than 2^31 elements: pages at its end."""
    torch, dc = env
    a = Attn(torch, 41, [500], 4, 1, 4, 128, 64, torch.bfloat16)
    pages = (1 << 31) // (64 * 128) + 20
    for name in ("k_cache", "v_cache"):
        pool = torch.empty(pages, 64, 1, 128, dtype=torch.bfloat16, device="cuda")
        pool[-a.pages:] = getattr(a, name)
        setattr(a, "small_" + name, getattr(a, name))
        setattr(a, name, pool)
    a.t_table += pages - a.pages
    out, lse = a.run(a.verifier(dc))
    a.k_cache, a.v_cache = a.small_k_cache, a.small_v_cache
    a.check(out, lse)


def test_attention_flags_bad_lengths_and_pages(env):
    """Lengths and pages out of range are clamped or left out by the kernel and recorded."""
    torch, dc = env
    a = Attn(torch, 51, [40, 40, 40, 40], 4, 1, 2, 64, 16, torch.bfloat16)
    v = a.verifier(dc)
    good, _ = a.run(v)
    assert v.status() == dc.DCOCO_OK
    a.t_ctx[1] = -5
    out, _ = a.run(v)
    assert v.status() == dc.DCOCO_EDEVICE and v.status() == dc.DCOCO_OK
    assert torch.equal(out[0], good[0]) and torch.equal(out[2:], good[2:])
    a.t_ctx[1] = 40
    for page in (-1, a.pages, 1 << 30, -(1 << 31)):
        keep = int(a.t_table[2, 1])
        a.t_table[2, 1] = page
        out, _ = a.run(v)
        assert v.status() == dc.DCOCO_EDEVICE
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[3], good[3])
        a.t_table[2, 1] = keep
    out, _ = a.run(v)
    assert v.status() == dc.DCOCO_OK and torch.equal(out, good)


def test_attention_refusals(env):
    torch, dc = env
    a = Attn(torch, 61, [40, 3], 4, 2, 2, 64, 16, torch.bfloat16)
    v = a.verifier(dc)
    before = dc.dcoco_tree_launches(v.handle)
    args = dict(q=a.q, k_new=a.k_new, v_new=a.v_new, k_cache=a.k_cache, v_cache=a.v_cache, page_table=a.t_table,
                ctx_len=a.t_ctx, out=torch.empty_like(a.q), tree_mask=a.mask)

    def call(batch=2, **kw):
        dc.dcoco_tree_attention(v.handle, batch, **{**args, **kw})

    for kw in (dict(q=a.q.float()), dict(k_cache=a.k_cache[:, :8]), dict(ctx_len=a.t_ctx.long()),
               dict(page_table=a.t_table[:, :1]), dict(out=torch.empty(2, 4, 4, 32, device="cuda")),
               dict(tree_mask=a.mask[:, :2]), dict(v_new=a.v_new.cpu()),
               dict(q=a.q.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            call(**kw)
    wide = torch.zeros(2, 4, 4, 68, dtype=torch.bfloat16, device="cuda")
    for kw, status in ((dict(q=wide[..., :64]), -1),          # a stride that is no multiple of 8
                       (dict(q=torch.zeros(2 * 4 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 4, 4, 64)), -1),
                       (dict(k_new=a.k_new[:, :, :1].expand(2, 4, 2, 64)), -1),  # a stride of zero
                       (dict(scale=math.nan), -1), (dict(scale=math.inf), -1)):
        with pytest.raises(dc.DcocoError) as e:
            call(**kw)
        assert e.value.status == status
    big = Attn(torch, 61, [40, 3, 1], 5, 2, 2, 64, 16, torch.bfloat16)
    with pytest.raises(dc.DcocoError) as e:
        big.run(v)
    assert e.value.status == dc.DCOCO_EBATCH
    big = Attn(torch, 61, [40, 3], 5, 2, 2, 64, 16, torch.bfloat16)
    with pytest.raises(dc.DcocoError) as e:
        big.run(v)
    assert e.value.status == dc.DCOCO_EINVAL
    assert dc.dcoco_tree_launches(v.handle) == before
    assert v.status() == dc.DCOCO_OK


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("N,T,L,H,D,page,dtype", [
    (1, 1, 1, 1, 64, 16, "bfloat16"), (3, 16, 2, 2, 128, 16, "float16"), (5, 40, 3, 1, 64, 32, "bfloat16"),
    (2, 256, 1, 3, 64, 64, "bfloat16"), (40, 7, 5, 8, 128, 16, "bfloat16"),
])
@pytest.mark.parametrize("chain", [False, True])
def test_commit(env, N, T, L, H, D, page, dtype, chain):
    torch, dc = env
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(N * T)
    ctx = rng.integers(0, 3 * page, N)
    ctx[0] = page - 1
    width = -(-(3 * page + T) // page)
    pages = N * width + 2
    table = rng.permutation(pages)[:N * width].reshape(N, width).astype(np.int32)
    par = np.full((N, T), -1, np.int32)
    for t in range(1, T):
        par[:, t] = t - 1 if chain else rng.integers(max(0, t - 5), t, N)
    tokens = rng.integers(0, 4, (N, T)).astype(np.int32)  # few tokens: siblings of the same token
    sampled = rng.integers(0, 4, (N, T)).astype(np.int32)
    if chain:
        sampled[:, :-1] = tokens[:, 1:]
        sampled[N // 2, T // 2] = 9
    length = rng.integers(0, T + 1, N).astype(np.int32)
    length[0] = T
    new = [torch.randn(L, N, T, 2 * H, D, device="cuda").to(dt)[:, :, :, ::2] for _ in range(2)]
    cache = [torch.randn(L, pages, H, page, D, device="cuda").to(dt).transpose(2, 3) for _ in range(2)]
    want = [c.clone() for c in cache]
    v = dc.TreeVerifier(H, H, D, page, width, max_batch=N, max_tree=T, dtype=dt)
    cuda = lambda x: torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).cuda()  # noqa: E731
    got = v.commit(cuda(tokens), cuda(par), cuda(sampled), *new, *cache, cuda(table), cuda(ctx), tree_len=cuda(length))
    for n in range(N):
        path, nxt = tree_ref.walk(tokens[n], par[n], sampled[n], int(length[n]))
        assert got["path"][n].tolist() == path + [-1] * (T - len(path))
        assert int(got["accept_len"][n]) == max(0, len(path) - 1)
        assert int(got["next_token"][n]) == nxt
        assert int(got["new_len"][n]) == ctx[n] + len(path)
        for i, t in enumerate(path):
            pos = int(ctx[n]) + i
            for w, x in zip(want, new):
                w[:, int(table[n, pos // page]), pos % page] = x[:, n, t]
    assert torch.equal(cache[0], want[0]) and torch.equal(cache[1], want[1])
    assert v.status() == dc.DCOCO_OK


def test_commit_flags_and_refuses(env):
    torch, dc = env
    v = dc.TreeVerifier(1, 1, 64, 16, 2, max_batch=2, max_tree=4)
    i32 = dict(dtype=torch.int32, device="cuda")
    tok = torch.tensor([[1, 2, 3, 4]] * 2, **i32)
    par = torch.tensor([[-1, 0, 1, 2]] * 2, **i32)
    nxt = torch.tensor([[2, 3, 4, 5]] * 2, **i32)
    new = torch.randn(1, 2, 4, 1, 64, device="cuda").bfloat16()
    cache = torch.zeros(1, 4, 16, 1, 64, device="cuda").bfloat16()
    other = cache.clone()
    table = torch.tensor([[0, 1], [2, 3]], **i32)
    # request 0 runs past its table after two tokens; request 1's second page is no page
    ctx = torch.tensor([30, 14], **i32)
    table[1, 1] = 9
    got = v.commit(tok, par, nxt, new, new, cache, other, table, ctx)
    assert v.status() == dc.DCOCO_EDEVICE and v.status() == dc.DCOCO_OK
    assert got["accept_len"].tolist() == [3, 3] and got["next_token"].tolist() == [5, 5]
    want = torch.zeros_like(cache)
    want[0, 1, 14:] = new[0, 0, :2]
    want[0, 2, 14:] = new[0, 1, :2]
    assert torch.equal(cache, want) and torch.equal(other, want)
    outs = {k: torch.empty(2, **i32) for k in ("accept_len", "next_token")}
    with pytest.raises(dc.DcocoError) as e:
        dc.dcoco_tree_commit(v.handle, 2, tok, par, nxt, new, new, cache, other, table, ctx, path=tok.clone(),
                             new_len=ctx, **outs)
    assert e.value.status == dc.DCOCO_EINVAL
    with pytest.raises(ValueError):
        v.commit(tok, par.long(), nxt, new, new, cache, other, table, ctx)


# ------------------------------------------------------------------ sampling
def rows_of_logits(rng, R, V):
    """Rows of several kinds: spread, peaked, few levels, constant, mostly -inf, one token, NaN and -inf mixed, +inf."""
    x = 2 * rng.standard_normal((R, V))
    for r in range(R):
        kind = r % 9
        if kind == 1:
            x[r, rng.integers(0, V, 5)] += 10
        elif kind == 2:
            x[r] = np.round(x[r])
        elif kind == 3:
            x[r] = 1.25
        elif kind == 4:
            x[r, rng.random(V) < 0.95] = -np.inf
            x[r, rng.integers(0, V)] = 0.5
        elif kind == 5:
            x[r] = -np.inf
            x[r, rng.integers(0, V)] = -3
        elif kind == 6:
            x[r, rng.random(V) < 0.3] = np.nan
            x[r, rng.random(V) < 0.3] = -np.inf
            x[r, rng.integers(0, V)] = 2.0
        elif kind == 7:
            x[r, rng.integers(0, V, 2)] = np.inf
        elif kind == 8:
            x[r] *= 40
    return x.astype(np.float32)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [1, 7, 8, 33, 1000, 1025, 4099, 32001, 151936])
@pytest.mark.parametrize("what", ["plain", "top_k", "top_p", "min_p", "all"])
def test_sample(env, V, f32, what):
    torch, dc = env
    R = 27 if V > 20000 else 108
    rng = np.random.default_rng(V + f32)
    stride = (V + 7) // 8 * 8 + 8
    x = torch.full((R, stride), 99.0)  # what lies past the vocabulary must not count
    x[:, :V] = torch.from_numpy(rows_of_logits(rng, R, V))
    x = x.cuda() if f32 else x.bfloat16().cuda()
    logits = x[:, :V]
    t = rng.uniform(0.3, 1.5, R).astype(np.float32)
    t[rng.random(R) < 0.1] = 0
    u = rng.random(R).astype(np.float32)
    u[:6] = [0, 1 - 2 ** -24, 0.5, 2 ** -40, 0.999, 0.001]
    k = rng.choice([0, 1, 2, 5, 50, 400, 2000, V, V + 5, -1], R).astype(np.int32) if what in ("top_k", "all") else None
    p = rng.choice([0.0, 1e-6, 0.1, 0.5, 0.9, 0.99, 0.9999, 1.0, 1.5], R).astype(np.float32) if what in ("top_p", "all") else None
    q = rng.choice([0.0, 1e-4, 0.01, 0.3, 1.0, 2.0], R).astype(np.float32) if what in ("min_p", "all") else None
    cuda = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    tokens = torch.empty(R, dtype=torch.int32, device="cuda")
    logprob = torch.empty(R, device="cuda")
    dc.dcoco_sample(logits, cuda(u), tokens, temperature=cuda(t), top_k=cuda(k), top_p=cuda(p), min_p=cuda(q),
                    logprob=logprob)
    host = logits.float().cpu().numpy()
    near_rows = 0
    for r in range(R):
        tok, lp, near = tree_ref.sample_row(host[r], u[r], t[r], 0 if k is None else int(k[r]),
                                            1.0 if p is None else p[r], 0.0 if q is None else q[r])
        # sums of weights with fp32 relative errors: a border nearer than 2^-22 of the mass may go either way
        if near < 2.0 ** -22 and tok != int(tokens[r]):
            near_rows += 1
            continue
        assert tok == int(tokens[r]), (r, r % 9, tok, int(tokens[r]), near)
        if tok < 0:
            assert float(logprob[r]) == -np.inf
        else:  # a border token in or out moves the kept mass by less than its nearness
            assert abs(lp - float(logprob[r])) <= 2.0 ** -20 + 2.0 ** -22 * abs(lp) + (2.0 ** -12 if near < 2.0 ** -22 else 0)
    assert near_rows <= max(1, R // 20)


def test_sample_does_not_depend_on_rows(env):
    torch, dc = env
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (2 * torch.randn(300, 50008, generator=g, device="cuda")).bfloat16()
    u = torch.rand(300, generator=g, device="cuda")
    p = torch.full((300,), 0.9, device="cuda")
    tokens, lp = torch.empty(300, dtype=torch.int32, device="cuda"), torch.empty(300, device="cuda")
    dc.dcoco_sample(x, u, tokens, top_p=p, logprob=lp)
    for a, b in ((0, 1), (17, 20), (100, 150)):
        t2, l2 = torch.empty(b - a, dtype=torch.int32, device="cuda"), torch.empty(b - a, device="cuda")
        dc.dcoco_sample(x[a:b], u[a:b], t2, top_p=p[a:b], logprob=l2)
        assert torch.equal(t2, tokens[a:b]) and torch.equal(l2, lp[a:b])


def test_sample_shares(env):
    """Evenly spaced uniforms give every token its share."""
    torch, dc = env
    R = 4096
    x = torch.log(torch.tensor([0.3, 0.1, 0.4, 0.2])).repeat(R, 2).cuda()  # eight columns: two copies of four
    u = (torch.arange(R, device="cuda") + 0.5) / R
    tokens = torch.empty(R, dtype=torch.int32, device="cuda")
    dc.dcoco_sample(x, u, tokens, top_p=torch.full((R,), 0.65, device="cuda"))
    # shares .2 .2 .15 .15: 0.65 of the mass takes the .2s and two of the .15s
    share = torch.bincount(tokens.long(), minlength=8).double().cpu().numpy() / R
    assert np.allclose(share, np.array([.15, 0, .2, 0, .15, 0, .2, 0]) / .7, atol=2 / R)


# ------------------------------------------------------------------ distillation
CASES = [  # R, V, K
    (1, 1, 1), (3, 7, 2), (5, 1000, 16), (2, 4099, 64), (4, 32001, 300), (3, 151936, 16), (2, 20008, 1024), (9, 513, 5),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("R,V,K", CASES)
def test_distill(env, R, V, K, full, f32):
    torch, dc = env
    rng = np.random.default_rng(V * K)
    stride = (V + 7) // 8 * 8 + 16
    T = float(rng.choice([0.5, 1.0, 2.0]))
    x = torch.from_numpy((3 * rng.standard_normal((R, stride))).astype(np.float32))
    if V > 8:
        x[:, 1:V:5] = -math.inf
    x = (x if f32 else x.bfloat16()).cuda()
    logits = x[:, :V]
    host = logits.float().cpu().numpy()
    finite = [np.flatnonzero(np.isfinite(h)) for h in host]
    ids = np.stack([rng.choice(f, K, replace=K > len(f)) for f in finite]).astype(np.int32)
    teacher = (2 * rng.standard_normal((R, K))).astype(np.float32)
    if K > 3:
        ids[:, 1] = -1               # padding
        ids[:, 2] = ids[:, 0]        # one token twice
        teacher[:, 3] = -np.inf      # no share
        ids[0, 3] = V + 5            # out of range: padding too
    if R > 2:
        ids[2] = -1                  # a row of padding alone
    lse_t = (teacher.max(1) / T + 1.5).astype(np.float32) if full else None
    g = rng.standard_normal(R).astype(np.float32)
    if R > 1:
        g[1] = 0
    cuda = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    kw = dict(teacher_lse=cuda(lse_t), temperature=T)
    f = lambda: torch.empty(R, device="cuda")  # noqa: E731
    loss, lse, loss2, lse2 = f(), f(), f(), f()
    grad = torch.full_like(x, 7.0)
    both = torch.full_like(x, 7.0)
    dc.dcoco_distill_loss(logits, cuda(ids), cuda(teacher), loss=loss, lse=lse, **kw)
    dc.dcoco_distill_grad(logits, cuda(ids), cuda(teacher), lse, cuda(g), grad=grad[:, :V], **kw)
    dc.dcoco_distill_step(logits, cuda(ids), cuda(teacher), cuda(g), loss=loss2, lse=lse2, grad=both[:, :V], **kw)
    assert (grad[:, V:] == 7).all() and (both[:, V:] == 7).all()  # nothing past the vocabulary is written
    own = x.clone()
    dc.dcoco_distill_step(own[:, :V], cuda(ids), cuda(teacher), cuda(g), loss=f(), lse=f(), grad=own[:, :V], **kw)
    assert torch.equal(own[:, :V], both[:, :V]) and torch.equal(own[:, V:], x[:, V:])
    own = x.clone()
    dc.dcoco_distill_grad(own[:, :V], cuda(ids), cuda(teacher), lse, cuda(g), grad=own[:, :V], **kw)
    assert torch.equal(own[:, :V], grad[:, :V])
    eps = torch.finfo(x.dtype).eps / 2
    for r in range(R):
        rl, rlse, rg = tree_ref.distill_row(host[r], ids[r], teacher[r], T, None if lse_t is None else lse_t[r])
        rg = rg * g[r]
        reach = np.abs(host[r][np.isfinite(host[r])]).max() / T + 12  # the largest exponent, and the sum's
        e = 2.0 ** -22 * reach  # of a log-sum-exp, and relative of an exponential
        for a in (lse, lse2):
            assert abs(float(a[r]) - rlse) <= e
        P = max(1.0, float(np.exp(teacher[r].max() / T - lse_t[r])) * K if full else 1.0)
        term = T * T * P * (reach + np.abs(teacher[r][np.isfinite(teacher[r])]).max() / T + 8)
        for a in (loss, loss2):
            assert abs(float(a[r]) - rl) <= 2.0 ** -20 * term
        for a in (grad, both):
            got = f64(a[r, :V])
            tol = eps * np.abs(rg) + abs(g[r]) * T * P * 8 * e * np.where(np.abs(rg) > 0, 1, 0) * np.maximum(
                np.exp(np.where(np.isfinite(host[r]), host[r], -np.inf) / T - rlse), np.isin(np.arange(V), ids[r])) + 2.0 ** -126
            assert (np.abs(got - rg) <= tol).all(), (np.abs(got - rg) / tol).max()
        if (ids[r] < 0).all():
            assert float(loss[r]) == 0 and (grad[r, :V] == 0).all()
        if g[r] == 0:
            assert (grad[r, :V] == 0).all() and (both[r, :V] == 0).all()


def test_distill_gradient_by_differences(env):
    torch, dc = env
    R, V, K, T = 2, 40, 6, 1.5
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(R, V, generator=g, device="cuda")
    ids = torch.randint(0, V, (R, K), generator=g, device="cuda", dtype=torch.int32)
    t = torch.randn(R, K, generator=g, device="cuda")
    one = torch.ones(R, device="cuda")
    loss, lse, grad = torch.empty(R, device="cuda"), torch.empty(R, device="cuda"), torch.empty_like(x)
    dc.dcoco_distill_step(x, ids, t, one, loss=loss, lse=lse, grad=grad, temperature=T)
    h = 2.0 ** -6
    for v in range(V):
        d = []
        for s in (h, -h):
            y = x.clone()
            y[:, v] += s
            dc.dcoco_distill_loss(y, ids, t, loss=loss, lse=lse, temperature=T)
            d.append(loss.double().clone())
        # losses of order 10 in fp32 (error 2^-20 each), and the third derivative (below 1 / T) times h^2 / 6
        assert ((d[0] - d[1]) / (2 * h) - grad[:, v].double()).abs().max() <= 2.0 ** -20 / h + h * h / 6


# ------------------------------------------------------------------ extremes of values and temperatures
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [40, 5003, 40009])
@pytest.mark.parametrize("what", ["plain", "top_k", "top_p", "min_p", "all"])
def test_sample_extremes(env, V, f32, what):
    """Rows masked with the type's lowest value, in part or whole, of one sign, around zero; temperatures from 1e-30 on."""
    torch, dc = env
    R = 48
    rng = np.random.default_rng(V + 2 * f32)
    dt = torch.float32 if f32 else torch.bfloat16
    low = torch.finfo(dt).min
    x = (2 * rng.standard_normal((R, V))).astype(np.float32)
    for r in range(R):
        if r % 6 == 1:
            x[r, rng.random(V) < 0.7] = low
        elif r % 6 == 2:
            x[r] = low
        elif r % 6 == 3:
            x[r] = -np.abs(x[r]) - 1
        elif r % 6 == 4:
            x[r] = -np.abs(x[r])
            x[r, rng.integers(0, V, 3)] = [0.0, -0.0, 0.0]
        elif r % 6 == 5:
            x[r, rng.random(V) < 0.5] = -np.inf
            x[r, 0] = 1.0
    logits = torch.zeros(R, (V + 7) // 8 * 8, dtype=dt)
    logits[:, :V] = torch.from_numpy(x).clamp(min=low).to(dt)
    logits[:, :V][torch.from_numpy(np.isneginf(x))] = -math.inf
    logits = logits.cuda()[:, :V]
    t = rng.choice([1e-30, 1e-10, 1e-3, 0.02, 0.1, 1.0, 30.0, 1e6], R).astype(np.float32)
    u = rng.random(R).astype(np.float32)
    k = rng.choice([3, 40, V], R).astype(np.int32) if what in ("top_k", "all") else None
    p = rng.choice([0.3, 0.9, 0.999], R).astype(np.float32) if what in ("top_p", "all") else None
    q = rng.choice([1e-4, 0.01, 0.3], R).astype(np.float32) if what in ("min_p", "all") else None
    cuda = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    tokens = torch.empty(R, dtype=torch.int32, device="cuda")
    dc.dcoco_sample(logits, cuda(u), tokens, temperature=cuda(t), top_k=cuda(k), top_p=cuda(p), min_p=cuda(q))
    host, near_rows = logits.float().cpu().numpy(), 0
    for r in range(R):
        tok, _, near = tree_ref.sample_row(host[r], u[r], t[r], 0 if k is None else int(k[r]),
                                           1.0 if p is None else p[r], 0.0 if q is None else q[r])
        if near < 2.0 ** -22 and tok != int(tokens[r]):  # as in test_sample
            near_rows += 1
            continue
        assert tok == int(tokens[r]), (r, r % 6, float(t[r]), tok, int(tokens[r]), near)
    assert near_rows <= max(1, R // 20)


# ------------------------------------------------------------------ largest rows, graphs
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("what", ["top_k", "all"])
def test_sample_largest_vocabulary(env, what, f32):
    test_sample(env, 1 << 20, f32, what)


@pytest.mark.parametrize("f32", [False, True])
def test_distill_largest_vocabulary(env, f32):
    test_distill(env, 3, (1 << 20) - 3, 16, True, f32)


def test_calls_in_a_graph(env):
    """Sampling, commit and distillation recorded once, replayed over changed inputs, equal the eager calls."""
    torch, dc = env
    N, T, V, K, H, D, page = 3, 5, 5003, 8, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(8)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.empty(N * T, (V + 7) // 8 * 8, device="cuda")[:, :V]
    u, lp = torch.empty(N * T, device="cuda"), torch.empty(N * T, device="cuda")
    tok, picked = torch.empty(N, T, **i32), torch.empty(N * T, **i32)
    par = torch.tensor([-1, 0, 0, 1, 2], **i32).repeat(N, 1).contiguous()
    new = torch.empty(2, N, T, H, D, device="cuda").bfloat16()
    cache, other = (torch.empty(2, 6, page, H, D, device="cuda").bfloat16() for _ in range(2))
    table, ctx = torch.arange(6, **i32).view(3, 2), torch.tensor([0, 7, 15], **i32)
    v = dc.TreeVerifier(H, H, D, page, 2, max_batch=N, max_tree=T)
    outs = dict(path=torch.empty(N, T, **i32), **{k: torch.empty(N, **i32) for k in ("accept_len", "next_token", "new_len")})
    ids, teacher, one = torch.empty(N * T, K, **i32), torch.empty(N * T, K, device="cuda"), torch.ones(N * T, device="cuda")
    loss, lse = torch.empty(N * T, device="cuda"), torch.empty(N * T, device="cuda")
    grad = torch.empty(N * T, (V + 7) // 8 * 8, device="cuda")[:, :V]

    def fill():
        x.copy_(3 * torch.randn(N * T, V, generator=g, device="cuda"))
        x[:, 1::3] = -math.inf
        u.uniform_(generator=g)
        new.normal_(generator=g), cache.normal_(generator=g), other.normal_(generator=g)
        ids.copy_(torch.randint(0, V, (N * T, K), generator=g, device="cuda") // 3 * 3)
        teacher.normal_(generator=g)
        picked.random_(0, 3, generator=g)
        tok.random_(0, 3, generator=g)

    def calls():
        dc.dcoco_sample(x, u, picked, logprob=lp)
        dc.dcoco_tree_commit(v.handle, N, tok, par, picked.view(N, T) % 3, new, new, cache, other, table, ctx, **outs)
        dc.dcoco_distill_step(x, ids, teacher, one, loss=loss, lse=lse, grad=grad)
        return [t.clone() for t in (picked, lp, cache, other, *outs.values(), loss, lse, grad)]

    fill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for _ in range(3):
        fill()
        before = cache.clone(), other.clone()
        graph.replay()
        again = [t.clone() for t in got]
        cache.copy_(before[0]), other.copy_(before[1])
        for a, b in zip(again, calls()):
            assert torch.equal(a, b)
    assert v.status() == dc.DCOCO_OK


# ------------------------------------------------------------------ blocks that start or end at different times
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [16392, 40000, 151936])
def test_distill_beside_other_work(env, V, f32):
    """Clusters of 2 to 8 blocks a row, whose sums meet in shared memory, under work of another stream: the same bits."""
    torch, dc = env
    R, K = 300, 16
    g = torch.Generator(device="cuda").manual_seed(V + f32)
    x = (3 * torch.randn(R, V, generator=g, device="cuda")).to(torch.float32 if f32 else torch.bfloat16)
    top = x.float().topk(K, dim=1)
    ids, teacher = top.indices.int(), top.values.contiguous()
    weight = torch.rand(R, generator=g, device="cuda")

    def calls():
        loss, lse, loss2, lse2 = (torch.empty(R, device="cuda") for _ in range(4))
        grad = torch.empty_like(x)
        dc.dcoco_distill_loss(x, ids, teacher, loss=loss, lse=lse)
        dc.dcoco_distill_step(x, ids, teacher, weight, loss=loss2, lse=lse2, grad=grad)
        return loss, lse, loss2, lse2, grad

    quiet = calls()
    assert torch.equal(quiet[0], quiet[2]) and torch.equal(quiet[1], quiet[3])
    torch.cuda.synchronize()
    side, big = torch.cuda.Stream(), torch.randn(4096, 4096, generator=g, device="cuda").bfloat16()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        with torch.cuda.stream(side):
            for _ in range(8):
                big @ big
        for a, b in zip(calls(), quiet):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)


@pytest.mark.parametrize("T,H,g,D,page,dtype", [(65, 4, 1, 128, 64, "bfloat16"), (70, 3, 2, 64, 32, "float16"),
                                                (130, 2, 2, 128, 16, "float16"), (256, 2, 3, 64, 128, "bfloat16")])
def test_attention_short_units_in_a_row(env, T, H, g, D, page, dtype):
    """More than 64 rows a K/V head, units of one to three tiles, many a block: what the two halves of a block tell
    each other of a unit is not the next one's."""
    torch, dc = env
    rng = np.random.default_rng(T + D)
    ctx = [int(rng.choice([0, 1, 100, 128, 129, 250])) for _ in range(90)]
    a = Attn(torch, T, ctx, T, H, g, D, page, getattr(torch, dtype), tree_len=[int(rng.choice([1, T // 2, T])) for _ in ctx])
    v = a.verifier(dc)
    out, lse = a.run(v)
    for _ in range(20):
        again, lse2 = a.run(v)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    for n in rng.choice(90, 6, replace=False):
        one = slice(n, n + 1)
        b = Attn.__new__(Attn)
        b.__dict__.update(a.__dict__)
        b.q, b.k_new, b.v_new = a.q[one], a.k_new[one], a.v_new[one]
        b.table, b.ctx, b.sees, b.len = a.table[one], a.ctx[one], a.sees[one], a.len[one]
        b.check(out[one], lse[one])
    assert v.status() == dc.DCOCO_OK


@pytest.mark.parametrize("T,H,g,D,page,dtype", [(65, 4, 1, 128, 64, "bfloat16"), (70, 3, 2, 64, 32, "float16"),
                                                (130, 2, 2, 128, 16, "float16"), (20, 4, 4, 64, 64, "bfloat16"),
                                                (16, 4, 4, 128, 16, "bfloat16"), (1, 8, 4, 64, 32, "float16")])
def test_attention_alone_and_among_others(env, T, H, g, D, page, dtype):
    """Odd and even numbers of tiles and units in a block before a request's own: the same bits alone."""
    torch, dc = env
    rng = np.random.default_rng(T + D + 1)
    ctx = [int(rng.choice([0, 1, 100, 128, 129, 250, 500, 1500])) for _ in range(90)]
    a = Attn(torch, T, ctx, T, H, g, D, page, getattr(torch, dtype), tree_len=[int(rng.choice([1, T // 2, T])) for _ in ctx])
    v = a.verifier(dc)
    out, lse = a.run(v)
    for n in range(90):
        one = slice(n, n + 1)
        o, l = v.attention(a.q[one], a.k_new[one], a.v_new[one], a.k_cache, a.v_cache, a.t_table[one], a.t_ctx[one],
                           tree_mask=a.mask[one], tree_len=a.t_len[one])
        assert torch.equal(o[0], out[n]), n
        assert torch.equal(l[0], lse[n]), n


@pytest.mark.parametrize("R", [40, 200])
@pytest.mark.parametrize("V", [40001, 70001, 200003])
def test_sample_borders_past_the_first_window(env, V, R):
    """Evenly spread fp32 logits, a histogram bin a fair share of the mass: the first window round top-p's border
    misses some rows' borders, and the blocks go over the tokens again."""
    torch, dc = env
    rng = np.random.default_rng(V + R)
    x = np.zeros((R, (V + 7) // 8 * 8), np.float32)
    x[:, :V] = rng.random((R, V), dtype=np.float32)
    t = (1.5 / 2048 / rng.uniform(0.2, 3.0, R)).astype(np.float32)  # a bin is 0.2 to 3 temperatures wide
    p, u = rng.uniform(0.05, 0.97, R).astype(np.float32), rng.random(R).astype(np.float32)
    cuda = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    tokens, logprob = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    dc.dcoco_sample(cuda(x)[:, :V], cuda(u), tokens, temperature=cuda(t), top_p=cuda(p), logprob=logprob)
    for r in range(R):
        tok, lp, near = tree_ref.sample_row(x[r, :V], u[r], t[r], 0, p[r])
        if near < 2.0 ** -22 and tok != int(tokens[r]):  # as in test_sample
            continue
        assert tok == int(tokens[r]), (r, float(t[r]), tok, int(tokens[r]), near)
        assert abs(lp - float(logprob[r])) <= 2.0 ** -20 + 2.0 ** -22 * abs(lp) + (2.0 ** -12 if near < 2.0 ** -22 else 0)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [4099, 40000, 200003])
@pytest.mark.parametrize("what", ["top_p", "top_k", "both"])
def test_sample_many_tokens_share_the_border(env, V, f32, what):
    """A border that 1022 to 1090 tokens share: as many candidates as the list of one row holds, a few less, and more."""
    torch, dc = env
    counts = [1022, 1023, 1024, 1025, 1050, 1087, 1088, 1089, 1090]
    R = 3 * len(counts)
    rng = np.random.default_rng(V + f32)
    x = np.full((R, (V + 7) // 8 * 8), -20, np.float32)
    for r in range(R):
        at = rng.choice(V, counts[r % len(counts)] + 1, replace=False)
        x[r, at] = 0
        x[r, at[0]] = 5
    p = rng.uniform(0.2, 0.95, R).astype(np.float32) if what != "top_k" else None
    k = rng.integers(2, 512, R).astype(np.int32) if what != "top_p" else None
    u = rng.random(R).astype(np.float32)
    logits = torch.from_numpy(x).to(torch.float32 if f32 else torch.bfloat16).cuda()[:, :V]
    cuda = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    tokens, logprob = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    dc.dcoco_sample(logits, cuda(u), tokens, top_k=cuda(k), top_p=cuda(p), logprob=logprob)
    for r in range(R):
        tok, lp, near = tree_ref.sample_row(x[r, :V], u[r], None, 0 if k is None else int(k[r]), 1.0 if p is None else p[r])
        assert near > 2.0 ** -22, (r, near)  # as in test_sample (no border and no draw of these rows is near another outcome)
        assert tok == int(tokens[r]), (r, counts[r % len(counts)], tok, int(tokens[r]))
        assert abs(lp - float(logprob[r])) <= 2.0 ** -20 + 2.0 ** -22 * abs(lp)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [1500, 4099, 40000, 200003])
def test_sample_far_below_one_peak(env, V, f32):
    """One token, and all others 28.5 to 31 temperatures below it: no one of them has half a unit of the sums, 16
    together do.  A row with finite logits gives a token, and the first one for u = 0 (or NaN)."""
    torch, dc = env
    rows = [(gap, at, u) for gap in (28.5, 29, 30, 31) for at in (5, 700, V // 2, V - 1)
            for u in (0.0, math.nan, 2.0 ** -30, 0.5, 1 - 2.0 ** -23, 1 - 2.0 ** -24)]
    R = len(rows)
    x = np.zeros((R, (V + 7) // 8 * 8), np.float32)
    for r, (gap, at, _) in enumerate(rows):
        x[r, :V] = -gap
        x[r, at] = 0
    u = np.array([w for _, _, w in rows], np.float32)
    logits = torch.from_numpy(x).to(torch.float32 if f32 else torch.bfloat16).cuda()[:, :V]
    tokens, logprob = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    dc.dcoco_sample(logits, torch.from_numpy(u).cuda(), tokens, logprob=logprob)
    for r, (gap, at, _) in enumerate(rows):
        got, low = int(tokens[r]), math.exp(-gap)
        assert 0 <= got < V, (rows[r], got)
        total = 1 + (V - 1) * low
        before = got * low + (1 - low if at < got else 0)  # mass before the token
        mass = 1 if got == at else low
        target = 0.0 if np.isnan(u[r]) else float(u[r]) * total
        if target == 0:
            assert got == 0, rows[r]
        # sums of weights with fp32 relative errors, as in test_sample
        assert before <= target + 2.0 ** -22 * total and before + mass > target - 2.0 ** -22 * total, (rows[r], got)
        lp = (0 if got == at else -gap) - math.log(total)
        assert abs(lp - float(logprob[r])) <= 2.0 ** -20 + 2.0 ** -22 * abs(lp)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [1500, 40000, 200003])
@pytest.mark.parametrize("what", ["plain", "top_k", "top_p", "min_p"])
def test_sample_large_logits_over_small_temperatures(env, V, f32, what):
    """A step of the logits' type, over the temperature, is past fp32's range: the best tokens share the mass."""
    torch, dc = env
    rng = np.random.default_rng(V + f32)
    rows = [(top, t) for top in (1e38, -1e38, 1e30, -1e30, 3e12, -3e12, 1e9, 1.0) for t in (1e-30, 1e-18, 1e-9, 1e-4, 1e-2)]
    R = len(rows)
    x = np.zeros((R, (V + 7) // 8 * 8), np.float32)
    for r, (top, _) in enumerate(rows):
        x[r, :V] = top - abs(top) * rng.choice([0.02, 0.5, 1.0], V)  # (0.02: some steps of bf16)
        x[r, rng.choice(V, 5, replace=False)] = top
        x[r, rng.choice(V, 5, replace=False)] = -math.inf
    logits = torch.from_numpy(x).to(torch.float32 if f32 else torch.bfloat16).cuda()[:, :V]
    host = logits.float().cpu().numpy()
    u, t = rng.random(R).astype(np.float32), np.array([t for _, t in rows], np.float32)
    k = np.full(R, 40, np.int32) if what == "top_k" else None
    p = rng.uniform(0.1, 0.95, R).astype(np.float32) if what == "top_p" else None
    q = np.full(R, 0.1, np.float32) if what == "min_p" else None
    cuda = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    tokens, logprob = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    dc.dcoco_sample(logits, cuda(u), tokens, temperature=cuda(t), top_k=cuda(k), top_p=cuda(p), min_p=cuda(q),
                    logprob=logprob)
    for r in range(R):
        tok, lp, near = tree_ref.sample_row(host[r], u[r], t[r], 0 if k is None else int(k[r]),
                                            1.0 if p is None else p[r], 0.0 if q is None else q[r])
        if near < 2.0 ** -22 and tok != int(tokens[r]):  # as in test_sample
            continue
        assert tok == int(tokens[r]), (r, rows[r], tok, int(tokens[r]), near)
        assert abs(lp - float(logprob[r])) <= 2.0 ** -20 + 2.0 ** -22 * abs(lp) + (2.0 ** -12 if near < 2.0 ** -22 else 0)


# ------------------------------------------------------------------ handles larger than the call
@pytest.mark.parametrize("kw,most_mb", [
    (dict(max_batch=8, max_tree=64, q_heads=40, kv_heads=8, head_dim=128, page_size=64, max_pages=501), 64),
    (dict(max_batch=32, max_tree=64, q_heads=32, kv_heads=8, head_dim=128, page_size=16, max_pages=2048), 192),
    (dict(max_batch=32, max_tree=16, q_heads=32, kv_heads=8, head_dim=128, page_size=16, max_pages=512), 48),
])
def test_tree_workspace(env, kw, most_mb):
    """A handle's memory: the chunks that a call can have times the rows of the kernel that has them, 4 D + 8 bytes each."""
    torch, dc = env
    one = dc.dcoco_tree_create(1, 1, 1, 1, 64, 16, 1)  # what the first handle of a process loads is not counted
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    h = dc.dcoco_tree_create(**kw)
    taken = before - torch.cuda.mem_get_info()[0]
    dc.dcoco_tree_destroy(h)
    dc.dcoco_tree_destroy(one)
    assert taken <= most_mb << 20


@pytest.mark.parametrize("Hkv,g,D,page,tree", [(2, 4, 128, 16, 70), (2, 5, 64, 64, 64), (1, 1, 128, 32, 256),
                                               (2, 71, 64, 16, 5), (1, 33, 128, 64, 9)])
def test_attention_on_a_larger_handle(env, Hkv, g, D, page, tree):
    """Calls of 1 to max_tree nodes on one handle, full batch and longest contexts among them: the same bits as on a
    handle for just that many nodes, and as the 64-bit reference says."""
    torch, dc = env
    rng = np.random.default_rng(tree + g)
    N, top = 6, 40 * 128
    v = dc.TreeVerifier(Hkv * g, Hkv, D, page, top // page, max_batch=N, max_tree=tree)
    edges = [1, tree, 16 // g, 64 // g, 64 // g + 1, 128 // g, 128 // g + 1, 2 * (128 // g) + 1]
    for T in sorted({min(max(e, 1), tree) for e in edges}):
        ctx = [top] * (N - 2) + [int(rng.integers(0, top)), 129]
        a = Attn(torch, T, ctx, T, Hkv, g, D, page, torch.bfloat16)
        out, lse = a.run(v)
        fit = dc.TreeVerifier(Hkv * g, Hkv, D, page, top // page, max_batch=N, max_tree=T)
        o, l = a.run(fit)
        assert torch.equal(out, o) and torch.equal(lse, l)
        fit.close()
        one = slice(N - 1, N)
        b = Attn.__new__(Attn)
        b.__dict__.update(a.__dict__)
        b.q, b.k_new, b.v_new = a.q[one], a.k_new[one], a.v_new[one]
        b.table, b.ctx, b.sees, b.len = a.table[one], a.ctx[one], a.sees[one], a.len[one]
        b.check(out[one], lse[one])
    assert v.status() == dc.DCOCO_OK
