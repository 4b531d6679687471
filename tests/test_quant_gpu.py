"""Attention, commit and append on a cache in 8 bits, and the pages of a cache,
on the GPU against 64-bit references.

Attention's tolerances count roundings.  A context token's weight keeps 2^-10 of
itself (rounded to fp16, 2^-11, and cut into three parts of e5m2, 2^-11) and what
is below 2^-31 of the row's largest product of weight and scale is lost; a tree
node's weight is rounded to the 16-bit type.  A query's elements keep 2^-17 of the
row's largest.  Output: half a step of its type.  The rest are fp32 sums.  What is
written into the cache, and the pages, are compared exactly."""
import math

import numpy as np
import pytest

import quant_ref
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


def values(torch, payload):
    """The payload's values in 64 bits, whatever its strides."""
    return payload.contiguous().view(torch.uint8).cpu().contiguous().view(torch.float8_e4m3fn).double().numpy()


# ------------------------------------------------------------------ attention
class Attn:
    """A problem with random trees; unseen cache slots, scales and nodes hold NaN (and infinities)."""

    def __init__(self, torch, seed, ctx, T, Hkv, g, D, page, block, dtype, heads_first=False, tree_len=None,
                 mask="tree", extra_pages=3, v_exp=(-9, -5), poison=True):
        rng = np.random.default_rng(seed)
        self.torch, self.N, self.T, self.H, self.g, self.D = torch, len(ctx), T, Hkv, g, D
        self.page, self.block, self.dtype = page, block, dtype
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
        seen = np.zeros((self.pages, page), bool)
        for n in range(N):
            pos = np.arange(ctx[n])
            seen[table[n, pos // page], pos % page] = True
        live = seen.reshape(self.pages, page // block, block).any(2)  # blocks with a token in sight
        caches, scales = [], []
        for which in range(2):
            x = np.clip(rng.standard_normal((self.pages, page, Hkv, D)) * 110, -448, 448).astype(np.float32)
            e = rng.integers(-9, -5, (self.pages, page // block, Hkv)) if which == 0 else \
                rng.integers(*v_exp, (self.pages, page // block, Hkv))
            s = np.exp2(e).astype(np.float32)
            if which == 1 and seed % 2:
                s *= rng.uniform(0.8, 1.6, s.shape).astype(np.float32)  # any scale can be read
            if poison:
                x[~seen] = np.nan
                s[~live] = rng.choice([np.nan, np.inf, -1.0, 0.0], (int((~live).sum()), Hkv))
            x = torch.from_numpy(x).to(torch.float8_e4m3fn)
            if heads_first:
                x = x.view(torch.uint8).transpose(1, 2).contiguous().cuda().view(torch.float8_e4m3fn).transpose(1, 2)
            caches.append(x.cuda())
            scales.append(torch.from_numpy(s).cuda())
        self.k_cache, self.v_cache = caches
        self.k_scale, self.v_scale = scales
        if heads_first:  # scales with the heads in front
            self.k_scale, self.v_scale = (s.permute(2, 0, 1).contiguous().permute(1, 2, 0) for s in scales)
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
                elif mask == "tree":
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
        return dc.QuantTreeVerifier(self.H * self.g, self.H, self.D, self.page, self.max_pages, scale_tokens=self.block,
                                    **{**dict(max_batch=self.N, max_tree=self.T, dtype=self.dtype), **kw})

    def run(self, v, **kw):
        return v.attention(self.q, self.k_new, self.v_new, self.k_cache, self.v_cache, self.k_scale, self.v_scale,
                           self.t_table, self.t_ctx, tree_mask=self.mask, tree_len=self.t_len, **kw)

    def one(self, n):
        b = Attn.__new__(Attn)
        b.__dict__.update(self.__dict__)
        s = slice(n, n + 1)
        b.q, b.k_new, b.v_new, b.table, b.ctx = self.q[s], self.k_new[s], self.v_new[s], self.table[s], self.ctx[s]
        b.sees, b.len, b.N = self.sees[s], self.len[s], 1
        return b

    def reference(self, scale):
        """-> out, lse, and the tolerance of out and of lse."""
        torch, N, T, D = self.torch, self.N, self.T, self.D
        k8, v8 = values(torch, self.k_cache), values(torch, self.v_cache)
        ks, vs = (np.repeat(f64(s), self.block, 1) for s in (self.k_scale, self.v_scale))  # [pages, page, heads]
        q, k_new, v_new = f64(self.q), f64(self.k_new), f64(self.v_new)
        out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
        tol, tol_lse = np.zeros(q.shape), np.zeros(q.shape[:3])
        eps = torch.finfo(self.dtype).eps / 2
        for n in range(N):
            pos = np.arange(self.ctx[n])
            pg, at = self.table[n, pos // self.page], pos % self.page
            for t in range(self.len[n]):
                nodes = np.flatnonzero(self.sees[n, t, :self.len[n]])
                if len(pos) + len(nodes) == 0:
                    continue
                for hq in range(self.H * self.g):
                    h = hq // self.g
                    x = q[n, t, hq]
                    k = np.concatenate([k8[pg, at, h] * ks[pg, at, h][:, None], k_new[n, nodes, h]])
                    v = np.concatenate([v8[pg, at, h], v_new[n, nodes, h]])
                    f = np.concatenate([vs[pg, at, h], np.ones(len(nodes))])
                    we = np.concatenate([np.full(len(pos), 2.0 ** -10), np.full(len(nodes), max(eps, 2.0 ** -11))])
                    s = k @ x * scale
                    m = s.max()
                    w = np.exp(s - m)
                    total = w.sum()
                    val = v * f[:, None]
                    out[n, t, hq] = w @ val / total
                    lse[n, t, hq] = m + math.log(total)
                    err_s = ((D + 16) * 2.0 ** -24 * (np.abs(k) @ np.abs(x)).max()
                             + 2.0 ** -17 * np.abs(x).max() * np.abs(k).sum(1).max()) * abs(scale)
                    mag = np.abs(val)
                    tol[n, t, hq] = ((w * we) @ mag + (2 * err_s + 2.0 ** -20) * (w @ mag)) / total \
                        + eps * np.abs(out[n, t, hq]) + 2.0 ** -31 * (w * f).max() * np.abs(v).sum(0) / total + 2.0 ** -24
                    tol_lse[n, t, hq] = 2 * err_s + 2.0 ** -20 + 2.0 ** -22 * abs(lse[n, t, hq])
        return out, lse, tol, tol_lse

    def check(self, out, lse, scale=None):
        ref, rl, tol, tol_lse = self.reference(self.D ** -0.5 if scale is None else scale)
        got, gl = f64(out), f64(lse)
        assert np.isfinite(got).all()
        empty = np.isneginf(rl)
        assert (np.isneginf(gl) == empty).all() and (got[empty] == 0).all()
        live = ~empty
        if live.any():
            worst = (np.abs(got - ref)[live] / tol[live]).max()
            assert worst <= 1, worst
            worst = (np.abs(gl[live] - rl[live]) / tol_lse[live]).max()
            assert worst <= 1, worst


SHAPES = [
    # ctx, T, Hkv, g, D, page, block
    ([0], 1, 1, 1, 64, 16, 16),
    ([1], 1, 2, 4, 128, 16, 16),
    ([0, 1, 15, 16, 17], 3, 1, 3, 64, 16, 16),
    ([127, 128, 129, 255, 256], 1, 2, 4, 128, 64, 32),
    ([257, 5, 700], 16, 2, 4, 128, 16, 16),
    ([64, 333], 7, 3, 5, 64, 32, 16),
    ([1000], 33, 1, 8, 128, 128, 128),
    ([300, 0], 64, 2, 5, 128, 64, 64),
    ([130], 65, 1, 2, 64, 1024, 1024),
    ([77, 513], 130, 1, 1, 128, 16, 16),
    ([200], 256, 1, 2, 64, 32, 32),
    ([90], 5, 1, 71, 64, 32, 16),
    ([129], 2, 1, 128, 128, 256, 64),
    ([2500, 3], 4, 2, 2, 128, 64, 16),
    ([40, 1999, 640, 0, 1280, 128, 127], 2, 4, 4, 64, 64, 32),
    ([3000, 1, 4100], 8, 2, 4, 64, 512, 256),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention_shapes(env, i, dtype):
    torch, dc = env
    ctx, T, H, g, D, page, block = SHAPES[i]
    a = Attn(torch, 10 + i, ctx, T, H, g, D, page, block, getattr(torch, dtype), heads_first=i % 2 == 1)
    v = a.verifier(dc)
    for _ in range(2):  # twice: barriers and workspaces are ready for the next call
        out, lse = a.run(v)
        a.check(out, lse)
    assert v.status() == dc.DCOCO_OK


@pytest.mark.parametrize("T,H,g,D,page,block", [
    (1, 4, 4, 64, 32, 32), (3, 4, 5, 128, 16, 16), (16, 4, 2, 64, 16, 16), (12, 4, 5, 128, 64, 16), (30, 4, 4, 128, 64, 64),
    (70, 3, 4, 64, 128, 64)])
def test_attention_more_units_than_blocks(env, T, H, g, D, page, block):
    """Each block takes several units, of one tile and of many, with empty ones between."""
    torch, dc = env
    rng = np.random.default_rng(T)
    ctx = [int(rng.choice([0, 1, 100, 128, 400, 900, 2500, 4500])) for _ in range(70)]
    a = Attn(torch, T, ctx, T, H, g, D, page, block, torch.bfloat16, tree_len=[int(rng.choice([0, 1, T, T])) for _ in ctx])
    v = a.verifier(dc)
    out, lse = a.run(v)
    assert v.status() == dc.DCOCO_OK
    again, lse2 = a.run(v)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    for n in rng.choice(70, 12, replace=False):  # the 64-bit reference of every request would take minutes
        a.one(n).check(out[n:n + 1], lse[n:n + 1])
    dead = torch.tensor([[t >= a.len[n] for t in range(T)] for n in range(70)], device="cuda")
    assert (out[dead] == 0).all() and int(torch.isneginf(lse[dead]).sum()) == int(dead.sum()) * H * g


@pytest.mark.parametrize("mask", ["causal", "random", "none"])
@pytest.mark.parametrize("ctx", [[0, 0, 0], [37, 128, 1]])
@pytest.mark.parametrize("T", [1, 9, 40, 129])
def test_attention_masks_and_lengths(env, mask, ctx, T):
    """Empty rows (no context, nothing seen), and trees shorter than the call's nodes."""
    torch, dc = env
    a = Attn(torch, T, ctx, T, 2, 2, 64, 32, 16, torch.bfloat16, tree_len=[0, (T + 1) // 2, T], mask=mask)
    v = a.verifier(dc)
    out, lse = a.run(v, scale=0.3)
    a.check(out, lse, scale=0.3)
    assert v.status() == dc.DCOCO_OK


@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_attention_scale_of_any_sign(env, scale):
    torch, dc = env
    a = Attn(torch, 5, [300, 20], 6, 1, 3, 128, 16, 16, torch.bfloat16)
    a.check(*a.run(a.verifier(dc), scale=scale), scale=scale)


def test_attention_unseen_nodes_hold_nan(env):
    """Infinities and NaN in the K/V of a node reach the nodes that see it, and no others."""
    torch, dc = env
    a = Attn(torch, 3, [150, 20], 24, 2, 4, 128, 16, 16, torch.bfloat16, poison=False)
    v = a.verifier(dc)
    clean, _ = a.run(v)
    for j, value in ((5, math.nan), (11, math.inf), (17, -math.inf)):
        a.v_new[:, j] = value
        a.k_new[:, j] = math.nan
    hit = torch.from_numpy(a.sees[:, :, [5, 11, 17]].any(-1)).cuda()
    for _ in range(2):
        out, _ = a.run(v)
        assert torch.equal(out[~hit], clean[~hit])
        assert int(torch.isfinite(out[hit].float()).sum()) == 0
        a.k_new[:, [5, 11, 17]] = 0


def test_attention_nan_queries_stay_alone(env):
    """A query that holds NaN or infinities spoils its own row, and no other."""
    torch, dc = env
    a = Attn(torch, 4, [150, 20], 10, 2, 4, 128, 16, 16, torch.float16, poison=False)
    v = a.verifier(dc)
    clean, _ = a.run(v)
    hit = torch.zeros(a.q.shape[:3], dtype=torch.bool, device="cuda")
    for (t, h), value in (((2, 1), math.nan), ((5, 7), math.inf), ((9, 0), -math.inf)):
        a.q[:, t, h, 7] = value
        hit[:, t, h] = True
    out, _ = a.run(v)
    assert torch.equal(out[~hit], clean[~hit])
    assert bool(torch.isnan(out[hit]).all())


def test_attention_large_scores(env):
    """Scores of hundreds, rising and falling along the context: the running maximum moves a lot."""
    torch, dc = env
    for dtype in (torch.bfloat16, torch.float16):
        for up in (False, True):
            a = Attn(torch, 8, [1500, 900], 6, 1, 4, 128, 64, 16, dtype)
            for n in range(2):
                blocks = np.arange(-(-a.ctx[n] // 16))
                ramp = torch.from_numpy(np.exp2(np.round(np.linspace(-3, 3, len(blocks)) * (1 if up else -1)))).float().cuda()
                pg = a.t_table[n].long()[torch.from_numpy(blocks // 4).cuda()]
                a.k_scale[pg, torch.from_numpy(blocks % 4).cuda()] *= ramp[:, None]
            a.check(*a.run(a.verifier(dc), scale=1.0), scale=1.0)


@pytest.mark.parametrize("v_exp", [(-50, 40), (-12, 12), (-64, -60), (50, 60)])
def test_attention_scales_far_apart(env, v_exp):
    """V scales that differ by many powers of two within a tile."""
    torch, dc = env
    a = Attn(torch, 12, [700, 130], 3, 2, 2, 128, 32, 16, torch.bfloat16, v_exp=v_exp)
    a.check(*a.run(a.verifier(dc)))


def test_attention_zero_values(env):
    """Blocks of zeros at the least scale, beside others and alone."""
    torch, dc = env
    a = Attn(torch, 14, [400, 64], 2, 1, 4, 64, 16, 16, torch.bfloat16, v_exp=(-8, -7))
    for n, blocks in ((0, range(3, 11)), (1, range(4))):
        pg = a.t_table[n, list(blocks)].long()
        a.v_cache.view(torch.uint8)[pg] = 0
        a.v_scale[pg] = 2.0 ** -64
    a.check(*a.run(a.verifier(dc)))


def test_attention_heavy_token_of_small_value(env):
    """A token that takes nearly all the weight but whose value is small: the rest decides the output."""
    torch, dc = env
    a = Attn(torch, 16, [2000], 1, 1, 4, 128, 16, 16, torch.bfloat16, mask="none")
    pg = int(a.table[0, 3])
    q = a.q[0, 0].float().mean(0)
    a.q[0, 0] = q.to(a.dtype)
    a.k_cache[pg, 5, 0] = (q * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    a.k_scale[pg] = 2.0 ** -6
    a.v_cache.view(torch.uint8)[pg, 5] = 1
    scale = 15.0 / float((a.k_cache[pg, 5, 0].float() * 2.0 ** -6) @ a.q[0, 0, 0].float())
    a.check(*a.run(a.verifier(dc), scale=scale), scale=scale)


def test_attention_alone_and_among_others(env):
    """A request's output has the same bits whatever runs beside it, on a stream of its own or not."""
    torch, dc = env
    a = Attn(torch, 21, [900, 64, 2000, 0, 129, 700, 1, 350], 16, 2, 4, 128, 32, 16, torch.bfloat16)
    v = a.verifier(dc)
    out, lse = a.run(v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for n in range(a.N):
        s = slice(n, n + 1)
        got, gl = v.attention(a.q[s], a.k_new[s], a.v_new[s], a.k_cache, a.v_cache, a.k_scale, a.v_scale, a.t_table[s],
                              a.t_ctx[s], tree_mask=a.mask[s], stream=side if n % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(got[0], out[n]) and torch.equal(gl[0], lse[n])


def test_attention_shared_mask(env):
    torch, dc = env
    a = Attn(torch, 31, [30, 31, 200], 12, 1, 4, 64, 16, 16, torch.float16)
    a.sees[:] = a.sees[0]
    a.mask = a.mask[:1].contiguous()
    a.check(*a.run(a.verifier(dc)))


def test_attention_far_pages(env):
    """A pool of more than 2^32 bytes: pages at its end."""
    torch, dc = env
    a = Attn(torch, 41, [500], 4, 1, 4, 128, 64, 32, torch.bfloat16)
    pages = (1 << 32) // (64 * 128) + 20
    small = {n: getattr(a, n) for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    for name, x in small.items():
        pool = torch.empty(pages, *x.shape[1:], dtype=x.dtype, device="cuda")
        (pool.view(torch.uint8) if "cache" in name else pool)[-a.pages:] = x.view(torch.uint8) if "cache" in name else x
        setattr(a, name, pool)
    a.t_table += pages - a.pages
    out, lse = a.run(a.verifier(dc))
    a.__dict__.update(small)
    a.check(out, lse)


def test_attention_flags_bad_lengths_and_pages(env):
    """Lengths and pages out of range are clamped or left out by the kernel and recorded."""
    torch, dc = env
    a = Attn(torch, 51, [40, 40, 40, 40], 4, 1, 2, 64, 16, 16, torch.bfloat16)
    v = a.verifier(dc)
    good, _ = a.run(v)
    assert v.status() == dc.DCOCO_OK
    for bad in (-5, 1 << 20, -(1 << 31)):
        a.t_ctx[1] = bad
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
    a = Attn(torch, 61, [40, 3], 4, 2, 2, 64, 16, 16, torch.bfloat16)
    v = a.verifier(dc)
    before = dc.dcoco_tree_launches(v.handle)
    args = dict(q=a.q, k_new=a.k_new, v_new=a.v_new, k_cache=a.k_cache, v_cache=a.v_cache, k_scale=a.k_scale,
                v_scale=a.v_scale, page_table=a.t_table, ctx_len=a.t_ctx, out=torch.empty_like(a.q), tree_mask=a.mask)

    def call(batch=2, **kw):
        dc.dcoco_tree_attention_quant(v.handle, batch, **{**args, **kw})

    for kw in (dict(q=a.q.float()), dict(k_cache=a.k_cache.view(torch.uint8)), dict(k_cache=a.k_cache[:, :8]),
               dict(v_scale=a.v_scale.double()), dict(k_scale=a.k_scale[:-1]), dict(k_scale=a.k_scale.cpu()),
               dict(ctx_len=a.t_ctx.long()), dict(page_table=a.t_table[:, :1]), dict(tree_mask=a.mask[:, :2])):
        with pytest.raises(ValueError):
            call(**kw)
    odd = torch.zeros(a.pages, 16, 2, 72, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[..., :64]
    for kw in (dict(k_cache=odd), dict(k_scale=a.k_scale[:, :, :1].expand(a.pages, 1, 2)), dict(scale=math.nan)):
        with pytest.raises(dc.DcocoError) as e:
            call(**kw)
        assert e.value.status == dc.DCOCO_EINVAL
    plain = dc.TreeVerifier(4, 2, 64, 16, a.max_pages, max_batch=2, max_tree=4)
    wide = torch.zeros(a.pages, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    for call_ in (lambda: dc.dcoco_tree_attention_quant(plain.handle, 2, **args),
                  lambda: dc.dcoco_tree_attention(v.handle, 2, a.q, a.k_new, a.v_new, wide, wide, a.t_table, a.t_ctx,
                                                  out=torch.empty_like(a.q))):
        with pytest.raises(dc.DcocoError) as e:
            call_()
        assert e.value.status == dc.DCOCO_EUNSUPPORTED
    big = Attn(torch, 61, [40, 3, 1], 5, 2, 2, 64, 16, 16, torch.bfloat16)
    with pytest.raises(dc.DcocoError) as e:
        big.run(v)
    assert e.value.status == dc.DCOCO_EBATCH
    assert dc.dcoco_tree_launches(v.handle) == before
    assert v.status() == dc.DCOCO_OK


@pytest.mark.parametrize("T", [2, 6, 16])
@pytest.mark.parametrize("max_batch", [1, 200])  # partial results of one tile, and of several teams
def test_attention_nan_of_a_light_token(env, T, max_batch):
    """A NaN of V reaches the rows that see it however little its token weighs: here its scores, and those of all the
    tokens that share its partial result, lie hundreds below the rows' largest."""
    torch, dc = env
    a = Attn(torch, 71, [1000], T, 1, 4, 128, 16, 16, torch.bfloat16, mask="none", poison=False)
    a.k_scale[torch.from_numpy(a.table[0, 8:63]).long().cuda()] *= 64.0  # tokens 128 and on: scores of hundreds
    v = a.verifier(dc, max_batch=max_batch)
    clean, lse = a.run(v, scale=1.0)
    a.check(clean, lse, scale=1.0)
    for token, e in ((37, 7), (400, 90)):  # (the second one beside heavier ones in its tile)
        a.v_cache.view(torch.uint8)[int(a.table[0, token // 16]), token % 16, 0, e] = 0x7F
    out, lse2 = a.run(v, scale=1.0)
    keep = torch.ones(128, dtype=torch.bool, device="cuda")
    keep[[7, 90]] = False
    assert bool(torch.isnan(out[..., ~keep]).all())
    assert torch.equal(out[..., keep], clean[..., keep]) and torch.equal(lse, lse2)


@pytest.mark.parametrize("ends", [(-64, 64), (-80, 80), (-80, -80), (80, 80)])
@pytest.mark.parametrize("how", ["mixed", "tiles", "rise", "fall"])
@pytest.mark.parametrize("max_batch", [2, 200])
def test_attention_scales_at_both_ends(env, ends, how, max_batch):
    """V scales as far apart as they may be, within a tile, from tile to tile and from chunk to chunk: the tokens of
    the small ones count in the sum of the weights all the same."""
    torch, dc = env
    a = Attn(torch, 18, [2000, 300], 3, 1, 4, 128, 16, 16, torch.bfloat16)
    rng = np.random.default_rng(3)
    for n in range(2):
        b = np.arange(-(-a.ctx[n] // 16))
        low = {"mixed": rng.random(len(b)) < 0.5, "tiles": b // 8 % 2 == 0, "rise": b < len(b) / 2, "fall": b > len(b) / 2}[how]
        s = np.exp2(np.where(low, ends[0], ends[1])).astype(np.float32)
        a.v_scale[torch.from_numpy(a.table[n, b]).long().cuda(), 0, 0] = torch.from_numpy(s).cuda()
    a.check(*a.run(a.verifier(dc, max_batch=max_batch)))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("octaves", [3, 12, 17, 20, 23, 25])
def test_attention_light_token_decides(env, dtype, octaves):
    """Two tokens: a heavy one whose value is zero, and one lighter by so many octaves, which is all the output."""
    torch, dc = env
    a = Attn(torch, 19, [2], 16, 1, 4, 64, 16, 16, getattr(torch, dtype), mask="none")
    page, e4m3 = int(a.table[0, 0]), torch.float8_e4m3fn
    k, v = torch.zeros(2, 64, device="cuda"), torch.zeros(2, 64, device="cuda")
    k[1, 0] = -128
    v[1] = torch.linspace(-448, 448, 64, device="cuda")
    a.k_cache.view(torch.uint8)[page, :2, 0] = k.to(e4m3).view(torch.uint8)
    a.v_cache.view(torch.uint8)[page, :2, 0] = v.to(e4m3).view(torch.uint8)
    a.k_scale[page], a.v_scale[page] = 2.0 ** -3, 2.0 ** 8
    a.q.zero_()
    a.q[0, :, :, 0] = torch.linspace(1, 1.2, 64, device="cuda").view(16, 4).to(a.dtype)
    scale = octaves * math.log(2) / 16
    a.check(*a.run(a.verifier(dc), scale=scale), scale=scale)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("ctx", [0, 40])
def test_attention_infinite_queries_are_nan(env, value, ctx):
    """A query that holds an infinity gives NaN, not the zeros of a row that sees nothing, whatever sign the
    products have; a row that does see nothing stays empty."""
    torch, dc = env
    a = Attn(torch, 20, [ctx, ctx], 3, 1, 2, 64, 16, 16, torch.bfloat16, mask="causal", poison=False)
    a.k_new[..., 7] = torch.tensor([1.0, -1.0], device="cuda").view(2, 1, 1).to(a.dtype)
    clean, _ = a.run(a.verifier(dc))
    a.q[:, 1, 0, 7] = value
    out, lse = a.run(a.verifier(dc))
    hit = torch.zeros(2, 3, 2, dtype=torch.bool, device="cuda")
    hit[:, 1, 0] = True
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], clean[~hit])
    if ctx == 0:
        a.mask = torch.zeros(1, 3, 1, dtype=torch.int32, device="cuda")
        out, lse = a.run(a.verifier(dc))
        assert (out == 0).all() and bool(torch.isneginf(lse).all())


# ------------------------------------------------------------------ writing
class Cache:
    """A random cache of all layers on the GPU and its copy in 64 bits."""

    def __init__(self, torch, rng, L, pages, page, H, D, block, heads_first, poison=True):
        self.torch = torch
        self.gpu, self.want = {}, {}
        for name in ("k", "v"):
            codes = rng.integers(0, 256, (L, pages, page, H, D)).astype(np.uint8)
            if not poison:
                codes[(codes & 0x7F) == 0x7F] = 0
            x = torch.from_numpy(codes)
            if heads_first:
                x = x.transpose(2, 3).contiguous().cuda().transpose(2, 3)
            x = x.cuda()
            s = np.exp2(rng.integers(-9, 3, (L, pages, page // block, H))).astype(np.float32)
            self.gpu[name + "_cache"] = x.view(torch.float8_e4m3fn)
            self.gpu[name + "_scale"] = torch.from_numpy(s).cuda()
            self.want[name] = (values(torch, self.gpu[name + "_cache"]), s.astype(np.float64))

    def write(self, name, layer, block, table, ctx, rows):
        quant_ref.write(self.want[name][0][layer], self.want[name][1][layer], block, table, ctx, rows)

    def check(self):
        for name, (x, s) in self.want.items():
            got = values(self.torch, self.gpu[name + "_cache"])
            np.testing.assert_array_equal(got, x)
            np.testing.assert_array_equal(f64(self.gpu[name + "_scale"]), s)


def fresh(torch, rng, *shape):
    """K or V of new tokens: magnitudes over many powers of two, zeros, and a few infinities and NaN."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 7, shape[:-1])[..., None])
    x[rng.random(shape[:-1]) < 0.1] = 0
    x[rng.random(shape) < 0.002] = np.nan
    x[rng.random(shape) < 0.002] = np.inf
    return torch.from_numpy(x.astype(np.float32))


APPENDS = [
    # counts, ctx, L, H, D, page, block
    ([1], [0], 1, 1, 64, 16, 16),
    ([5, 0, 1, 40], [3, 7, 15, 16], 2, 2, 128, 16, 16),
    ([100, 33], [0, 50], 1, 3, 64, 64, 32),
    ([300], [77], 2, 1, 128, 128, 128),
    ([700, 1, 9], [1, 255, 0], 1, 2, 64, 256, 256),
    ([40] * 40 + [0] * 3 + [17], [(7 * i) % 33 for i in range(44)], 1, 2, 64, 32, 16),
    ([0, 0], [4, 0], 1, 1, 64, 16, 16),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append(env, i, dtype):
    torch, dc = env
    counts, ctx, L, H, D, page, block = APPENDS[i]
    rng = np.random.default_rng(i)
    N, dt = len(counts), getattr(torch, dtype)
    width = max(-(-(a + b) // page) for a, b in zip(counts, ctx)) + 1
    pages = N * width + 1
    table = rng.permutation(pages)[:N * width].reshape(N, width).astype(np.int32)
    total = sum(counts)
    new = [fresh(torch, rng, L, total + 2, 2 * H, D).to(dt).cuda()[:, :total, ::2] for _ in "kv"]  # strided; rows past the last
    c = Cache(torch, rng, L, pages, page, H, D, block, heads_first=i % 2 == 1)
    first = np.concatenate([[0], np.cumsum(counts)])
    v = dc.QuantTreeVerifier(H, H, D, page, width, max_batch=N, max_tree=1, dtype=dt, scale_tokens=block)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    got = v.append(i32(first), *new, **c.gpu, page_table=i32(table), ctx_len=i32(ctx))
    assert got.tolist() == [a + b for a, b in zip(counts, ctx)]
    rows = [f64(x) for x in new]
    for n in range(N):
        for layer in range(L):
            for name, x in zip("kv", rows):
                c.write(name, layer, block, table[n], ctx[n], x[layer, first[n]:first[n + 1]])
    c.check()
    assert v.status() == dc.DCOCO_OK


def test_append_in_pieces(env):
    """Token by token, in pieces, or at once: the same scales; payloads differ by the re-rounding alone."""
    torch, dc = env
    rng = np.random.default_rng(9)
    D, page, block, total = 64, 32, 32, 50
    new = [torch.from_numpy(rng.standard_normal((1, total, 1, D)) * np.exp2(np.arange(total) / 12)[:, None, None]).bfloat16().cuda()
           for _ in "kv"]
    v = dc.QuantTreeVerifier(1, 1, D, page, 2, max_batch=1, max_tree=1, scale_tokens=block)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    got = []
    for step in (1, 7, total):
        c = Cache(torch, np.random.default_rng(1), 1, 2, page, 1, D, block, False)
        for a in range(0, total, step):
            n = min(step, total - a)
            v.append(i32(0, n), *(x[:, a:a + n] for x in new), **c.gpu, page_table=table, ctx_len=i32(a))
            for name, x in zip("kv", new):
                c.write(name, 0, block, [1, 0], a, f64(x)[0, a:a + n])
        c.check()
        got.append(c.gpu)
    for g in got[:2]:
        assert torch.equal(g["k_scale"], got[2]["k_scale"]) and torch.equal(g["v_scale"], got[2]["v_scale"])
    x, s = f64(new[0])[0, :32, 0], float(got[0]["k_scale"][0, 1, 0, 0])
    back = values(torch, got[0]["k_cache"])[0, 1, :, 0] * s
    # half a step of the value, and per raise half of the least step: raises halve, together below one
    assert (np.abs(back - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * s).all()


def test_append_flags(env):
    """Requests with bad rows or lengths are left out, pages outside the pool are not written, both are recorded."""
    torch, dc = env
    rng = np.random.default_rng(10)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    new = [fresh(torch, rng, 1, 40, 1, 64).bfloat16().cuda() for _ in "kv"]
    v = dc.QuantTreeVerifier(1, 1, 64, 16, 2, max_batch=3, max_tree=1, scale_tokens=16)
    table = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    for first, ctx, tab, ok in (
            ([0, 10, 20, 30], [0, 0, 25], table, [1, 1, 0]),     # does not fit the table
            ([0, 10, 20, 30], [-1, 33, 2], table, [0, 0, 1]),    # lengths
            ([0, 10, 5, 15], [0, 0, 0], table, [1, 0, 1]),       # rows that go back
            ([0, 10, 20, 41], [0, 0, 0], table, [1, 1, 0]),      # rows past the last
            ([-1, 10, 20, 30], [0, 0, 0], table, [0, 1, 1]),
            ([0, 10, 20, 30], [0, 9, 0], [[0, 1], [2, 99], [-1, 5]], [1, 2, 0])):  # pages: 2: only the first
        c = Cache(torch, np.random.default_rng(1), 1, 6, 16, 1, 64, 16, False)
        got = v.append(i32(first), *new, **c.gpu, page_table=i32(tab), ctx_len=i32(ctx))
        assert v.status() == dc.DCOCO_EDEVICE and v.status() == dc.DCOCO_OK
        for n in range(3):
            x = [f64(a)[0, first[n]:first[n + 1]] for a in new]
            if ok[n] == 2:
                x = [a[:16 - ctx[n]] for a in x]
            if ok[n]:
                for name, a in zip("kv", x):
                    c.write(name, 0, 16, tab[n], ctx[n], a)
            elif tab is table:
                assert int(got[n]) == min(max(ctx[n], 0), 32)
        c.check()


@pytest.mark.parametrize("first", [[0, 4000, 0, 4000], [0, 700] * 20 + [0], [0, 3000, 3000, 10, 2900, 5, 3000], [0, 20, 0, 20, 0, 20, 0, 20]])
def test_append_rows_that_go_back(env, first):
    """A request whose rows end before they begin is left out; all others are written to their last token, also where
    requests share rows and have more of them together than there are."""
    torch, dc = env
    rng = np.random.default_rng(len(first))
    N, D, page = len(first) - 1, 64, 16
    total = max(first)
    width = -(-(total + 20) // page)
    ctx = rng.integers(0, 20, N)
    table = rng.permutation(N * width).reshape(N, width).astype(np.int32)
    new = [fresh(torch, rng, 2, total, 1, D).bfloat16().cuda() for _ in "kv"]
    c = Cache(torch, rng, 2, N * width, page, 1, D, page, False)
    v = dc.QuantTreeVerifier(1, 1, D, page, width, max_batch=N, max_tree=1, scale_tokens=page)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    got = v.append(i32(first), *new, **c.gpu, page_table=i32(table), ctx_len=i32(ctx)).tolist()
    assert v.status() == dc.DCOCO_EDEVICE
    rows = [f64(x) for x in new]
    for n in range(N):
        count = max(0, first[n + 1] - first[n])
        assert got[n] == ctx[n] + count
        for layer in range(2):
            for name, x in zip("kv", rows):
                c.write(name, layer, page, table[n], int(ctx[n]), x[layer, first[n]:first[n] + count])
    c.check()


def test_write_refusals(env):
    torch, dc = env
    v = dc.QuantTreeVerifier(1, 1, 64, 16, 2, max_batch=2, max_tree=4, scale_tokens=16)
    c = Cache(torch, np.random.default_rng(1), 1, 4, 16, 1, 64, 16, False).gpu
    i32 = dict(dtype=torch.int32, device="cuda")
    new = torch.zeros(1, 6, 1, 64, dtype=torch.bfloat16, device="cuda")
    first, ctx, table = torch.tensor([0, 2, 6], **i32), torch.zeros(2, **i32), torch.zeros(2, 2, **i32)
    args = dict(first=first, k_new=new, v_new=new, **c, page_table=table, ctx_len=ctx, new_len=ctx.clone())

    def append(batch=2, **kw):
        dc.dcoco_tree_append_quant(v.handle, batch, **{**args, **kw})

    for kw in (dict(first=first[:2]), dict(k_new=new.half()), dict(v_new=new[:, :5]), dict(k_cache=c["k_cache"].view(torch.uint8)),
               dict(k_scale=c["k_scale"].half()), dict(ctx_len=ctx.long()), dict(new_len=ctx.cpu())):
        with pytest.raises(ValueError):
            append(**kw)
    three = dict(first=torch.zeros(4, **i32), ctx_len=torch.zeros(3, **i32), new_len=torch.zeros(3, **i32),
                 page_table=torch.zeros(3, 2, **i32))
    for kw, status in ((dict(new_len=ctx), dc.DCOCO_EINVAL), (dict(batch=3, **three), dc.DCOCO_EBATCH),
                       (dict(k_new=torch.zeros(1, 6, 1, 68, dtype=torch.bfloat16, device="cuda")[..., :64]), dc.DCOCO_EINVAL)):
        with pytest.raises(dc.DcocoError) as e:
            append(**kw)
        assert e.value.status == status
    tree = torch.zeros(2, 4, **i32)
    new4 = torch.zeros(1, 2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    outs = {k: torch.empty(2, **i32) for k in ("accept_len", "next_token")}
    with pytest.raises(dc.DcocoError) as e:
        dc.dcoco_tree_commit_quant(v.handle, 2, tree, tree, tree, new4, new4, **c, page_table=table, ctx_len=ctx,
                                   path=tree.clone(), new_len=ctx, **outs)
    assert e.value.status == dc.DCOCO_EINVAL
    wide = torch.zeros(1, 4, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dc.DcocoError) as e:
        dc.dcoco_tree_commit(v.handle, 2, tree, tree, tree, new4, new4, wide, wide, table, ctx, path=tree.clone(),
                             new_len=ctx.clone(), **outs)
    assert e.value.status == dc.DCOCO_EUNSUPPORTED
    assert v.status() == dc.DCOCO_OK and dc.dcoco_tree_launches(v.handle) == 0


@pytest.mark.parametrize("N,T,L,H,D,page,block,dtype", [
    (1, 1, 1, 1, 64, 16, 16, "bfloat16"), (3, 16, 2, 2, 128, 16, 16, "float16"), (5, 40, 3, 1, 64, 32, 16, "bfloat16"),
    (2, 256, 1, 3, 64, 64, 64, "bfloat16"), (40, 7, 5, 8, 128, 32, 32, "bfloat16"), (4, 100, 2, 2, 64, 256, 256, "float16"),
])
@pytest.mark.parametrize("chain", [False, True])
def test_commit(env, N, T, L, H, D, page, block, dtype, chain):
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
    new = [fresh(torch, rng, L, N, T, 2 * H, D).to(dt).cuda()[:, :, :, ::2] for _ in "kv"]
    c = Cache(torch, rng, L, pages, page, H, D, block, heads_first=chain)
    v = dc.QuantTreeVerifier(H, H, D, page, width, max_batch=N, max_tree=T, dtype=dt, scale_tokens=block)
    cuda = lambda x: torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).cuda()  # noqa: E731
    got = v.commit(cuda(tokens), cuda(par), cuda(sampled), *new, **c.gpu, page_table=cuda(table), ctx_len=cuda(ctx),
                   tree_len=cuda(length))
    rows = [f64(x) for x in new]
    for n in range(N):
        path, nxt = tree_ref.walk(tokens[n], par[n], sampled[n], int(length[n]))
        assert got["path"][n].tolist() == path + [-1] * (T - len(path))
        assert int(got["accept_len"][n]) == max(0, len(path) - 1)
        assert int(got["next_token"][n]) == nxt
        assert int(got["new_len"][n]) == ctx[n] + len(path)
        for layer in range(L):
            for name, x in zip("kv", rows):
                c.write(name, layer, block, table[n], int(ctx[n]), x[layer, n, path])
    c.check()
    assert v.status() == dc.DCOCO_OK


def test_commit_flags(env):
    torch, dc = env
    v = dc.QuantTreeVerifier(1, 1, 64, 16, 2, max_batch=2, max_tree=4, scale_tokens=16)
    i32 = dict(dtype=torch.int32, device="cuda")
    tok, par = torch.tensor([[1, 2, 3, 4]] * 2, **i32), torch.tensor([[-1, 0, 1, 2]] * 2, **i32)
    nxt = torch.tensor([[2, 3, 4, 5]] * 2, **i32)
    new = torch.randn(1, 2, 4, 1, 64, device="cuda").bfloat16()
    c = Cache(torch, np.random.default_rng(1), 1, 4, 16, 1, 64, 16, False)
    table = torch.tensor([[0, 1], [2, 9]], **i32)  # request 0 runs past its table; request 1's second page is no page
    got = v.commit(tok, par, nxt, new, new, **c.gpu, page_table=table, ctx_len=torch.tensor([30, 14], **i32))
    assert v.status() == dc.DCOCO_EDEVICE and v.status() == dc.DCOCO_OK
    assert got["accept_len"].tolist() == [3, 3] and got["next_token"].tolist() == [5, 5]
    for name in "kv":
        c.write(name, 0, 16, [0, 1], 30, f64(new)[0, 0, :2])
        c.write(name, 0, 16, [2, 9], 14, f64(new)[0, 1, :2])
    c.check()


# ------------------------------------------------------------------ pages
def make_planes(torch, L, pages, heads_first=False):
    """A wide plane, a transposed one, a narrow one (4-byte steps) and one of a single layer."""
    mk = lambda *s: torch.randint(0, 255, s, dtype=torch.uint8, device="cuda")  # noqa: E731
    return [mk(L, pages, 16, 2, 64), mk(L, pages, 2, 16, 64).transpose(2, 3), mk(L, pages, 3, 4).view(torch.float32),
            mk(pages, 2, 16, 32).unsqueeze(0)[:, :, 1], mk(pages, L, 16, 80).transpose(0, 1)]


class Watched:
    """A PagePool and its reference; what a page holds is a tuple of its planes' bytes."""

    def __init__(self, env, pages, page, max_pages, rows, L=3):
        self.torch, self.dc = env
        self.planes = make_planes(self.torch, L, pages)
        self.pool = self.dc.PagePool(self.planes, page, max_pages, rows)
        self.ref = quant_ref.Pool(pages, page, max_pages, rows)
        self.ref.cache = self.content()

    def content(self):
        flat = [p.contiguous().view(self.torch.uint8).transpose(0, 1).reshape(p.shape[1], -1).cpu().numpy() for p in self.planes]
        return [tuple(f[i].tobytes() for f in flat) for i in range(len(flat[0]))]

    def i32(self, x):
        return self.torch.tensor(list(x), dtype=self.torch.int32, device="cuda")

    def set_len(self, row, n):
        self.pool.lens[row] = n
        self.ref.lens[row] = n

    def check(self):
        p, r = self.pool, self.ref
        assert p.held.tolist() == [len(t) for t in r.table]
        assert p.refs.tolist() == r.refs and p.lens.tolist() == r.lens
        table = p.table.cpu().tolist()
        for got, want in zip(table, r.table):
            assert got[:len(want)] == want
        got = self.content()
        for i in range(len(got)):
            if r.refs[i]:  # what a free page holds does not matter
                assert got[i] == r.cache[i], i


@pytest.mark.parametrize("pages,page,max_pages,rows", [(40, 16, 6, 9), (300, 4, 20, 60), (5000, 1, 40, 300), (1, 16, 1, 2)])
def test_pool_against_reference(env, pages, page, max_pages, rows):
    """Random calls, some of which cannot be served, in place."""
    torch, dc = env
    rng = np.random.default_rng(pages)
    w = Watched(env, pages, page, max_pages, rows)
    for step in range(30):
        n = int(rng.integers(0, rows + 1))
        bad = False
        kind = step % 5
        if kind in (0, 3):
            r = rng.integers(0, rows, n).tolist() if step % 2 else rng.permutation(rows)[:n].tolist()
            t = rng.integers(0, max_pages * page + 1, n).tolist()
            want = w.ref.reserve(r, t)
            assert w.pool.reserve(w.i32(r), w.i32(t)).tolist() == want
            bad = 0 in want
            for row in r:
                w.set_len(row, int(rng.integers(0, len(w.ref.table[row]) * page + 1)))
        elif kind in (1, 4):
            n //= 2
            empty = [i for i in range(rows) if not w.ref.table[i]]
            dst = rng.permutation(rows)[:n].tolist() if step % 2 or not empty else rng.choice(empty, n).tolist()
            src = rng.integers(0, rows, n).tolist()
            want = w.ref.fork(src, dst)
            assert w.pool.fork(w.i32(src), w.i32(dst)).tolist() == want
            bad = 0 in want
        else:
            r = rng.integers(0, rows, n // 2).tolist()
            w.ref.free(r)
            w.pool.free(w.i32(r))
        assert w.pool.status() == (dc.DCOCO_EDEVICE if bad else dc.DCOCO_OK)
        w.check()
        if step % 3 == 2:
            live = w.ref.compact()
            assert w.pool.compact().tolist() == [live] and w.pool.status() == dc.DCOCO_OK
            w.check()


def test_pool_large(env):
    """More rows, pages and forks than a step of the plan takes."""
    torch, dc = env
    rng = np.random.default_rng(7)
    w = Watched(env, 20000, 2, 8, 3000, L=1)
    rows = rng.permutation(3000)[:1400].tolist()
    t = rng.integers(0, 17, 1400).tolist()
    assert w.pool.reserve(w.i32(rows), w.i32(t)).tolist() == w.ref.reserve(rows, t)
    for r, n in zip(rows, t):
        w.ref.lens[r] = n
    w.pool.lens.copy_(w.i32(w.ref.lens))
    free = [i for i in range(3000) if not w.ref.table[i]]
    src, dst = rng.choice(rows, len(free)).tolist(), rng.permutation(free).tolist()
    assert w.pool.status() == dc.DCOCO_OK
    want = w.ref.fork(src, dst)  # (some sources hold nothing, and are forked into)
    assert 0 in want and 1 in want
    assert w.pool.fork(w.i32(src), w.i32(dst)).tolist() == want and w.pool.status() == dc.DCOCO_EDEVICE
    w.check()
    gone = rng.permutation(3000)[:2000].tolist()
    w.ref.free(gone)
    w.pool.free(w.i32(gone))
    assert w.pool.compact().tolist() == [w.ref.compact()]
    w.check()
    assert w.pool.status() == dc.DCOCO_OK


def test_pool_flags_bad_state(env):
    """Rows, lengths and entries out of range are recorded and never followed."""
    torch, dc = env
    w = Watched(env, 20, 16, 4, 4)
    p = w.pool
    assert p.reserve(w.i32([0, 1]), w.i32([40, 64])).tolist() == [1, 1] == w.ref.reserve([0, 1], [40, 64])
    w.set_len(0, 40)
    w.set_len(1, 64)
    for call in (lambda: p.reserve(w.i32([-1, 4, 1 << 30]), w.i32([1, 1, 1])), lambda: p.reserve(w.i32([2, 3]), w.i32([-1, 65])),
                 lambda: p.fork(w.i32([0, -1, 4]), w.i32([9, 2, 3])), lambda: p.fork(w.i32([0, 0]), w.i32([0, 1])),
                 lambda: p.fork(w.i32([0, 2]), w.i32([2, 3]))[1:]):
        done = call()
        assert done.sum() == 0 and p.status() == dc.DCOCO_EDEVICE and p.status() == dc.DCOCO_OK
    w.ref.fork([0], [2])
    w.check()
    p.free(w.i32([-1, 4]))
    assert p.status() == dc.DCOCO_EDEVICE
    w.check()
    p.lens[1] = 65  # more than it holds
    assert p.fork(w.i32([1]), w.i32([3])).tolist() == [0] and p.status() == dc.DCOCO_EDEVICE
    p.lens[1] = 64
    keep = p.table.clone()
    for page in (-1, 20, 1 << 30):
        p.table[1, 2] = page
        p.compact()
        assert p.status() == dc.DCOCO_EDEVICE and int(p.table[1, 2]) == page
    p.table.copy_(keep)
    p.table[1, 2] = 19  # nobody holds it
    p.free(w.i32([1]))
    assert p.status() == dc.DCOCO_EDEVICE and int(p.refs[19]) == 0
    assert int(p.refs[int(keep[1, 2])]) == 1


def test_pool_flags_entries_nobody_holds(env):
    """An entry to a page that nobody holds is recorded, wherever the page lies, and left as it is."""
    torch, dc = env
    for page in (1, 15):  # below the pages in use after compaction, above
        w = Watched(env, 20, 16, 4, 4)
        p = w.pool
        assert p.reserve(w.i32([0, 1, 2]), w.i32([64, 64, 48])).tolist() == [1, 1, 1]
        p.lens.copy_(w.i32([64, 64, 40, 0]))
        p.free(w.i32([0]))
        assert p.status() == dc.DCOCO_OK and p.refs.tolist() == [0] * 4 + [1] * 7 + [0] * 9
        held = p.table[1, 1].item()
        p.table[1, 1] = page
        assert int(p.compact()) == 7 and p.status() == dc.DCOCO_EDEVICE and int(p.table[1, 1]) == page
        assert p.compact().tolist() == [7]  # the other entries are in order
        assert p.table[2, :3].tolist() == [1, 2, 3] and p.refs.tolist() == [1] * 7 + [0] * 13 and held == 5
    # a fork: of a full page, and of the one filled in part
    for row, at in ((0, 1), (0, 2)):
        w = Watched(env, 20, 16, 4, 4)
        p = w.pool
        assert p.reserve(w.i32([0]), w.i32([40])).tolist() == [1]
        p.lens[0] = 40
        p.table[row, at] = 17
        assert p.fork(w.i32([0]), w.i32([1])).tolist() == [1] and p.status() == dc.DCOCO_EDEVICE
        assert int(p.refs[17]) == 0
        assert p.refs[:5].tolist() == ([2, 1, 1, 1, 0] if at == 1 else [2, 2, 1, 1, 0])


def test_pool_refusals(env):
    torch, dc = env
    w = Watched(env, 8, 16, 4, 4)
    p = w.pool
    state = (p.table, p.held, p.lens, p.refs)
    one = w.i32([0])
    for call in (lambda: dc.dcoco_pages_free(p.handle, one.long(), *state),
                 lambda: dc.dcoco_pages_free(p.handle, one, p.table[:, :3], *state[1:]),
                 lambda: dc.dcoco_pages_free(p.handle, one, p.table, p.held[:2], *state[2:]),
                 lambda: dc.dcoco_pages_fork(p.handle, dc.page_planes(make_planes(torch, 1, 9)), one, one, *state),
                 lambda: dc.dcoco_pages_fork(p.handle, p.planes, one, w.i32([0, 1]), *state),
                 lambda: dc.page_planes([torch.zeros(2, 4, 8, 2, device="cuda")[..., 0]]),
                 lambda: dc.page_planes([torch.zeros(2, 4, 8, device="cuda"), torch.zeros(2, 5, 8, device="cuda")]),
                 lambda: dc.page_planes([torch.zeros(2, 4, device="cuda")])):
        with pytest.raises(ValueError):
            call()
    many = w.i32([0, 1, 2, 3, 0])
    for call, status in ((lambda: dc.dcoco_pages_free(p.handle, many, *state), dc.DCOCO_EBATCH),
                         (lambda: dc.dcoco_pages_reserve(p.handle, many, many, p.table, p.held, p.refs), dc.DCOCO_EBATCH),
                         (lambda: dc.dcoco_pages_free(p.handle, one, p.table, p.held, None, p.refs), dc.DCOCO_EINVAL),
                         (lambda: dc.dcoco_pages_fork(p.handle, dc.page_planes(
                             [torch.zeros(1, 8, 6, dtype=torch.uint8, device="cuda")]), one, w.i32([1]), *state), dc.DCOCO_EINVAL),
                         (lambda: dc.dcoco_pages_fork(p.handle, dc.page_planes(
                             [torch.zeros(1, 1, 8, device="cuda").expand(3, 8, 8)]), one, w.i32([1]), *state), dc.DCOCO_EINVAL),
                         (lambda: dc.dcoco_pages_fork(p.handle, dc.page_planes(
                             [torch.zeros(1, 8, 8, device="cuda")] * 65), one, w.i32([1]), *state), dc.DCOCO_EINVAL)):
        with pytest.raises(dc.DcocoError) as e:
            call()
        assert e.value.status == status
    assert dc.dcoco_pages_launches(p.handle) == 0 and p.status() == dc.DCOCO_OK
    assert p.reserve(w.i32([]), w.i32([])).tolist() == [] and dc.dcoco_pages_launches(p.handle) == 0


def test_pool_lists_have_one_axis(env):
    """A list of rows of another shape is refused, not cut off."""
    torch, dc = env
    w = Watched(env, 8, 16, 4, 4)
    p, two = w.pool, w.i32([0, 1, 2, 3]).view(2, 2)
    for rows in (two, two[0, 0]):
        for call in (lambda: p.free(rows), lambda: p.reserve(rows, rows), lambda: p.fork(rows, rows)):
            with pytest.raises(ValueError):
                call()
    assert dc.dcoco_pages_launches(p.handle) == 0 and p.status() == dc.DCOCO_OK


def test_pool_forks_in_a_row(env):
    """A row cannot be forked into and be a source in one call: the fork into it is served, the one from it is not."""
    torch, dc = env
    w = Watched(env, 20, 16, 4, 4)
    w.pool.reserve(w.i32([0]), w.i32([40]))
    w.ref.reserve([0], [40])
    w.set_len(0, 40)
    for order in ([0, 1], [1, 0]):
        src, dst = np.array([0, 1])[order].tolist(), np.array([1, 2])[order].tolist()
        want = [int(a == 0) for a in src]
        assert w.ref.fork(src, dst) == want and w.pool.fork(w.i32(src), w.i32(dst)).tolist() == want
        assert w.pool.status() == dc.DCOCO_EDEVICE
        w.check()
        w.ref.free([1])
        w.pool.free(w.i32([1]))
        w.check()


def test_pool_out_of_place(env):
    """Compaction into other arrays leaves the state as it was, but for the pages' content."""
    torch, dc = env
    w = Watched(env, 30, 16, 4, 5)
    rows, t = [0, 1, 2, 3], [64, 20, 50, 64]
    w.pool.reserve(w.i32(rows), w.i32(t))
    w.ref.reserve(rows, t)
    w.ref.free([0, 2])
    w.pool.free(w.i32([0, 2]))
    p = w.pool
    table, refs = p.table.clone(), p.refs.clone()
    out, refs_out, live = torch.full_like(table, -5), torch.full_like(refs, -5), torch.empty(1, dtype=torch.int32, device="cuda")
    dc.dcoco_pages_compact(p.handle, p.planes, p.table, p.held, p.refs, page_table_out=out, refs_out=refs_out, live=live)
    assert torch.equal(p.table, table) and torch.equal(p.refs, refs)
    assert live.tolist() == [w.ref.compact()] and refs_out.tolist() == w.ref.refs
    for row, want in enumerate(w.ref.table):
        assert out[row].tolist() == want + [-5] * (4 - len(want))
    got = w.content()
    for i in range(30):
        if w.ref.refs[i]:
            assert got[i] == w.ref.cache[i]


# ------------------------------------------------------------------ together
def serving(env, seed=3):
    """A cache of two layers with its pool, two prompts appended, one forked twice."""
    torch, dc = env
    g = torch.Generator(device="cuda").manual_seed(seed)
    L, pages, page, H, hq, D, block, rows = 2, 40, 16, 2, 4, 64, 16, 5
    cache = {n: torch.zeros(L, pages, page, H, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for n in ("k_cache", "v_cache")}
    cache.update({n: torch.ones(L, pages, page // block, H, device="cuda") for n in ("k_scale", "v_scale")})
    pool = dc.PagePool(list(cache.values()), page, 8, rows)
    v = dc.QuantTreeVerifier(hq, H, D, page, 8, max_batch=rows, max_tree=6, scale_tokens=block)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    assert pool.reserve(i32(0, 3), i32(37, 70)).tolist() == [1, 1]
    prompt = [randn(L, 37 + 70, H, D) for _ in "kv"]
    first = i32(0, 37, 37, 37, 107, 107)  # rows 1, 2 and 4 get nothing
    pool.lens.copy_(v.append(first, *prompt, **cache, page_table=pool.table, ctx_len=pool.lens))
    return cache, pool, v, i32, randn, prompt


def test_serving_step(env):
    """Prompts, forks, a tree a row, its commit, freeing and compaction: what attends afterwards finds what a cache
    of the same tokens without any of it holds."""
    torch, dc = env
    cache, pool, v, i32, randn, prompt = serving(env)
    L, H, D, T = 2, 2, 64, 6
    assert pool.fork(i32(0, 3), i32(1, 4)).tolist() == [1, 1]
    assert pool.reserve(i32(0, 1, 3, 4), pool.lens[[0, 1, 3, 4]] + T).tolist() == [1] * 4
    parents = i32(-1, 0, 0, 1, 2, 4).repeat(5, 1)
    tokens = torch.randint(0, 3, (5, T), device="cuda", dtype=torch.int32)
    sampled = torch.randint(0, 3, (5, T), device="cuda", dtype=torch.int32)
    k_new, v_new = randn(L, 5, T, H, D), randn(L, 5, T, H, D)
    length = torch.where(pool.held > 0, T, 0).int()
    before = pool.lens.clone()
    done = v.commit(tokens, parents, sampled, k_new, v_new, **cache, page_table=pool.table, ctx_len=before, tree_len=length)
    pool.lens.copy_(done["new_len"])
    q, kn, vn = randn(5, 1, 4, D), randn(5, 1, H, D), randn(5, 1, H, D)
    layer = lambda i: {n: x[i] for n, x in cache.items()}  # noqa: E731
    out, lse = v.attention(q, kn, vn, **layer(1), page_table=pool.table, ctx_len=pool.lens)
    assert v.status() == dc.DCOCO_OK and pool.status() == dc.DCOCO_OK
    # the same tokens, row by row, into a cache of their own
    alone = {n: torch.zeros_like(x.view(torch.uint8) if "cache" in n else x) for n, x in cache.items()}
    alone = {n: x.view(torch.float8_e4m3fn) if "cache" in n else x + 1 for n, x in alone.items()}
    table = torch.arange(40, device="cuda", dtype=torch.int32).view(5, 8)
    lens = torch.zeros(5, dtype=torch.int32, device="cuda")
    source = {0: slice(0, 37), 1: slice(0, 37), 3: slice(37, 107), 4: slice(37, 107)}
    for piece in ("prompt", "path"):
        rows, counts = [[], []], []
        for n in range(5):
            path = [t for t in done["path"][n].tolist() if t >= 0]
            counts.append(0 if n == 2 else 70 if piece == "prompt" and n > 2 else 37 if piece == "prompt" else len(path))
            if n != 2:
                for r, p, t in zip(rows, prompt, (k_new, v_new)):
                    r.append(p[:, source[n]] if piece == "prompt" else t[:, n, path])
        first = i32(0, *np.cumsum(counts).tolist())
        lens = v.append(first, *(torch.cat(r, 1) for r in rows), **alone, page_table=table, ctx_len=lens)
    assert torch.equal(lens, pool.lens)
    want, want_lse = v.attention(q, kn, vn, **{n: x[1] for n, x in alone.items()}, page_table=table, ctx_len=lens)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # two rows go, the rest moves together: nobody notices
    pool.free(i32(0, 4, 0))
    live = pool.compact()
    assert int(live) == int((pool.refs > 0).sum()) and int(pool.table[[1, 3]][:, :1].max()) < int(live)
    again, _ = v.attention(q, kn, vn, **layer(1), page_table=pool.table, ctx_len=pool.lens)
    assert torch.equal(again[[1, 3]], want[[1, 3]])
    assert v.status() == dc.DCOCO_OK and pool.status() == dc.DCOCO_OK


def test_calls_in_a_graph(env):
    """A step recorded once and replayed gives what the calls give, on two copies of the state."""
    torch, dc = env
    results = []
    for graphed in (False, True):
        cache, pool, v, i32, randn, prompt = serving(env)
        T, rows = 6, 5
        src, dst, parents = i32(3, 0), i32(1, 2), i32(-1, 0, 0, 1, 2, 4).repeat(5, 1)
        all_rows, want = i32(*range(rows)), torch.zeros(rows, dtype=torch.int32, device="cuda")
        tokens, sampled = (torch.randint(0, 3, (rows, T), device="cuda", dtype=torch.int32,
                                         generator=torch.Generator(device="cuda").manual_seed(s)) for s in (1, 2))
        k_new, v_new, q = randn(2, rows, T, 2, 64), randn(2, rows, T, 2, 64), randn(rows, T, 4, 64)
        outs = {}

        def step():
            pool.free(dst)
            outs["done"] = pool.fork(src, dst)
            want.copy_(pool.lens + T)
            pool.reserve(all_rows, want)
            outs["out"], outs["lse"] = v.attention(q, k_new[0], v_new[0], **{n: x[0] for n, x in cache.items()},
                                                   page_table=pool.table, ctx_len=pool.lens)
            got = v.commit(tokens, parents, sampled, k_new, v_new, **cache, page_table=pool.table, ctx_len=pool.lens.clone())
            pool.lens.copy_(got["new_len"])
            outs.update(got)
            pool.compact()

        if graphed:
            # warm up on the side, on another state
            side = torch.cuda.Stream()
            keep = {n: x.clone() for n, x in dict(cache, table=pool.table, held=pool.held, lens=pool.lens, refs=pool.refs).items()}
            with torch.cuda.stream(side):
                side.wait_stream(torch.cuda.default_stream())
                step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for n, x in keep.items():
                (cache[n] if n in cache else getattr(pool, n)).copy_(x)
            for _ in range(3):
                graph.replay()
        else:
            for _ in range(3):
                step()
        torch.cuda.synchronize()
        assert v.status() == dc.DCOCO_OK and pool.status() == dc.DCOCO_OK
        results.append([*(x.clone() for x in outs.values()), pool.table, pool.held, pool.lens, pool.refs,
                        cache["k_cache"].view(torch.uint8), cache["v_scale"]])
    for a, b in zip(*results):
        assert torch.equal(a, b)
