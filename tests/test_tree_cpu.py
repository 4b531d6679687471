"""CPU checks of the tree, sampling and distillation entries: refusals before
any CUDA call, the mask words, and the 64-bit references against brute force."""
import ctypes as C
import itertools
import math

import numpy as np
import pytest

import tree_ref


@pytest.fixture(scope="module")
def dc():
    import __graft_entry__
    __graft_entry__.build()
    import draft_correction_slot_gb300 as dc
    return dc


GOOD = dict(max_batch=4, max_tree=16, q_heads=8, kv_heads=2, head_dim=128, page_size=64, max_pages=8)


@pytest.mark.parametrize("kw,status", [
    (dict(max_batch=0), -1), (dict(max_batch=5000), -1), (dict(max_tree=0), -1), (dict(max_tree=257), -1),
    (dict(kv_heads=0), -1), (dict(q_heads=9), -1), (dict(q_heads=0), -1), (dict(max_pages=0), -1),
    (dict(max_pages=1 << 25), -1), (dict(page_size=0), -1), (dict(head_dim=96), -2), (dict(page_size=24), -2),
    (dict(page_size=8), -2), (dict(page_size=2048), -2), (dict(q_heads=258, kv_heads=2), -2), (dict(dtype=None), -2),
])
def test_tree_create_refuses_without_cuda(dc, kw, status):
    with pytest.raises(dc.DcocoError) as e:
        dc.dcoco_tree_create(**{**GOOD, **kw})
    assert e.value.status == status


def test_null_handles(dc):
    lib = dc.lib()
    assert lib.dcoco_tree_create(None, None) == -1
    assert lib.dcoco_tree_attention(None, 1, 1, None, None, None, None) == -1
    assert lib.dcoco_tree_commit(None, 1, 1, None, None, None, None, None, None) == -1
    assert lib.dcoco_tree_status(None) == -1
    assert lib.dcoco_tree_launches(None) == -1
    lib.dcoco_tree_destroy(None)


A = 1 << 20  # an aligned address that no call below may touch


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(vocab=(1 << 20) + 1, stride=(1 << 20) + 8), -1), (dict(dtype=1), -1),
    (dict(stride=96), -1), (dict(stride=108), -1), (dict(logits=None), -1), (dict(logits=A + 8), -1),
    (dict(u=None), -1), (dict(tokens=None), -1), (dict(rows=0, logits=None), 0),
])
def test_sample_refusals(dc, kw, status):
    a = {**dict(rows=2, vocab=100, logits=A, dtype=0, stride=104, u=A, tokens=A), **kw}
    assert dc.lib().dcoco_sample(a["rows"], a["vocab"], a["logits"], a["dtype"], a["stride"], None, None, None, None,
                                 a["u"], a["tokens"], None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(dtype=1), -1), (dict(stride=96), -1), (dict(k=0), -1),
    (dict(k=1025), -1), (dict(T=0.0), -1), (dict(T=-1.0), -1), (dict(T=math.inf), -1), (dict(T=math.nan), -1),
    (dict(logits=None), -1), (dict(ids=None), -1), (dict(teacher=None), -1), (dict(lse=None), -1),
    (dict(rows=0, logits=None, ids=None), 0),
])
@pytest.mark.parametrize("call", ["loss", "grad", "step"])
def test_distill_refusals(dc, call, kw, status):
    a = {**dict(rows=2, vocab=100, logits=A, dtype=2, stride=104, k=4, ids=A, teacher=A, T=1.0, lse=A), **kw}
    head = (a["rows"], a["vocab"], a["logits"], a["dtype"], a["stride"], a["k"], a["ids"], a["teacher"], None, a["T"])
    tail = {"loss": (A, a["lse"], None), "grad": (a["lse"], A, 2 * A, 104, None),
            "step": (A, A, a["lse"], 2 * A, 104, None)}[call]
    assert getattr(dc.lib(), f"dcoco_distill_{call}")(*head, *tail) == status


def test_distill_grad_refusals(dc):
    head = (2, 100, A, 2, 104, 4, A, A, None, 1.0)
    f = dc.lib().dcoco_distill_grad
    assert f(*head, A, None, 2 * A, 104, None) == -1       # no grad_loss
    assert f(*head, A, A, None, 104, None) == -1           # no grad
    assert f(*head, A, A, 2 * A + 4, 104, None) == -1      # misaligned
    assert f(*head, A, A, 2 * A, 96, None) == -1           # stride below the vocabulary
    assert f(*head, A, A, A, 112, None) == -1              # in place with another stride


def test_tree_mask_words(dc):
    import torch
    rng = np.random.default_rng(5)
    for t in (1, 2, 31, 32, 33, 64, 100):
        par = np.stack([[-1] + [int(rng.integers(-1 if n else 0, i)) for i in range(1, t)] for n in range(3)])
        words = dc.tree_mask(torch.from_numpy(par.astype(np.int32))).numpy()
        assert words.shape == (3, t, (t + 31) // 32)
        for n, i in itertools.product(range(3), range(t)):
            want, a = set(), i
            while a >= 0:
                want.add(a)
                a = par[n, a]
            got = {j for j in range(words.shape[2] * 32) if (int(words[n, i, j // 32]) >> (j % 32)) & 1}
            assert got == want


def test_python_checks(dc):
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        dc.dcoco_sample(x, x, x)  # not on the GPU
    with pytest.raises(ValueError):
        dc.dcoco_distill_loss(x, x.int(), x, loss=x, lse=x)


def test_sample_reference_by_enumeration():
    """The filters on a row whose shares can be read off: p = 0.4, 0.3, 0.2, 0.1 at ids 2, 0, 3, 1."""
    x = np.log(np.array([0.3, 0.1, 0.4, 0.2]))
    share = lambda **kw: np.bincount([tree_ref.sample_row(x, (i + .5) / 1000, **kw)[0] for i in range(1000)],  # noqa: E731
                                     minlength=4) / 1000
    assert np.allclose(share(), [.3, .1, .4, .2], atol=2e-3)
    assert np.allclose(share(k=2), [3 / 7, 0, 4 / 7, 0], atol=2e-3)
    assert np.allclose(share(p=0.65), [3 / 7, 0, 4 / 7, 0], atol=2e-3)
    assert np.allclose(share(p=0.75), [3 / 9, 0, 4 / 9, 2 / 9], atol=2e-3)
    assert np.allclose(share(q=0.6), [3 / 7, 0, 4 / 7, 0], atol=2e-3)
    assert np.allclose(share(k=3, p=0.5), [3 / 7, 0, 4 / 7, 0], atol=2e-3)  # 0.4 / 0.9 < 0.5
    assert np.allclose(share(p=0.0), [0, 0, 1, 0])
    assert share(t=0.0)[2] == 1
    tied = np.zeros(5)
    assert {tree_ref.sample_row(tied, i / 50, k=2)[0] for i in range(50)} == {0, 1}  # ties to the lowest ids


def test_distill_reference_gradient():
    rng = np.random.default_rng(3)
    x, ids, t = rng.standard_normal(12), np.array([3, 7, -1, 7]), rng.standard_normal(4)
    for T, lse in ((1.0, None), (2.5, 1.7)):
        _, _, grad = tree_ref.distill_row(x, ids, t, T, lse)
        for v in range(12):
            e = np.zeros(12)
            e[v] = 1e-5
            d = (tree_ref.distill_row(x + e, ids, t, T, lse)[0] - tree_ref.distill_row(x - e, ids, t, T, lse)[0]) / 2e-5
            assert abs(d - grad[v]) < 1e-8
