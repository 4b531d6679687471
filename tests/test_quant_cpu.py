"""CPU checks of the calls on a cache in 8 bits and of its pages: refusals before
any CUDA call, and the references against what defines them."""
import ctypes as C

import numpy as np
import pytest

import quant_ref


@pytest.fixture(scope="module")
def dc():
    import __graft_entry__
    __graft_entry__.build()
    import draft_correction_slot_gb300 as dc
    return dc


GOOD = dict(max_batch=4, max_tree=16, q_heads=8, kv_heads=2, head_dim=128, page_size=64, max_pages=8, scale_tokens=32)


@pytest.mark.parametrize("kw,status", [
    (dict(max_batch=0), -1), (dict(max_tree=257), -1), (dict(q_heads=9), -1), (dict(max_pages=1 << 25), -1),
    (dict(head_dim=96), -2), (dict(page_size=24), -2), (dict(dtype=None), -2), (dict(scale_tokens=0), -2),
    (dict(scale_tokens=8), -2), (dict(scale_tokens=24), -2), (dict(scale_tokens=128), -2), (dict(scale_tokens=-32), -2),
])
def test_create_refuses_without_cuda(dc, kw, status):
    with pytest.raises(dc.DcocoError) as e:
        dc.dcoco_tree_create_quant(**{**GOOD, **kw})
    assert e.value.status == status


@pytest.mark.parametrize("kw", [dict(num_pages=0), dict(num_pages=(1 << 20) + 1), dict(page_size=0), dict(max_pages=0),
                                dict(max_rows=0), dict(max_rows=(1 << 20) + 1), dict(page_size=1 << 20, max_pages=1 << 11)])
def test_pages_create_refuses_without_cuda(dc, kw):
    with pytest.raises(dc.DcocoError) as e:
        dc.dcoco_pages_create(**{**dict(num_pages=8, page_size=16, max_pages=4, max_rows=2), **kw})
    assert e.value.status == -1


def test_null_handles(dc):
    lib = dc.lib()
    assert lib.dcoco_tree_create_quant(None, 16, None) == -1
    assert lib.dcoco_tree_attention_quant(None, 1, 1, None, None, None, None, None) == -1
    assert lib.dcoco_tree_commit_quant(None, 1, 1, None, None, None, None, None, None, None) == -1
    assert lib.dcoco_tree_append_quant(None, 1, None, None, None, None) == -1
    assert lib.dcoco_pages_create(None, None) == -1
    assert lib.dcoco_pages_reserve(None, None, 1, None, None, None, None) == -1
    assert lib.dcoco_pages_fork(None, None, 0, None, 1, None, None, None, None) == -1
    assert lib.dcoco_pages_free(None, None, 1, None, None) == -1
    assert lib.dcoco_pages_compact(None, None, 0, None, None, 8, None, None, None) == -1
    assert lib.dcoco_pages_status(None) == -1
    assert lib.dcoco_pages_launches(None) == -1
    lib.dcoco_pages_destroy(None)


def test_exported_names(dc):
    lib = C.CDLL(dc.LIB_PATH)
    for n in dc.EXPORTED:
        assert hasattr(lib, n) and callable(getattr(dc, n))


def test_python_checks(dc):
    import torch
    with pytest.raises(ValueError):
        dc.page_planes([torch.zeros(2, 4, 8)])  # not on the GPU
    h = dc._TreeHandle()
    h.sizes = (1, 1, 64, 16, 1, torch.bfloat16)  # a handle for a cache in 16 bits
    x = torch.zeros(1, 1, 1, 64)
    for call in (lambda: dc.dcoco_tree_attention_quant(h, 1, x, x, x, x, x, x, x, x, x, out=x),
                 lambda: dc.dcoco_tree_append_quant(h, 1, x, x, x, x, x, x, x, x, x, new_len=x)):
        with pytest.raises(dc.DcocoError) as e:
            call()
        assert e.value.status == -2


def test_reference_rounding():
    """Every e4m3 value is its own nearest, midpoints go to the even one, as torch's conversion has it."""
    import torch
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    ok = np.isfinite(vals)
    assert (quant_ref.e4m3(vals[ok]) == vals[ok]).all()
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * np.exp2(rng.integers(-12, 8, 20000)), (vals[ok][1:] + vals[ok][:-1]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    assert (quant_ref.e4m3(x) == torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()).all()
    assert np.isnan(quant_ref.e4m3([np.inf, -np.inf, np.nan])).all()
    assert quant_ref.need(448.0) == 1 and quant_ref.need(448.5) == 2 and quant_ref.need(0.0) == 2.0 ** -64
    assert quant_ref.need(3e38) == 2.0 ** 64 and quant_ref.need(1e-30) == 2.0 ** -64


def test_reference_pool():
    p = quant_ref.Pool(6, 4, 3, 4)
    assert p.reserve([1, 0, 1, 9], [9, 4, 4, 1]) == [1, 1, 0, 0] and p.table[1] == [0, 1, 2] and p.table[0] == [3]
    p.lens[:2] = [4, 9]
    p.cache = list("abcdef")
    assert p.fork([1, 0, 1], [2, 3, 2]) == [1, 1, 0]
    assert p.table[2] == [0, 1, 4] and p.cache[4] == "c" and p.table[3] == [3] and p.refs == [2, 2, 1, 2, 1, 0]
    p.free([1, 0, 1])
    assert p.refs == [1, 1, 0, 1, 1, 0]
    assert p.compact() == 4 and p.table[2] == [0, 1, 2] and p.cache[2] == "c" and p.refs == [1, 1, 1, 1, 0, 0]


def test_weight_parts():
    """What the attention makes of a weight: fp16 into three parts of e5m2 (three significant bits, 2^4 and 2^8 times
    in the second and third), whose sum is the fp16 number for every one up to 2^15."""
    f16 = np.float16
    top = lambda x: ((x.view(np.uint16).astype(np.uint32) + 0x80) & 0xFF00).astype(np.uint16).view(f16)  # noqa: E731
    p = np.arange(f16(2.0 ** 15).view(np.uint16) + 1, dtype=np.uint16).view(f16)
    hi = top(p)
    rest = (p - hi) * f16(16)
    mid = top(rest)
    lo = top((rest - mid) * f16(16))
    assert hi.dtype == rest.dtype == mid.dtype == lo.dtype == f16
    assert np.isfinite([hi, mid, lo]).all()
    assert (hi.astype(np.float64) + mid.astype(np.float64) / 16 + lo.astype(np.float64) / 256 == p.astype(np.float64)).all()


def test_copies_in_flight_are_waited_for(tmp_path):
    """What a block whose waits have expired waits for before it returns: every copy begun for its units, whichever
    of them are still in flight, and nothing else (a wait for a phase that has not begun would run to its limit)."""
    import os
    import subprocess
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "draft_correction_slot_gb300", "csrc")
    (tmp_path / "model.cpp").write_text("""
#include <cstdio>
#include <initializer_list>
#include "ring.h"
// A ring of barriers: uses begun and completed on each; a use begins after the one before it on its barrier.
struct Ring {
  int slots, begun[32] = {}, waits = 0;
  bool bad = false, landed[32] = {};
  void wait(int i, int parity) {  // for the phase of that parity: the one in flight, not the one before or to come
    ++waits;
    if (i >= slots || begun[i] == 0 || ((begun[i] - 1) & 1) != parity) bad = true;
    else landed[i] = true;
  }
};
int main() {
  for (int units = 0; units < 200; ++units) {
    Ring q{2}, factors{dc::kAheadUnits};
    for (int u = 0; u < units; ++u) ++q.begun[u % 2], ++factors.begun[u % dc::kAheadUnits];
    dc::unit_copies(units, [&](int i, int p) { q.wait(i, p); }, [&](int i, int p) { factors.wait(i, p); });
    for (Ring *r : {&q, &factors}) {
      if (r->bad || r->waits > r->slots) return printf("%d units: a wait for nothing\\n", units), 1;
      for (int i = 0; i < r->slots; ++i)
        if (r->begun[i] > 0 && !r->landed[i]) return printf("%d units: a copy in flight\\n", units), 1;
    }
  }
}
""")
    exe = str(tmp_path / "model")
    subprocess.check_call(["g++", "-std=c++17", "-I", csrc, str(tmp_path / "model.cpp"), "-o", exe])
    assert subprocess.run([exe]).returncode == 0
    # the kernel's rings that copies complete on are these, and K's and V's
    src = open(os.path.join(csrc, "tree_attn_quant.cu")).read()
    tail = src[src.index("if (s_abort && warp == G::kPrepWarp"):src.index("tmem_dealloc(tmem, G::kTmem)")]
    for ring in ("q_full", "factors", "k_full", "v_full"):
        assert f"mbar_drain(smem_u32(&b.{ring}[i]), parity)" in tail


def test_lists_of_rows_have_one_axis(dc):
    import torch
    h = dc._PagesHandle()
    h.sizes = (8, 4, 4)
    x = torch.zeros(2, 2, dtype=torch.int32)
    for rows in (x, x[0, 0]):
        for call in (lambda: dc.dcoco_pages_free(h, rows, x, x, x, x), lambda: dc.dcoco_pages_reserve(h, rows, rows, x, x, x),
                     lambda: dc.dcoco_pages_fork(h, None, rows, rows, x, x, x, x)):
            with pytest.raises(ValueError, match="one axis"):
                call()
