"""The example runs, and its cache after several committed trees gives the
logits that the same text gives as one causal block on an empty cache."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_tree_step_example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import tree_step as ex
    import draft_correction_slot_gb300 as dc
    r = ex.run(n=3, steps=4, verbose=False)
    assert all(x > 0 for x in r["losses"])
    for i in range(3):
        text = r["text"][i]
        assert all(0 <= t < ex.V for t in text)
        last = r["anchor"][i:i + 1, None]
        one, _, _ = r["target"].forward(r["verifier"], last, None, r["cache"], r["table"][i:i + 1],
                                        r["ctx_len"][i:i + 1])
        # the whole text at once, nothing in the cache
        v = dc.TreeVerifier(ex.HEADS, ex.KV_HEADS, ex.HEAD, ex.PAGE, ex.PAGES, max_batch=1, max_tree=256)
        whole, _, _ = r["target"].forward(v, torch.tensor([text], dtype=torch.int32, device="cuda"), None, r["cache"],
                                          r["table"][i:i + 1], torch.zeros(1, dtype=torch.int32, device="cuda"))
        a, b = one[0, 0].float(), whole[0, -1].float()
        # two bf16 layers: each rounding (2^-9 rms of the value) of states, products and weights, some twenty in a row
        assert (a - b).norm() <= 20 * 2 ** -9 * b.norm()
    r["verifier"].close()
