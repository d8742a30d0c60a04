"""The paged decoding example where pages run out: the step is refused before anything changes."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import paged_decode
    return paged_decode


@pytest.mark.parametrize("logits", [False, True])
@pytest.mark.parametrize("pages,blocks", [(2, 16), (16, 2)], ids=["no free pages", "table full"])
def test_a_step_without_pages_changes_nothing(ex, logits, pages, blocks):
    import quantized_decode_gemv_block_gb300 as kq
    dec = ex.PagedDecoder(slots=2, n_pages=pages, max_blocks=blocks)
    first = dec.step({0: list(range(32))})
    state = (list(dec.lens), dec.length.clone(), dec.n_free.clone(), dec.free.clone(), dec.table.clone(),
             *(t.clone() for c in dec.caches for t in (c.k, c.v, c.k_scale, c.v_scale)))
    with pytest.raises(RuntimeError, match="refused"):
        dec.step({0: [first[0]]}, logits=logits)
    after = (list(dec.lens), dec.length, dec.n_free, dec.free, dec.table,
             *(t for c in dec.caches for t in (c.k, c.v, c.k_scale, c.v_scale)))
    assert state[0] == after[0] and all(torch.equal(a, b) for a, b in zip(state[1:], after[1:]))
    dec.release([0])
    assert dec.n_free.item() == pages and sorted(dec.free[:pages].tolist()) == list(range(pages))
    assert len(dec.step({1: [3, 4, 5]})) == 1 and kq.device_errors() == 0
