"""A total_len below the truth leaves the workspace too small: the requests that find no room in it are left out and reported,
the others are computed, and nothing is written behind the workspace."""
import numpy as np
import pytest
import torch

import quantized_decode_gemv_block_gb300 as kq
from test_gpu_kv8 import dev, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    assert kq.device_errors() == 0


# (lengths, the requests that find room). Two kv heads of two query heads: segments of 256 positions, two rows a token.
#   tokens: 6 requests' rows of one segment, 12; 301 positions take 2 x 2, 2001 take 8 x 2 (4 to 20), 401 the next 4
#   windows of 20: 6 x 40 rows; 320 positions take 2 x 40, 1020 take 4 x 40 (to 240, all of them), 2020 the next 320
#   a prompt of 40: 5 x 64 rows; 5040 positions in 8 segments of 80 rows, more than there are
CASES = {
    "tokens": ([(300, 1), (2000, 1), (100, 1), (400, 1), (255, 1), (0, 0)], [0, 2, 4]),
    "windows": ([(300, 20), (1000, 20), (50, 3), (2000, 20), (10, 1), (0, 0)], [0, 1, 2, 4]),
    "prompt": ([(5000, 40), (20, 2), (30, 60), (100, 1), (10, 1)], [1, 2, 3, 4])}


@pytest.mark.parametrize("y", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", CASES)
def test_requests_without_room_are_left_out(name, y):
    P, D, n_q, n_kv = 16, 64, 4, 2
    lens, fit = CASES[name]
    cache, _, table, ctx, new, q = make(lens, P, D, n_q, n_kv, "bf16", 31)
    clean = run(cache, table, ctx, new, q, "f32" if y == torch.float32 else "bf16")
    assert kq.device_errors() == 0
    need = kq.attention_kv8_workspace_size(len(lens), 0, int(new.max()), n_q, n_kv, D)
    assert 0 < need < kq.attention_kv8_workspace_size(len(lens), int((ctx + new).sum()), int(new.max()), n_q, n_kv, D)
    memory = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full_like(clean, 3.0)
    kq.attention_kv8(q, cache, dev(table), dev(ctx), dev(new), int(new.max()), int((ctx + new).max()), total_len=0, out=out,
                     workspace=memory[:need])
    assert kq.device_errors() == 2
    assert (memory[need:] == 0xA5).all()
    cu = np.concatenate([[0], np.cumsum(new)])
    for r in range(len(lens)):
        rows = slice(int(cu[r]), int(cu[r + 1]))
        if r in fit:
            assert torch.equal(out[rows], clean[rows]), r
        else:
            assert (out[rows] == 3).all(), r
