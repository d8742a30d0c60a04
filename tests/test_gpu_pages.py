"""Block tables and slot maps (kq_pages_plan, kq_pages_release) against a host simulation: every value is a
whole number and has to be equal."""
import numpy as np
import pytest
import torch

import quantized_decode_gemv_block_gb300 as kq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def dev(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def plan_host(ctx, new, table, free, P, T):
    table, free = table.copy(), list(free)
    cu, pos, slot = [0], np.zeros(T, np.int32), np.full(T, -1, np.int32)
    for r, (c, n) in enumerate(zip(ctx, new)):
        for b in range(-(-c // P), -(-(c + n) // P)):
            table[r, b] = free.pop()
        for i in range(n):
            pos[cu[-1] + i] = c + i
            slot[cu[-1] + i] = table[r, (c + i) // P] * P + (c + i) % P
        cu.append(cu[-1] + n)
    return table, free, np.array(cu, np.int32), pos, slot


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("B,ctx_hi,new_hi,pad", [(1, 0, 1, 0), (1, 0, 300, 5), (7, 40, 1, 0), (257, 200, 3, 1), (300, 100, 40, 77),
                                                 (4096, 50, 4, 0)])
def test_plan(P, B, ctx_hi, new_hi, pad):
    rng = np.random.default_rng(B + P)
    ctx, new = rng.integers(0, ctx_hi + 1, B), rng.integers(0, new_hi + 1, B)
    if B == 1:
        new[:] = new_hi
    width = (ctx_hi + new_hi) // P + 2
    held = -(-ctx // P)
    pages = rng.permutation(int((-(-(ctx + new) // P)).sum()) + 9)
    table = np.full((B, width), -7, np.int32)
    at = 0
    for r in range(B):
        table[r, :held[r]] = pages[at:at + held[r]]
        at += held[r]
    free = pages[at:]
    T = int(new.sum()) + pad
    want = plan_host(ctx, new, table, free, P, T)
    td, fd = dev(table), dev(np.concatenate([free, [-3] * 4]))
    nf = dev([len(free)])
    for _ in range(2):  # the same inputs give the same outputs again
        p = kq.pages_plan(dev(ctx), dev(new), td, fd, nf, P, T)
        assert p.status.item() == 0
        assert np.array_equal(td.cpu(), want[0]) and p.n_free.item() == len(want[1])
        assert np.array_equal(p.cu.cpu(), want[2]) and np.array_equal(p.pos.cpu(), want[3]) and np.array_equal(p.slot.cpu(), want[4])


def test_empty_batches():
    p = kq.pages_plan(dev([]), dev([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda"), dev([1]), dev([1]), 16, 3)
    assert p.status.item() == 0 and p.cu.tolist() == [0] and p.slot.tolist() == [-1] * 3 and p.n_free.item() == 1
    p = kq.pages_plan(dev([5]), dev([0]), dev([[2]]), dev([]), dev([0]), 16, 0)
    assert p.status.item() == 0 and p.cu.tolist() == [0, 0] and p.n_free.item() == 0


@pytest.mark.parametrize("ctx,new,n_free,T,status", [
    ([0, 10], [16, 30], 2, 100, "PAGES_OUT_OF_PAGES"), ([0, 60], [5, 5], 9, 100, "PAGES_TABLE_FULL"),
    ([0, 1], [8, 9], 9, 16, "PAGES_TOKENS_FULL"), ([0, -1], [1, 1], 9, 100, "PAGES_BAD_ARG"), ([0, 0], [1, -1], 9, 100, "PAGES_BAD_ARG"),
    ([0, 0], [1, 1], 10, 100, "PAGES_BAD_ARG"), ([0, 0], [1, 1], -1, 100, "PAGES_BAD_ARG"),
    ([2 ** 31 - 1, 0], [2 ** 31 - 1, 1], 9, 100, "PAGES_TABLE_FULL")])
def test_refused_plans_change_nothing(ctx, new, n_free, T, status):
    table = np.full((2, 4), 3, np.int32)
    td, fd = dev(table), dev(range(9))
    p = kq.pages_plan(dev(ctx), dev(new), td, fd, dev([n_free]), 16, T)
    assert p.status.item() & getattr(kq, status)
    assert np.array_equal(td.cpu(), table) and p.n_free.item() == n_free
    assert p.cu.tolist() == [0, 0, 0] and (p.slot == -1).all() and (p.pos == 0).all()


def test_plan_and_release_over_many_steps():
    """A queue of requests that grow, end and are replaced: pages never belong to two requests."""
    rng = np.random.default_rng(3)
    B, P, width, pages = 19, 16, 12, 90
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, a, b = dev(rng.permutation(pages)), dev([pages]), dev([0])
    free_h, table_h = list(free.cpu().numpy()), table.cpu().numpy()
    length = np.zeros(B, np.int64)
    for _ in range(30):
        new = np.minimum(rng.integers(0, 20, B), width * P - length)
        while (-(-(length + new) // P)).sum() > pages:
            new[rng.integers(B)] = 0
        want = plan_host(length, new, table_h, free_h, P, 400)
        p = kq.pages_plan(dev(length), dev(new), table, free, a, P, 400)
        table_h, free_h = want[0], want[1]
        assert p.status.item() == 0 and np.array_equal(table.cpu(), table_h) and np.array_equal(p.slot.cpu(), want[4])
        length += new
        done = rng.random(B) < 0.25
        for r in range(B):
            if done[r]:
                n = -(-length[r] // P)
                free_h += list(table_h[r, :n])
                table_h[r, :n] = -1
        st = kq.pages_release(dev(length), torch.tensor(done, device="cuda"), table, free, p.n_free, b, P)
        assert st.item() == 0 and b.item() == len(free_h)
        assert np.array_equal(free.cpu()[:len(free_h)], free_h) and np.array_equal(table.cpu(), table_h)
        held = table_h[table_h >= 0]
        assert len(set(held) | set(free_h)) == pages == len(held) + len(free_h)
        length[done] = 0
        a, b = b, torch.empty_like(a)


def test_release_refuses_more_pages_than_the_list_holds():
    table, free = dev([[4, 5], [6, 7]]), dev([0, 1, 2])
    out = dev([0])
    st = kq.pages_release(dev([20, 5]), torch.tensor([True, False], device="cuda"), table, free, dev([2]), out, 16)
    assert st.item() == kq.PAGES_OUT_OF_PAGES and out.item() == 2 and table.tolist() == [[4, 5], [6, 7]] and free.tolist() == [0, 1, 2]
    st = kq.pages_release(dev([-1, 5]), torch.tensor([True, False], device="cuda"), table, free, dev([2]), out, 16)
    assert st.item() == kq.PAGES_BAD_ARG and table.tolist() == [[4, 5], [6, 7]]
