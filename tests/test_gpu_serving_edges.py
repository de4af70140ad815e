"""Edges of the serving calls on the GPU: page ids that are no pages."""
import numpy as np
import pytest
import torch

import two_tier_sparse_gb300 as dsa
from test_gpu_serving import i32, small_ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from two_tier_sparse_gb300 import build
    build.build()
    dsa.load()
    torch.cuda.set_device(cuda_device)


@pytest.mark.parametrize("max_new", [8, 20000])  # one CTA, several
@pytest.mark.parametrize("B,held", [(3, 3), (61, 37), (700, 9)])
def test_ids_outside_the_pool_do_not_enter_the_ring(B, held, max_new):
    """Requests end whose table rows hold ids that are no pages: the step is reported with such a
    request, the ring holds -1 for them, and who pops that is reported in turn."""
    rng = np.random.default_rng(B + max_new)
    n_pages = B * held + 5
    table = rng.permutation(n_pages)[:B * held].reshape(B, held).astype(np.int32)
    free = sorted(set(range(n_pages)) - set(table.ravel().tolist()))
    bad = rng.random((B, held)) < 0.2
    bad[0, 1] = True
    table[bad] = rng.choice([-1, -2 ** 31, n_pages, n_pages + 1, 2 ** 31 - 1], int(bad.sum()))
    table[0, 1] = n_pages
    head = n_pages - 3  # the free pages run over the ring's end
    ring = np.full(n_pages, -7, np.int32)
    ring[(head + np.arange(5)) % n_pages] = free
    pool = dsa.PagePool(i32(table), 64, i32(ring), torch.tensor([head, head + 5], device="cuda"))
    n = i32([held * 64] * B)
    plan, ws = dsa.StepPlan.empty(B, max_new, n_tokens=n), small_ws()
    ends = np.ones(B, bool)
    ends[2::5] = False  # these stay, and keep what they hold
    back = np.where(bad, -1, table)[ends].ravel().tolist()
    for new in (np.where(ends, -1, 0), np.zeros(B)):  # then a step in which nobody ends
        dsa.plan_step(dsa.config(), n, i32(new), pool, plan, ws)
        h, t = pool.ring_state.tolist()
        assert (h, t) == (head, head + 5 + len(back))
        r = pool.free_ring.cpu().numpy()
        assert [int(r[i % n_pages]) for i in range(h, t)] == free + back
        assert n.tolist() == np.where(ends, 0, held * 64).tolist()
        code, info = dsa.read_device_status(ws)
        if new.any():
            assert code == 6 and info >> 24 == 7
            b = info & 0xFFFFFF
            assert ends[b] and (bad[b] & (table[b] != -1)).any()
        else:
            assert code == 0


@pytest.mark.parametrize("bad", [-1, 8, 2 ** 31 - 1, -2 ** 31])
def test_a_ring_entry_outside_the_pool_gives_no_page(bad):
    pool = dsa.PagePool.empty(3, 64, 2, 8)
    pool.free_ring[1] = bad
    n, ws = i32([0, 0, 0]), small_ws()
    plan = dsa.StepPlan.empty(3, 300, n_tokens=n)
    dsa.plan_step(dsa.config(), n, i32([64, 65, 1]), pool, plan, ws)
    assert pool.table.tolist() == [[0, -1], [-1, 2], [3, -1]] and pool.ring_state.tolist() == [4, 8]
    slots = plan.latent_slots.tolist()
    assert slots[:64] == list(range(64)) and slots[64:128] == [-1] * 64
    assert slots[128:130] == [128, 192]
    code, info = dsa.read_device_status(ws)
    assert code == 6 and info == (7 << 24) + 1
    # its end: what it was given goes back, a page and none
    dsa.plan_step(dsa.config(), n, i32([0, -1, -1]), pool, plan, ws)
    assert pool.ring_state.tolist() == [4, 11]
    assert [int(pool.free_ring[i % 8]) for i in range(4, 11)] == [4, 5, 6, 7, -1, 2, 3]
    assert dsa.read_device_status(ws)[0] == 0
