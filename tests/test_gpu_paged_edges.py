"""The paged serving calls at their edges: what they refuse or leave as it was, NaN and waits that run out, sizes at a limit, and
long contexts whose outputs show the loss of a single key."""
import numpy as np
import pytest
import torch

import gqa_head_folding_gb300 as g
from _paged import ref_release
from test_gpu_paged_run import Loop

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def _clean():
    g.device_status()
    yield
    g.set_option(g.GQAQ_OPT_MAX_CTAS, 0)
    g.set_option(g.GQAQ_OPT_WAIT_TIMEOUT_NS, 2_000_000_000)


# ---------------------------------------------------------------------------
# Lengths and pages of a PagedCache stay in step
# ---------------------------------------------------------------------------
def release_some(L, keep):
    """A release of which some may be refused: those requests keep their length and their pages."""
    keep = np.asarray(keep, np.int64)
    L.free, L.count = ref_release(L.len, keep, L.free, L.count, L.table, L.S)
    L.c.release(ints(keep))
    L.len = np.where((keep >= 0) & (keep <= L.len), keep, L.len)
    assert L.c.cache_len.tolist() == L.len.tolist() and L.c.free_count.item() == L.count
    assert np.array_equal(L.c.free_pages.cpu().numpy()[:L.count], L.free[:L.count])


def test_refused_release_keeps_the_length():
    """Request 0 gives a page back, request 1 takes it; then request 0 is released to the length it had before, and
    request 1 to a negative one. Both stay as they were, and the next steps write and read their own pages only."""
    L = Loop(3, 4, 2, 64, 16, torch.float16, 24, 160, 120, seed=1)
    L.step([40, 20, 33])
    release_some(L, [20, 20, 33])
    L.step([0, 15, 0])
    assert g.device_status() == 0
    release_some(L, [40, -3, 30])
    assert g.device_status() == g.GQAQ_DEV_BAD_LEN and L.len.tolist() == [20, 35, 30]
    L.step([30, 1, 1])
    L.step([1, 20, 2])
    assert g.device_status() == 0
    assert len(set(L.table[0, :4]) | set(L.table[1, :4]) | set(L.table[2, :3])) == 11  # no page has two owners


def test_release_of_a_request_that_the_plan_refused():
    """The host expects the length that the step would have given; the plan had no pages for it."""
    L = Loop(2, 4, 2, 64, 16, torch.bfloat16, 5, 96, 80, seed=2)
    L.step([30, 40])                 # 2 + 3 of 5 pages
    L.step([1, 20])                  # the second would need another page
    assert g.device_status() == g.GQAQ_DEV_NO_PAGES and L.len.tolist() == [31, 40]
    release_some(L, [31, 58])        # "all of its 60 tokens but the last two"
    assert g.device_status() == g.GQAQ_DEV_BAD_LEN and L.len.tolist() == [31, 40]
    release_some(L, [0, 40])
    L.step([0, 20])
    assert g.device_status() == 0 and L.len.tolist() == [0, 60]


def test_commit_after_a_release_brings_nothing_back():
    L = Loop(3, 4, 2, 64, 16, torch.float16, 24, 160, 120, seed=3)
    L.step([40, 20, 33])
    release_some(L, [0, 20, 17])
    L.c.commit()
    assert L.c.cache_len.tolist() == [0, 20, 17]
    L.step([35, 5, 5])
    assert g.device_status() == 0 and L.len.tolist() == [35, 25, 22]


def test_release_of_a_planned_step():
    """Before commit, release counts from the planned lengths: a step can be given up, or kept in part, and its pages go back."""
    L = Loop(3, 4, 2, 64, 16, torch.float16, 24, 160, 120, seed=4)
    L.step([40, 20, 33])
    count = L.count
    for keep in ([40, 20, 33], [45, 20, 60], [40, 20, 33]):
        new = [20, 0, 40] if L.len[2] == 33 else [0, 0, 0]
        kv = L.model_plan(new)[0]
        L.c.plan(ints(new))
        assert L.c.kv_len.tolist() == kv.tolist()
        L.len = kv
        release_some(L, keep)
        L.c.commit()
        assert L.c.cache_len.tolist() == keep
    assert L.count == count
    L.model_plan([20, 0, 40])
    L.c.plan(ints([20, 0, 40]))
    L.c.release(ints([61, 20, 33]))  # one too many: refused, its step stays planned; the other's is given up
    assert g.device_status() == g.GQAQ_DEV_BAD_LEN
    L.c.commit()
    assert L.c.cache_len.tolist() == [60, 20, 33]
