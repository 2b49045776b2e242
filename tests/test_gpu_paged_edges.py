"""The paged serving calls at their edges: what they refuse or leave as it was, NaN and waits that run out, sizes at a limit, and
long contexts whose outputs show the loss of a single key."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import gqa_head_folding_gb300 as g
from _paged import DTYPES, angles, counting_case, dominant_case, pages_of, paged_inputs, ref_attn, ref_release
from gqa_head_folding_gb300.paged import PagedCache
from test_gpu_paged import append_case
from test_gpu_paged_run import Loop

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def test_drafting_step_captured_with_its_release():
    """A step of drafted tokens and the release of the rejected ones in one graph, replayed with other lengths, one of them refused."""
    caches = [PagedCache(1, 3, 4, 2, 64, 30, 100, 20, DEV) for _ in range(2)]
    gen = torch.Generator(device=DEV).manual_seed(12)
    x = torch.zeros(15, 8, 64, dtype=torch.float16, device=DEV)
    q, k, v = x.split([4, 2, 2], dim=1)
    new, keep = (torch.zeros(3, dtype=torch.int32, device=DEV) for _ in range(2))
    outs = [torch.zeros(15, 4, 64, dtype=torch.float16, device=DEV) for _ in range(2)]
    q_out = torch.zeros_like(outs[0])

    def step(i):
        c = caches[i]
        c.plan(new, 15)
        c.attend(0, c.append(0, q, k, v, q_out=q_out), 5, outs[i])
        c.commit()
        c.release(keep)

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step(0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step(0)
    lens = [0, 0, 0]
    for n, k_ in (([5, 5, 5], [4, 5, 2]), ([5, 1, 5], [9, 3, 99]), ([0, 5, 5], [0, 8, -1]), ([5, 5, 5], [5, 13, 15])):
        x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
        new.copy_(ints(n))
        keep.copy_(ints(k_))
        torch.cuda.synchronize()
        g.device_status()
        graph.replay()
        torch.cuda.synchronize()
        step(1)
        torch.cuda.synchronize()
        lens = [w if 0 <= w <= a + b else a + b for a, b, w in zip(lens, n, k_)]
        assert g.device_status() == (g.GQAQ_DEV_BAD_LEN if 99 in k_ or -1 in k_ else 0)
        assert torch.equal(*outs) and caches[0].cache_len.tolist() == lens
        for name in ("cache_len", "kv_len", "block_table", "free_count", "free_pages"):
            assert torch.equal(*(getattr(c, name) for c in caches)), name


# ---------------------------------------------------------------------------
# NaN and infinity in live rows
# ---------------------------------------------------------------------------
def softmax_rows(q, kp, vp, table, cu, kv, scale):
    """The definition row by row in 64 bits, NaN and infinity included."""
    out = torch.zeros_like(q, dtype=torch.float64)
    S, G = kp.shape[2], q.shape[1] // kp.shape[1]
    for b in range(len(kv)):
        n, L = cu[b + 1] - cu[b], kv[b]
        pg = table[b, :pages_of(L, S)].long()
        k, v = (x[pg].double().transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:L] for x in (kp, vp))
        for i in range(n):
            seen = L - n + i + 1
            for h in range(q.shape[1]):
                s = k[:seen, h // G] @ q[cu[b] + i, h].double() * scale
                out[cu[b] + i, h] = torch.softmax(s, 0) @ v[:seen, h // G]
    return out


@pytest.mark.parametrize("what", ["a row of q", "a channel of q", "many keys", "an infinite key"])
@pytest.mark.parametrize("ctas", [0, 5])
@pytest.mark.parametrize("q_lens, kv_lens, G, D", [([1], [5000], 4, 128), ([1, 2], [300, 5000], 2, 64), ([40], [6000], 1, 128),
                                                   ([40, 9], [100, 3100], 2, 64), ([200], [6000], 1, 64), ([150, 1], [150, 900], 2, 128)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attn_nan_and_infinity_reach_the_rows_that_see_them(dtype, q_lens, kv_lens, G, D, ctas, what):
    """Whether one CTA holds an item or many share it, a row whose scores hold NaN (or +inf) is NaN, and no other is touched."""
    g.set_option(g.GQAQ_OPT_MAX_CTAS, ctas)
    q, kp, vp, table, cu, kv = paged_inputs(q_lens, kv_lens, G, 1, D, 16, DTYPES[dtype], 11, DEV)
    scale = D ** -0.5
    last = len(q_lens) - 1
    row = int(cu[last]) + q_lens[last] // 2
    q[row, 0, 9] = 1.0
    _, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), scale, torch.zeros_like(q))
    if what == "a row of q":
        q[row, 0] = float("nan")
    elif what == "a channel of q":
        q[row, G - 1, 7] = float("inf")
    elif what == "many keys":
        kp[table[last, :kv_lens[last] // 32].long()] = float("nan")  # the first half, whole pages
    else:
        kp[table[last, 3].long(), 0, 5, 9] = float("inf")
    ref = softmax_rows(q, kp, vp, table, cu.tolist(), kv.tolist(), scale)
    ws = g.alloc_paged_workspace(g.paged_dims_of(q, kp, table), DEV)
    out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, scale, max(q_lens), workspace=ws)
    torch.cuda.synchronize()
    assert g.device_status() == 0 and int(ws[:4096].count_nonzero()) == 0
    assert ref.isnan().any() and torch.equal(out.isnan(), ref.isnan())
    fine = ~ref.isnan()
    # a key whose score is -inf takes part in no finite row: the others then weigh a little more than the tolerance counts with
    assert ((out.double() - ref).abs() <= 2 * tol)[fine].all()


# ---------------------------------------------------------------------------
# Rows that are no token of the item's request
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("q_lens, kv_lens, G", [([9, 30], [2000, 1500], 2), ([60], [1900], 4), ([150, 3], [800, 900], 1), ([3, 20], [900, 700], 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_does_not_depend_on_other_rows(q_lens, kv_lens, G, D):
    """Bit for bit the same whatever the rows behind the requests, and the rows of the other requests, hold."""
    q, kp, vp, table, cu, kv = paged_inputs(q_lens, kv_lens, 2 * G, 2, D, 16, torch.float16, 13, DEV, rows_behind=140)
    n = q_lens[0]
    outs = []
    for fill in (0.0, 1.0, 30.0, float("nan")):
        x = q.clone()
        x[n:] = x[n:] * fill if fill == fill else fill
        outs.append(g.gqa_paged_attn(x, kp, vp, table, cu, kv, 1.0, max(q_lens))[:n])
    torch.cuda.synchronize()
    assert torch.isfinite(outs[0]).all() and g.device_status() == 0
    for out in outs[1:]:
        assert torch.equal(out, outs[0])


# ---------------------------------------------------------------------------
# Waits that run out while copies and products are in flight
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("ns", [0, 500, 4000])
@pytest.mark.parametrize("q_lens, kv_lens", [([1, 1], [300, 3000]), ([40], [3000]), ([200, 3], [900, 500])])
def test_short_waits_leave_nothing_in_flight(q_lens, kv_lens, ns):
    """Every wait gives up after ns: the call ends, the counters are zero and the next call is right."""
    q, kp, vp, table, cu, kv = paged_inputs(q_lens, kv_lens, 4, 2, 128, 16, torch.float16, 6, DEV)
    ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), 0.09, torch.zeros_like(q))
    ws = g.alloc_paged_workspace(g.paged_dims_of(q, kp, table), DEV)
    g.set_option(g.GQAQ_OPT_WAIT_TIMEOUT_NS, ns)
    for _ in range(4):
        g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.09, max(q_lens), workspace=ws)
    torch.cuda.synchronize()
    assert g.device_status() in (0, g.GQAQ_DEV_TIMEOUT)  # a wait whose barrier was ready in time did not run out
    g.set_option(g.GQAQ_OPT_WAIT_TIMEOUT_NS, 2_000_000_000)
    assert int(ws[:4096].count_nonzero()) == 0
    out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.09, max(q_lens), workspace=ws)
    torch.cuda.synchronize()
    assert ((out.double() - ref).abs() <= tol).all() and g.device_status() == 0


@pytest.mark.parametrize("T", [3, 3000])
def test_short_waits_of_the_append(T):
    gen = torch.Generator(device=DEV).manual_seed(8)
    q, k, v = (torch.randn(T, h, 128, generator=gen, device=DEV).half() for h in (8, 2, 2))
    kp, vp = (torch.zeros(pages_of(T, 16), 2, 16, 128, dtype=torch.float16, device=DEV) for _ in range(2))
    pos = slots = torch.arange(T, dtype=torch.int32, device=DEV)
    g.set_option(g.GQAQ_OPT_WAIT_TIMEOUT_NS, 0)
    for _ in range(4):
        g.paged_norm_rope_append(q, k, v, pos, slots, kp, vp)
    torch.cuda.synchronize()
    assert g.device_status() in (0, g.GQAQ_DEV_TIMEOUT)
    g.set_option(g.GQAQ_OPT_WAIT_TIMEOUT_NS, 2_000_000_000)
    out = g.paged_norm_rope_append(q, k, v, pos, slots, kp, vp)
    torch.cuda.synchronize()
    rows = lambda p: p.transpose(1, 2).reshape(-1, 2, 128)[:T]  # noqa: E731
    assert torch.equal(out, q) and torch.equal(rows(kp), k) and torch.equal(rows(vp), v) and g.device_status() == 0


# ---------------------------------------------------------------------------
# Batches whose sums need more shared memory than a kernel has without asking
# ---------------------------------------------------------------------------
CHILD = """
import sys, torch
import gqa_head_folding_gb300 as g
call, B = sys.argv[1], int(sys.argv[2])
full = lambda n, v: torch.full((n,), v, dtype=torch.int32, device="cuda:0")
pages = torch.arange(B, dtype=torch.int32, device="cuda:0")
if call == "plan":
    kv, cu, pos, slots, count = g.paged_build_tables(full(B, 0), full(B, 1), pages, full(1, B), full(B, -1)[:, None], B, 8)
    assert int(kv.sum()) == B and int(cu[-1]) == B and count.item() == 0 and torch.equal(slots, 8 * pages.flip(0))
else:
    free = full(B, -1)
    count = g.paged_release_pages(full(B, 1), full(B, 0), pages[:, None].contiguous(), free, full(1, 0), 8)
    assert count.item() == B and torch.equal(free, pages)
assert g.device_status() == 0
"""


@pytest.mark.parametrize("call, B", [("plan", 4063), ("plan", 4064), ("plan", 4095), ("plan", 4096), ("release", 6112), ("release", 6143),
                                     ("release", 6144)])
def test_batches_in_a_process_of_their_own(call, B):
    """The first call of a process, where no larger batch has asked for the room before."""
    r = subprocess.run([sys.executable, "-c", CHILD, call, str(B)], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0, r.stderr[-2000:]


def test_plans_of_two_threads():
    """Two host threads plan batches of unlike size on streams of their own."""
    wrong = []

    def work(B):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                zero, one = torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
                pages = torch.arange(B, dtype=torch.int32, device=DEV)
                count, table = torch.full((1,), B, dtype=torch.int32, device=DEV), torch.zeros(B, 1, dtype=torch.int32, device=DEV)
                for _ in range(400):
                    slots = g.paged_build_tables(zero, one, pages, count, table, B, 8)[3]
                torch.cuda.current_stream().synchronize()
                if not torch.equal(slots, 8 * pages.flip(0)):
                    wrong.append(B)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(B,)) for B in (8192, 4200, 5000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and g.device_status() == 0


def test_first_calls_of_many_threads():
    """The first append and attention of a process, from eight host threads at once."""
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300, env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0, r.stderr[-2000:]


FIRST = """
import threading, torch
import gqa_head_folding_gb300 as g
wrong, gate = [], threading.Barrier(8)
def work(i):
    try:
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            n = 1 if i % 2 else 40
            q, k, v = (torch.ones(n, h, 64, dtype=torch.float16, device="cuda:0") for h in (4, 2, 2))
            kp, vp = (torch.zeros(4, 2, 16, 64, dtype=torch.float16, device="cuda:0") for _ in range(2))
            at = torch.arange(n, dtype=torch.int32, device="cuda:0")
            table = torch.arange(3, dtype=torch.int32, device="cuda:0")[None]
            cu, kv = torch.tensor([0, n], dtype=torch.int32, device="cuda:0"), torch.tensor([n], dtype=torch.int32, device="cuda:0")
            torch.cuda.current_stream().synchronize()
            gate.wait()
            q = g.paged_norm_rope_append(q, k, v, at, at, kp, vp)
            out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.125, n)
            torch.cuda.current_stream().synchronize()
            if not bool((out == 1).all()):
                wrong.append(i)
    except Exception as e:
        wrong.append(e)
threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not wrong and g.device_status() == 0, wrong
"""


@pytest.mark.parametrize("Hq, Hkv", [(4096, 512), (1, 1), (30000, 30000)])
def test_append_many_heads(Hq, Hkv):
    append_case(2, Hq, Hkv, 64, 8, "f16", 64, False, True, True, seed=Hq)


# ---------------------------------------------------------------------------
# Bad pages
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("in_place", [True, False])
def test_release_reports_bad_pages(in_place):
    table = ints([[5, -1, 4], [6, 2, 9], [2 ** 31 - 1, -2 ** 31, 0]])
    free, count = ints([3] + [-9] * 5), ints([1])
    out = g.paged_release_pages(ints([32, 32, 33]), ints([0, 3, 17]), table, free, count, 16, free_count_out=count if in_place else None)
    assert free.tolist() == [3, 5, -1, 2, 0, -9] and out.item() == 5 and g.device_status() == g.GQAQ_DEV_BAD_PAGE
    free, count = ints([3] + [-9] * 5), ints([1])
    g.paged_release_pages(ints([32, 32, 33]), ints([16, 16, 33]), table, free, count, 16)
    assert free.tolist() == [3, -1, 2, -9, -9, -9] and g.device_status() == g.GQAQ_DEV_BAD_PAGE
    g.paged_release_pages(ints([16, 32, 33]), ints([0, 16, 33]), table, free, count, 16)  # bad entries that are not released
    assert free.tolist() == [3, 5, 2, -9, -9, -9] and g.device_status() == 0


# ---------------------------------------------------------------------------
# A request's most tokens, where they end inside a page
# ---------------------------------------------------------------------------
def test_plan_refuses_tokens_past_max_len():
    args = dict(free_pages=ints([0, 1, 2, 3]), free_count=ints([4]), max_tokens=12, page_size=16)
    for most, kv in ((20, [0, 20, 3]), (21, [21, 20, 3]), (0, [21, 20, 3]), (1000, [21, 20, 3])):
        out = g.paged_build_tables(ints([15, 19, 0]), ints([6, 1, 3]), block_table=ints([[3, 0], [3, 2], [0, 0]]), max_len=most, **args)
        assert out[0].tolist() == kv and out[1].tolist() == [0, 6, 7, 10]  # a refused request's rows are counted
        assert g.device_status() == (g.GQAQ_DEV_BAD_LEN if kv[0] == 0 else 0)
    with pytest.raises(g.GqaqError):
        g.paged_build_tables(ints([0]), ints([1]), block_table=ints([[0, 0]]), max_len=-1, **args)


@pytest.mark.parametrize("max_len", [100, 128, 7])
def test_cache_ends_requests_at_max_len(max_len):
    """Pages of 64 tokens hold more than max_len; the table of angles does not reach further."""
    L = Loop(2, 4, 2, 64, 64, torch.float16, 8, max_len, 2 * max_len + 2, seed=5)
    L.c.plan(ints([max_len + 1, 5]))
    assert L.c.kv_len.tolist() == [0, 5] and g.device_status() == g.GQAQ_DEV_BAD_LEN
    assert L.c.slots[:max_len + 1].max() == -1
    L.c.release(ints([0, 0]))
    L.free, L.count = L.c.free_pages.cpu().numpy().astype(np.int64), L.c.free_count.item()
    L.table = L.c.block_table.cpu().numpy().astype(np.int64)
    assert L.count == 8
    L.step([max_len - 1, 3])
    L.step([1, 4])
    assert g.device_status() == 0 and L.len.tolist() == [max_len, 7]
    L.c.plan(ints([1, 0]))
    assert L.c.kv_len.tolist() == [0, 7] and g.device_status() == g.GQAQ_DEV_BAD_LEN
    L.c.commit()
    assert L.c.cache_len.tolist() == [max_len, 7]


# ---------------------------------------------------------------------------
# Steps of fewer rows than the object's most
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_steps_of_few_rows(dtype):
    """The same steps through projections of max_tokens rows and of the step's own rows."""
    wide, tight = (PagedCache(1, 3, 8, 2, 64, 40, 200, 150, DEV, 16, dtype) for _ in range(2))
    gen = torch.Generator(device=DEV).manual_seed(9)
    cs = angles(200, 64).to(DEV)
    for n in ([60, 3, 20], [1, 1, 1], [0, 1, 0], [4, 4, 4], [1, 0, 30]):
        x = torch.randn(150, 12, 64, generator=gen, device=DEV).to(dtype)
        rows, outs = sum(n), []
        for c, t in ((wide, None), (tight, rows)):
            q, k, v = x[:t].split([8, 2, 2], dim=1)
            c.plan(ints(n), t)
            out = c.attend(0, c.append(0, q, k, v, cos_sin=cs), max(n))
            c.commit()
            outs.append(out[:rows])
        assert outs[1].shape[0] == rows and torch.equal(*outs) and torch.equal(wide.slots[:rows], tight.slots[:rows])
        for a, b in ((wide.cache_len, tight.cache_len), (wide.block_table, tight.block_table), (wide.free_count, tight.free_count)):
            assert torch.equal(a, b)
    assert g.device_status() == 0


def test_steps_of_few_rows_refusals():
    c = PagedCache(1, 2, 4, 2, 64, 10, 64, 30, DEV)
    q, k, v = (torch.zeros(30, h, 64, dtype=torch.float16, device=DEV) for h in (4, 2, 2))
    for rows in (0, -1, 31):
        with pytest.raises(ValueError):
            c.plan(ints([1, 1]), rows)
    c.plan(ints([3, 9]), 8)          # 12 tokens in 8 rows
    assert g.device_status() == g.GQAQ_DEV_BAD_POS and c.kv_len.tolist() == [3, 0]
    for n in (7, 9, 30):             # rows behind the plan's hold what an earlier step left
        with pytest.raises(ValueError):
            c.append(0, q[:n], k[:n], v[:n])
    c.append(0, q[:8], k[:8], v[:8])
    with pytest.raises(ValueError):
        c.attend(0, q, 3)
    c.attend(0, q[:8], 3)            # the refused request's five rows are above the bound
    c.commit()
    assert g.device_status() == g.GQAQ_DEV_BAD_LEN and c.cache_len.tolist() == [3, 0]


# ---------------------------------------------------------------------------
# Workspace and arguments
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128])
def test_only_the_counters_of_a_workspace_need_zeros(D):
    dims = g.make_paged_dims(1, 8, 2, D, 16, 1, 1, 1)
    n = g.paged_workspace_bytes(dims)
    torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # what the allocator hands out next has been used
    ws = g.alloc_paged_workspace(dims, DEV)
    assert ws.numel() == n and int(ws[:4096].count_nonzero()) == 0
    ws[4096:] = 255  # NaN as floats
    for q_lens, kv_lens in (([1, 1], [300, 3000]), ([40], [6000]), ([200, 3], [5900, 500])):
        q, kp, vp, table, cu, kv = paged_inputs(q_lens, kv_lens, 4, 2, D, 16, torch.float16, 6, DEV)
        ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), 0.09, torch.zeros_like(q))
        for w in (ws, None):
            out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.09, max(q_lens), workspace=w)
            assert ((out.double() - ref).abs() <= tol).all()
    assert g.device_status() == 0


def test_numbers_past_32_bits_are_refused():
    q, kp, vp, table, cu, kv = paged_inputs([2], [40], 4, 2, 64, 16, torch.float16, 1, DEV)
    for most in (2 ** 31, 2 ** 32 + 2, -2 ** 40):
        with pytest.raises(ValueError, match="max_q_len"):
            g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.1, most)
    with pytest.raises(ValueError):
        g.paged_build_tables(kv, kv, ints([0]), ints([0]), table, 4, page_size=2 ** 32 + 16)
    with pytest.raises(ValueError):
        g.make_paged_dims(1, 4, 2, 64, 16, 2 ** 32 + 4, 3, 2)


# ---------------------------------------------------------------------------
# Long contexts: outputs that show the loss of a key, a page, a tile or a part
# ---------------------------------------------------------------------------
LONG = [([1], [39990], 2), ([1, 1, 1], [39990, 17, 20001], 4), ([4], [39990], 2), ([5], [30001], 2), ([70], [39990], 1), ([300, 1], [20000, 9001], 1)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("S, D", [(16, 64), (128, 128)])
@pytest.mark.parametrize("q_lens, kv_lens, G", LONG)
def test_attn_long_contexts_count_their_keys(q_lens, kv_lens, G, S, D, dtype):
    q, kp, vp, table, cu, kv, ref, tol = counting_case(q_lens, kv_lens, 8 * G, 8, D, S, DTYPES[dtype], 3, DEV)
    out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, D ** -0.5, max(q_lens))
    torch.cuda.synchronize()
    assert g.device_status() == 0
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), f"max err {err.max():.3e}, {(err / tol.clamp(min=1e-30)).max():.2f} of its bound"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("S, D", [(16, 64), (64, 128)])
@pytest.mark.parametrize("q_lens, kv_lens, G", LONG)
def test_attn_long_contexts_find_their_keys(q_lens, kv_lens, G, S, D, dtype):
    for seed in range(3):
        q, kp, vp, table, cu, kv, scale, ref, tol = dominant_case(q_lens, kv_lens, 8 * G, 8, D, S, DTYPES[dtype], seed, DEV)
        out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, scale, max(q_lens))
        torch.cuda.synchronize()
        assert g.device_status() == 0
        err = (out.double() - ref).abs()
        assert (err <= tol).all(), f"max err {err.max():.3e}, {(err / tol.clamp(min=1e-30)).max():.2f} of its bound"
