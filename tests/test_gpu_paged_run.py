"""The paged operators together, as a serving loop uses them: plan, append, attention, commit, release over several
steps of a ragged batch, checked against the plain definitions and against the contiguous kernels; replayed from a
CUDA graph; on other streams and two at once; and after a stall."""
import numpy as np
import pytest
import torch

import gqa_head_folding_gb300 as g
from _paged import angles, paged_inputs, pages_of, ref_attn, ref_head_rows, ref_release, ref_tables, rows_tolerance
from gqa_head_folding_gb300.paged import PagedCache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def _clean():
    g.device_status()
    yield
    g.set_option(g.GQAQ_OPT_TEST_STALL, 0)
    g.set_option(g.GQAQ_OPT_WAIT_TIMEOUT_NS, 2_000_000_000)


class Loop:
    """A PagedCache of two layers beside a host model of its tables."""

    def __init__(self, batch, Hq, Hkv, D, S, dtype, pool, max_len, max_tokens, seed):
        self.c = PagedCache(2, batch, Hq, Hkv, D, pool, max_len, max_tokens, DEV, S, dtype)
        for p in (*self.c.k_pages, *self.c.v_pages):
            p.fill_(float("nan"))  # what no token wrote must not matter
        self.Hq, self.Hkv, self.D, self.S, self.dt, self.T = Hq, Hkv, D, S, dtype, max_tokens
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.cs = angles(max_len, D).to(DEV)
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=self.gen, device=DEV)).to(dtype) for _ in range(2))
        self.free, self.count = self.c.free_pages.cpu().numpy().astype(np.int64), pool
        self.table, self.len = self.c.block_table.cpu().numpy().astype(np.int64), np.zeros(batch, np.int64)
        self.pool = pool

    def inputs(self):
        x = torch.randn(self.T, self.Hq + 2 * self.Hkv, self.D, generator=self.gen, device=DEV).to(self.dt)
        return x.split([self.Hq, self.Hkv, self.Hkv], dim=1)

    def model_plan(self, new):
        kv, cu, pos, slots, count, table = ref_tables(self.len, new, self.free, self.count, self.table, self.T, self.S, self.pool)
        self.count, self.table = count, table
        return kv, cu, pos, slots

    def step(self, new):
        c = self.c
        kv, cu, pos, slots = self.model_plan(new)
        c.plan(ints(new))
        for name, got, ref in (("kv_len", c.kv_len, kv), ("cu_q", c.cu_q, cu), ("positions", c.positions, pos), ("slots", c.slots, slots),
                               ("table", c.block_table, self.table), ("count", c.free_count, [self.count])):
            assert np.array_equal(got.cpu().numpy(), np.asarray(ref)), name
        most = max(int(max(new)), 1)
        for layer in range(2):
            q, k, v = self.inputs()
            out = torch.full((self.T, self.Hq, self.D), 5.0, dtype=self.dt, device=DEV)
            qr = c.append(layer, q, k, v, self.wq, self.wk, 1e-6, self.cs, q_out=torch.zeros(self.T, self.Hq, self.D, dtype=self.dt, device=DEV))
            c.attend(layer, qr, most, out)
            live = torch.from_numpy(slots >= 0).to(DEV)
            at = torch.from_numpy(slots[slots >= 0]).to(DEV)
            for x, w, got in ((q, self.wq, qr[live]), (k, self.wk, c.k_pages[layer].transpose(1, 2).reshape(-1, self.Hkv, self.D)[at])):
                ref, size = ref_head_rows(x, w, 1e-6, self.cs, torch.from_numpy(pos).to(DEV), False)
                assert ((got.double() - ref[live]).abs() <= rows_tolerance(ref, size, self.dt)[live]).all()
            assert torch.equal(c.v_pages[layer].transpose(1, 2).reshape(-1, self.Hkv, self.D)[at], v[live])
            ref, tol = ref_attn(qr, c.k_pages[layer], c.v_pages[layer], c.block_table, cu.tolist(), kv.tolist(), c.scale,
                                torch.full_like(out, 5.0))
            assert ((out.double() - ref).abs() <= tol).all()
            self.against_contiguous(layer, qr, out, new, kv, cu)
        c.commit()
        self.len = np.maximum(self.len, kv)

    def against_contiguous(self, layer, q, out, new, kv, cu):
        """The framework's contiguous kernels over the same rows (fp16): both lie within the tolerance of the truth."""
        if self.dt != torch.float16:
            return
        for b, n in enumerate(new):
            if n == 0 or kv[b] == 0:
                continue
            pg = self.c.block_table[b, :pages_of(int(kv[b]), self.S)].long()
            kc, vc = (x[layer][pg].transpose(0, 1).reshape(1, self.Hkv, -1, self.D).contiguous() for x in (self.c.k_pages, self.c.v_pages))
            rows = q[cu[b]:cu[b + 1]].transpose(0, 1).contiguous()[None]  # [1,Hq,n,D]
            if n == 1:
                dense = g.gqa_decode_attn(rows[:, :, 0].contiguous(), kc, vc, ints([kv[b]]), self.c.scale)[:, :, None]
            else:
                dense = g.gqa_prefill_attn(rows, kc, vc, ints([kv[b] - n]), self.c.scale)
            err = (dense[0].transpose(0, 1).double() - out[cu[b]:cu[b + 1]].double()).abs()
            assert err.max() <= 4e-3 and err.mean() <= 4e-4  # twice the contiguous kernels' own tolerance

    def release(self, keep):
        self.free, self.count = ref_release(self.len, keep, self.free, self.count, self.table, self.S)
        self.c.release(ints(keep))
        self.len = np.asarray(keep, np.int64)
        assert np.array_equal(self.c.free_pages.cpu().numpy()[:self.count], self.free[:self.count])
        assert self.c.free_count.item() == self.count and np.array_equal(self.c.cache_len.cpu().numpy(), self.len)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hq, Hkv, D, S", [(8, 2, 64, 16), (4, 4, 128, 8), (8, 1, 128, 64)])
def test_serving_loop(dtype, Hq, Hkv, D, S):
    L = Loop(5, Hq, Hkv, D, S, dtype, 1400 // S + 6, 400, 420, seed=D + S)
    L.step([150, 3, 0, 77, 1])           # prompts
    L.step([1, 1, 260, 1, 1])            # a prompt among decoding requests
    for _ in range(3):
        L.step([1, 1, 1, 1, 1])
    L.step([5, 5, 0, 5, 5])              # drafted tokens
    L.release(np.array([L.len[0] - 3, L.len[1], L.len[2], L.len[3] - 5, L.len[4] - 1]))  # rejected tails
    L.release(np.array([0, L.len[1], 0, L.len[3], L.len[4]]))                           # two requests end
    L.step([40, 1, 200, 1, 1])           # others take their places
    L.step([1, 0, 1, 1, 0])
    assert g.device_status() == 0


def test_serving_loop_out_of_pages():
    L = Loop(3, 4, 2, 64, 16, torch.float16, 12, 192, 200, seed=9)
    L.step([100, 60, 20])                # 7 + 4 of 12 pages; the third needs two
    assert g.device_status() == g.GQAQ_DEV_NO_PAGES and L.len.tolist() == [100, 60, 0]
    L.step([1, 1, 10])
    assert g.device_status() == 0 and L.len.tolist() == [101, 61, 10]
    L.step([20, 1, 1])                   # the first would need another page
    assert g.device_status() == g.GQAQ_DEV_NO_PAGES and L.len.tolist() == [101, 62, 11]
    L.release(np.array([101, 0, 11]))
    L.step([20, 30, 1])
    assert g.device_status() == 0 and L.len.tolist() == [121, 30, 12]


@pytest.mark.parametrize("most", [1, 40])
def test_step_captured_and_replayed(most):
    """One graph of a whole step, replayed with other lengths, equals eager steps bit for bit."""
    B, Hq, Hkv, D, S, T = 4, 8, 2, 64, 16, 4 * most + 3
    eager, graph = (PagedCache(1, B, Hq, Hkv, D, 80, 300, T, DEV, S) for _ in range(2))
    cs = angles(300, D).to(DEV)
    gen = torch.Generator(device=DEV).manual_seed(4)
    x = torch.zeros(T, Hq + 2 * Hkv, D, dtype=torch.float16, device=DEV)
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    new = torch.zeros(B, dtype=torch.int32, device=DEV)
    outs = {c: torch.zeros(T, Hq, D, dtype=torch.float16, device=DEV) for c in (eager, graph)}
    qs = {c: torch.zeros(T, Hq, D, dtype=torch.float16, device=DEV) for c in (eager, graph)}

    def step(c):
        c.plan(new)
        c.append(0, q, k, v, None, None, 1e-6, cs, q_out=qs[c])
        c.attend(0, qs[c], most, outs[c])
        c.commit()

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step(graph)  # no new tokens: loads the kernels
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            step(graph)
    for n in ([most, 1, 0, most], [1, 1, 1, 1], [0, most, 1, 1], [1, 0, most, 0]):
        x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
        new.copy_(ints(n))
        torch.cuda.synchronize()
        gr.replay()
        step(eager)
        torch.cuda.synchronize()
        assert torch.equal(outs[eager], outs[graph]) and torch.equal(eager.block_table, graph.block_table)
        assert torch.equal(eager.cache_len, graph.cache_len) and torch.equal(eager.free_count, graph.free_count)
    assert g.device_status() == 0


def test_two_calls_at_once_with_their_own_workspaces():
    """Overlapping calls on two streams, each with its workspace; and many in a row that share one."""
    cases = [([1] * 6, [3000, 100, 129, 2500, 1, 777]), ([70, 1, 200], [2000, 1500, 200])]
    streams = [torch.cuda.Stream() for _ in cases]
    work = []
    for i, (ql, kl) in enumerate(cases):
        q, kp, vp, table, cu, kv = paged_inputs(ql, kl, 8, 2, 128, 16, torch.float16, i, DEV)
        ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), 0.09, torch.zeros_like(q))
        ws = g.alloc_paged_workspace(g.paged_dims_of(q, kp, table), DEV)
        work.append((q, kp, vp, table, cu, kv, max(ql), ws, ref, tol))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (q, kp, vp, table, cu, kv, most, ws, _, _) in enumerate(work):
            with torch.cuda.stream(streams[i]):
                outs[i].append(g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.09, most, workspace=ws))
    torch.cuda.synchronize()
    for i, w in enumerate(work):
        for o in outs[i]:
            assert ((o.double() - w[8]).abs() <= w[9]).all()
            assert torch.equal(o, outs[i][0])  # the same split, the same sums
        assert int(w[7][:4096].count_nonzero()) == 0
    assert g.device_status() == 0


def test_inputs_written_on_the_same_side_stream():
    q, kp, vp, table, cu, kv = paged_inputs([1, 30], [500, 600], 4, 2, 64, 16, torch.bfloat16, 3, DEV)
    ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), 0.125, torch.zeros_like(q))
    big = torch.randn(8192, 8192, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q2 = torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(3):
            big = big @ big * 1e-4
        q2.copy_(q)
        out = g.gqa_paged_attn(q2, kp, vp, table, cu, kv, 0.125, 30)
    st.synchronize()
    assert ((out.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [150, 1, 40], [20, 20, 20]])
@pytest.mark.parametrize("ctas", [0, 3])
def test_stall_times_out_and_recovers(q_lens, ctas):
    """The loaders issue nothing: every wait runs out, the call reports it, and the workspace stays usable."""
    q, kp, vp, table, cu, kv = paged_inputs(q_lens, [900, 500, 700], 4, 2, 128, 16, torch.float16, 5, DEV)
    ws = g.alloc_paged_workspace(g.paged_dims_of(q, kp, table), DEV)
    g.set_option(g.GQAQ_OPT_MAX_CTAS, ctas)
    g.set_option(g.GQAQ_OPT_WAIT_TIMEOUT_NS, 2_000_000)
    g.set_option(g.GQAQ_OPT_TEST_STALL, 1)
    g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.09, max(q_lens), workspace=ws)
    torch.cuda.synchronize()
    assert g.device_status() & g.GQAQ_DEV_TIMEOUT
    assert int(ws[:4096].count_nonzero()) == 0  # arrivals balanced: counters back at zero
    g.set_option(g.GQAQ_OPT_TEST_STALL, 0)
    g.set_option(g.GQAQ_OPT_WAIT_TIMEOUT_NS, 2_000_000_000)
    out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.09, max(q_lens), workspace=ws)
    torch.cuda.synchronize()
    g.set_option(g.GQAQ_OPT_MAX_CTAS, 0)
    ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), 0.09, torch.zeros_like(q))
    assert ((out.double() - ref).abs() <= tol).all() and g.device_status() == 0
