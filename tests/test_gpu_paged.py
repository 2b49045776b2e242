"""GPU parity of the paged serving operators (block tables and slots, page release, norm + rotation + append, paged
attention) against their plain definitions in 64 bits (_paged.py), at the sizes, masks and bad inputs where they can
go wrong."""
import numpy as np
import pytest
import torch

import gqa_head_folding_gb300 as g
from _paged import (DTYPES, angles, pages_of, paged_inputs, ref_attn, ref_head_rows, ref_release, ref_tables, rows_tolerance)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def _clean():
    g.device_status()
    yield
    g.set_option(g.GQAQ_OPT_MAX_CTAS, 0)
    g.set_option(g.GQAQ_OPT_TEST_STALL, 0)
    g.set_option(g.GQAQ_OPT_WAIT_TIMEOUT_NS, 2_000_000_000)


# ---------------------------------------------------------------------------
# Tables
# ---------------------------------------------------------------------------
def plan(cache_len, new_len, S, T, spare, width=None, seed=0, in_place=False):
    """Runs the plan against the reference; spare: free pages beyond (or short of) what is needed."""
    B = len(cache_len)
    rng = np.random.default_rng(seed)
    width = max(pages_of(max(c, 0) + max(n, 0), S) for c, n in zip(cache_len, new_len)) + 1 if width is None else width
    held = [min(pages_of(max(c, 0), S), width) for c in cache_len]  # a row of the table holds no more
    need = sum(min(pages_of(max(c, 0) + max(n, 0), S), width) - h for c, n, h in zip(cache_len, new_len, held))
    count = max(need + spare, 0)
    pool = sum(held) + count + 5
    order = rng.permutation(pool)
    table = np.full((B, width), -7, np.int64)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    free = np.full(pool, -3, np.int64)
    free[:count] = order[at:at + count]
    ref = ref_tables(cache_len, new_len, free, count, table, T, S, pool)
    t, c = ints(table), ints([count])
    got = g.paged_build_tables(ints(cache_len), ints(new_len), ints(free), c, t, T, S, free_count_out=c if in_place else None)
    torch.cuda.synchronize()
    for name, x, y in zip(("kv_len", "cu_q", "positions", "slots", "count", "table"), (*got, t), (*ref[:4], np.array([ref[4]]), ref[5])):
        assert np.array_equal(x.cpu().numpy(), y), name
    return g.device_status()


@pytest.mark.parametrize("S", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("B", [1, 3, 32, 33, 257])
def test_tables_ragged(B, S):
    rng = np.random.default_rng(B * S)
    c, n = rng.integers(0, 4 * S, B), rng.integers(0, 3 * S, B)
    n[rng.random(B) < 0.3] = 1
    assert plan(c, n, S, int(n.sum()) + 7, 2, seed=B) == 0


@pytest.mark.parametrize("c, n", [([0], [0]), ([0], [1]), ([16], [1]), ([15], [1]), ([0, 0, 0], [0, 5, 0]), ([31], [18]), ([0], [4000]),
                                  ([7, 16, 32], [0, 0, 0])])
def test_tables_edges(c, n):
    assert plan(c, n, 16, max(sum(n), 1), 0, in_place=True) == 0


def test_tables_many_rows_and_requests():
    rng = np.random.default_rng(5)
    c, n = rng.integers(0, 300, 300), rng.integers(0, 200, 300)
    assert plan(c, n, 16, int(n.sum()) + 1000, 40, in_place=True) == 0  # eight CTAs
    assert plan(rng.integers(0, 40, 8192), rng.integers(0, 3, 8192), 8, 20000, 1) == 0  # the largest batch


@pytest.mark.parametrize("spare", [-1, -3, -20, -10 ** 6])
def test_tables_pool_runs_dry(spare):
    c, n = [5, 16, 30, 31, 64, 10], [12, 1, 2, 40, 0, 90]
    assert plan(c, n, 16, 200, spare, in_place=True) == g.GQAQ_DEV_NO_PAGES


def test_tables_refuse_lengths_and_rows():
    assert plan([5, -1, 20, 3], [2, 3, 1, 1], 16, 10, 1) == g.GQAQ_DEV_BAD_LEN
    assert plan([5, 9, 20, 3], [2, -3, 1, 1], 16, 10, 1) == g.GQAQ_DEV_BAD_LEN
    assert plan([5, 40, 20], [2, 30, 1], 16, 40, 1, width=4) == g.GQAQ_DEV_BAD_LEN  # 70 tokens in 4 pages
    assert plan([5, 9, 20, 3], [2, 9, 1, 1], 16, 10, 1) == g.GQAQ_DEV_BAD_POS       # 13 rows in 10
    assert plan([2 ** 31 - 1, 5], [2 ** 31 - 1, 1], 16, 10, 1, width=3) & g.GQAQ_DEV_BAD_LEN


def test_tables_bad_pages_and_counts():
    free, table = ints([4, 99, -2, 3]), ints([[50, -1, -1], [1, -1, -1]])
    kv, cu, pos, slots, count = g.paged_build_tables(ints([3, 16]), ints([14, 17]), free, ints([4]), table, 31, 16)
    assert g.device_status() == g.GQAQ_DEV_BAD_PAGE
    # request 0: page 50 of 4, then page 3; request 1: pages -2 and 99
    assert slots.tolist() == [-1] * 13 + [48] + [-1] * 17 and count.item() == 1 and kv.tolist() == [17, 33]
    assert g.paged_build_tables(ints([0]), ints([16]), ints([0, 1]), ints([7]), ints([[-1]]), 16, 16)[4].item() == 1
    assert g.device_status() == g.GQAQ_DEV_BAD_LEN


@pytest.mark.parametrize("B, S, hi", [(1, 16, 40), (32, 16, 300), (500, 8, 3000), (8192, 128, 600)])
@pytest.mark.parametrize("in_place", [True, False])
def test_release(B, S, hi, in_place):
    rng = np.random.default_rng(B + S)
    kv = rng.integers(0, hi, B)
    keep = np.where(rng.random(B) < 0.4, kv, np.where(rng.random(B) < 0.5, 0, rng.integers(0, kv + 1)))
    width = pages_of(hi, S)
    held = [pages_of(int(n), S) for n in kv]
    pool = sum(held) + 9
    order = rng.permutation(pool)
    table = np.full((B, width), -1, np.int64)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    free = np.full(pool, -3, np.int64)
    free[:pool - at] = order[at:]
    ref, n = ref_release(kv, keep, free, pool - at, table, S)
    f, c = ints(free), ints([pool - at])
    out = g.paged_release_pages(ints(kv), ints(keep), ints(table), f, c, S, free_count_out=c if in_place else None)
    torch.cuda.synchronize()
    assert np.array_equal(f.cpu().numpy(), ref) and out.item() == n and g.device_status() == 0


def test_release_refusals():
    table = ints([[5, 6], [7, 8], [9, 10], [1, 2]])
    f = ints([3, -1, -1, -1, -1, -1])
    out = g.paged_release_pages(ints([20, 33, 20, 32]), ints([21, 0, -1, 5]), table, f, ints([1]), 16)
    assert f.tolist() == [3, 2, -1, -1, -1, -1] and out.item() == 2 and g.device_status() == g.GQAQ_DEV_BAD_LEN
    f = ints([3, 0, -1])  # two pages too many
    out = g.paged_release_pages(ints([20, 16, 0, 20]), ints([16, 0, 0, 16]), table, f, ints([2]), 16)
    assert f.tolist() == [3, 0, 6] and out.item() == 3 and g.device_status() == g.GQAQ_DEV_BAD_LEN


# ---------------------------------------------------------------------------
# Norm, rotation, append
# ---------------------------------------------------------------------------
def append_case(T, Hq, Hkv, D, S, dtype, rope, inter, norm, fused, seed, pad=0, most=5000, in_place=False, spread=1.0):
    dt = DTYPES[dtype]
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = T + pad
    x = (spread * torch.randn(n, Hq + 2 * Hkv, D, generator=gen, device=DEV)).to(dt)
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    wq = wk = None
    if norm in (True, "q"):
        wq = (1 + 0.3 * torch.randn(D, generator=gen, device=DEV)).to(dt)
    if norm in (True, "k"):
        wk = (1 + 0.3 * torch.randn(D, generator=gen, device=DEV)).to(dt)
    cs = angles(most, rope).to(DEV) if rope else None
    pos = torch.randint(0, most, (n,), generator=gen, device=DEV).to(torch.int32)
    pages = pages_of(T, S) + 2
    slots = torch.randperm(pages * S, generator=gen, device=DEV)[:n].to(torch.int32)
    slots = torch.cat([slots, slots.new_zeros(max(0, n - slots.numel()))])
    slots[T:] = -1
    kp, vp = (torch.randn(pages, Hkv, S, D, generator=gen, device=DEV).to(dt) for _ in range(2))
    (rq, szq), (rk, szk) = ref_head_rows(q, wq, 1e-5, cs, pos, inter), ref_head_rows(k, wk, 1e-5, cs, pos, inter)
    old_k, old_v, old_q, v0 = kp.clone(), vp.clone(), q.clone(), v.clone()
    q_out = q if in_place else torch.full((n, Hq, D), 7.0, dtype=dt, device=DEV)
    res = g.paged_norm_rope_append(q, k, v, pos, slots, kp, vp, q_weight=wq, k_weight=wk, eps=1e-5, cos_sin=cs, interleaved=inter,
                                   q_out=q_out)
    torch.cuda.synchronize()
    assert g.device_status() == 0 and res is q_out
    err = (q_out[:T].double() - rq[:T]).abs()
    assert (err <= rows_tolerance(rq, szq, dt)[:T]).all(), err.max()
    assert torch.equal(q_out[T:], old_q[T:] if in_place else torch.full_like(q_out[T:], 7.0))
    at = slots[:T].long()
    got_k, got_v = (p.transpose(1, 2).reshape(-1, Hkv, D)[at] for p in (kp, vp))
    err = (got_k.double() - rk[:T]).abs()
    assert (err <= rows_tolerance(rk, szk, dt)[:T]).all(), err.max()
    assert torch.equal(got_v, v0[:T])
    if not rope and wk is None:
        assert torch.equal(got_k, k[:T])  # nothing to compute: the row as it is
    for pool, old in ((kp, old_k), (vp, old_v)):  # every other row as it was
        rest = torch.ones(pages * S, dtype=torch.bool, device=DEV)
        rest[at] = False
        assert torch.equal(pool.transpose(1, 2).reshape(-1, Hkv, D)[rest], old.transpose(1, 2).reshape(-1, Hkv, D)[rest])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D, rope", [(64, 0), (64, 16), (64, 48), (64, 64), (128, 32), (128, 64), (128, 128), (128, 112)])
@pytest.mark.parametrize("inter", [False, True])
def test_append_rotations(dtype, D, rope, inter):
    append_case(9, 8, 2, D, 16, dtype, rope, inter, True, True, seed=D + rope, pad=2)


@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (2, 1), (3, 3), (8, 1), (32, 8), (32, 32), (40, 5), (71, 71)])
@pytest.mark.parametrize("D", [64, 128])
def test_append_heads(Hq, Hkv, D):
    append_case(5, Hq, Hkv, D, 8, "f16", 32, False, True, False, seed=Hq)


@pytest.mark.parametrize("T", [1, 2, 31, 200, 1500])
@pytest.mark.parametrize("norm", [True, False, "q", "k"])
def test_append_lengths_and_norms(T, norm):
    append_case(T, 8, 2, 128, 32, "bf16", 128, False, norm, T % 2 == 0, seed=T, pad=T % 3)


def test_append_in_place_and_sizes():
    append_case(33, 16, 4, 64, 16, "f16", 64, False, True, False, seed=1, in_place=True, pad=3)
    append_case(33, 16, 4, 128, 16, "bf16", 128, True, True, False, seed=2, in_place=True)
    append_case(20, 4, 4, 64, 16, "f16", 64, False, True, True, seed=3, spread=300.0)   # large activations
    append_case(20, 4, 4, 64, 16, "f16", 64, False, True, True, seed=4, spread=1e-4)    # near eps
    append_case(20, 4, 4, 64, 16, "bf16", 0, False, False, True, seed=5, spread=0.0)


def test_append_skips_bad_slots_and_positions():
    T, Hq, Hkv, D, S = 6, 4, 2, 64, 16
    gen = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn(T, h, D, generator=gen, device=DEV).half() for h in (Hq, Hkv, Hkv))
    kp, vp, q_out = torch.zeros(2, Hkv, S, D, device=DEV).half(), torch.zeros(2, Hkv, S, D, device=DEV).half(), torch.zeros_like(q)
    cs = angles(10, 64).to(DEV)
    pos, slots = ints([0, 9, 10, -1, 5, 2 ** 31 - 1]), ints([0, 32, 2, 3, 2 ** 31 - 1, -5])
    g.paged_norm_rope_append(q, k, v, pos, slots, kp, vp, cos_sin=cs, q_out=q_out)
    torch.cuda.synchronize()
    assert g.device_status() == g.GQAQ_DEV_BAD_PAGE | g.GQAQ_DEV_BAD_POS
    assert [bool(x.any()) for x in q_out] == [True] + [False] * 5
    assert kp.transpose(1, 2).reshape(-1, Hkv, D).any(-1).any(-1).nonzero().flatten().tolist() == [0]


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def attn_case(q_lens, kv_lens, G, Hkv, D, S, dtype, seed=0, max_q=None, scale=None, status=0, workspace=None, mess=None, **kw):
    q, kp, vp, table, cu, kv = paged_inputs(q_lens, kv_lens, G * Hkv, Hkv, D, S, DTYPES[dtype], seed, DEV, **kw)
    scale = D ** -0.5 if scale is None else scale
    if mess is not None:
        q, kp, vp, table, cu, kv = mess(q, kp, vp, table, cu, kv)
    out = torch.full_like(q, 3.0)
    most = max(max(q_lens), 1) if max_q is None else max_q
    ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), scale, out, most)
    g.gqa_paged_attn(q, kp, vp, table, cu, kv, scale, most, out=out, workspace=workspace)
    torch.cuda.synchronize()
    assert g.device_status() == status
    assert torch.isfinite(out).all()
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), f"max err {err.max():.3e}, {(err / tol.clamp(min=1e-30)).max():.2f} of its bound"
    return out


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_attn_single_tokens(dtype, D, G):
    attn_case([1, 1, 1, 1], [1, 300, 129, 1000], G, 2, D, 16, dtype, seed=G)


@pytest.mark.parametrize("S", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("q_lens, kv_lens", [([1, 1, 1], [127, 128, 257]), ([40, 1, 3], [40, 500, 131]), ([130], [1000])])
def test_attn_page_sizes(S, q_lens, kv_lens):
    attn_case(q_lens, kv_lens, 4, 2, 128, S, "bf16", seed=S)
    attn_case(q_lens, kv_lens, 2, 3, 64, S, "f16", seed=S + 1)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_attn_chunks(dtype, D, G):
    attn_case([70, 1, 33], [70, 200, 500], G, 2, D, 16, dtype, seed=D + G)


@pytest.mark.parametrize("n", [2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_attn_chunk_lengths(n):
    attn_case([n, 1], [n, 140], 1, 2, 64, 16, "f16", seed=n)           # a whole prompt
    attn_case([n, n], [n + 261, n + 1], 4, 1, 128, 16, "bf16", seed=n)


def test_attn_empty_and_short_requests():
    # no rows, no tokens, fewer tokens than rows
    attn_case([0, 1, 3, 0, 2], [50, 0, 2, 0, 300], 4, 2, 64, 16, "f16", seed=1)
    attn_case([0, 20, 40, 1], [50, 0, 25, 300], 8, 2, 128, 16, "bf16", seed=2)
    attn_case([200, 300], [0, 100], 2, 1, 64, 8, "f16", seed=3)
    attn_case([0, 0], [10, 10], 2, 1, 64, 8, "f16", seed=3, rows_behind=4)


def test_attn_leaves_rows_around_requests():
    out = attn_case([5, 0, 9], [100, 4, 9], 4, 2, 64, 16, "f16", seed=4, gap=3, rows_behind=11)
    assert (out[:3] == 3).all() and (out[17:] == 3).all()
    out = attn_case([1, 1], [100, 4], 2, 2, 128, 16, "bf16", seed=4, gap=2, rows_behind=5)
    assert (out[:2] == 3).all() and (out[4:] == 3).all()


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 4.0])
def test_attn_scales(scale):
    attn_case([1, 1], [300, 77], 4, 2, 64, 16, "f16", seed=5, scale=scale)
    attn_case([50, 3], [300, 77], 4, 2, 64, 16, "f16", seed=6, scale=scale)


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [40, 2, 1]])
def test_attn_bad_pages_read_as_zeros(q_lens):
    def mess(q, kp, vp, table, cu, kv):
        table[0, 1], table[1, 0], table[2, 3] = -1, kp.shape[0], 2 ** 31 - 1
        return q, kp, vp, table, cu, kv
    attn_case(q_lens, [100, 90, 61], 2, 2, 64, 16, "f16", seed=7, status=g.GQAQ_DEV_BAD_PAGE, mess=mess)


def test_attn_bad_lengths():
    attn_case([5, 1], [50, 60], 2, 2, 64, 16, "f16", seed=8, max_q=3, status=g.GQAQ_DEV_BAD_LEN)
    attn_case([50, 1], [50, 60], 2, 2, 64, 16, "f16", seed=8, max_q=33, status=g.GQAQ_DEV_BAD_LEN)
    for n in (1, 40):
        q, kp, vp, table, cu, kv = paged_inputs([n, n, n], [64, 64, 64], 4, 2, 64, 16, torch.float16, 9, DEV)
        kv[0], kv[1] = -5, 2 ** 31 - 1  # read as 0 and as 64
        out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.125, n)
        ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), [0, 64, 64], 0.125, torch.zeros_like(q))
        assert ((out.double() - ref).abs() <= tol).all() and g.device_status() == g.GQAQ_DEV_BAD_LEN
        cu[1], cu[2], cu[3] = 2 ** 31 - 1, -9, 3 * n + 7
        g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.125, n)
        assert g.device_status() & g.GQAQ_DEV_BAD_POS


@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 40])
@pytest.mark.parametrize("q_lens, kv_lens", [([1] * 5, [700, 1, 128, 1500, 129]), ([300, 1, 20], [900, 1500, 20]), ([3] * 3, [900, 64, 513])])
def test_attn_work_split(ctas, q_lens, kv_lens):
    g.set_option(g.GQAQ_OPT_MAX_CTAS, ctas)
    attn_case(q_lens, kv_lens, 2, 2, 64, 16, "f16", seed=ctas)
    attn_case(q_lens, kv_lens, 4, 1, 128, 32, "bf16", seed=ctas)


def test_attn_rising_scores_move_the_reference():
    """Scores that climb by a large step from tile to tile, then fall: every tile moves the running maximum."""
    for D, n in ((64, 1), (128, 1), (64, 40), (128, 200)):
        q, kp, vp, table, cu, kv = paged_inputs([n], [1100], 2, 1, D, 16, torch.float16, 10, DEV)
        ramp = torch.cat([torch.linspace(0, 40, 800, device=DEV), torch.linspace(40, -40, 300, device=DEV)])
        rows = torch.zeros(pages_of(1100, 16) * 16, device=DEV)
        rows[:1100] = ramp
        q[:] = 1.0
        kp[table[0].long(), 0] = rows.reshape(-1, 16, 1).expand(-1, 16, D).half() * 0.9
        out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, 1.0 / D ** 0.5, n)
        ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), 1.0 / D ** 0.5, torch.zeros_like(q))
        assert ((out.double() - ref).abs() <= tol).all() and g.device_status() == 0


def test_attn_long_context_and_wide_offsets():
    """A pool of more than 2^31 elements, its last pages in use; 40,000 tokens."""
    Hkv, S, D = 8, 128, 128
    pages = 17000  # 17000 * 8 * 128 * 128 = 2.2e9 elements a pool
    kp, vp = (torch.zeros(pages, Hkv, S, D, dtype=torch.float16, device=DEV) for _ in range(2))
    n = pages_of(40000, S)
    for pool in (kp, vp):
        pool[-n:] = torch.randn(n, Hkv, S, D, device=DEV).half()
    table = torch.arange(pages - n, pages, dtype=torch.int32, device=DEV).flip(0)[None].contiguous()
    for rows in (1, 70):
        q = torch.randn(rows, 16, D, device=DEV).half()
        cu, kv = ints([0, rows]), ints([39990])
        out = g.gqa_paged_attn(q, kp, vp, table, cu, kv, D ** -0.5, rows)
        ref, tol = ref_attn(q, kp, vp, table, [0, rows], [39990], D ** -0.5, torch.zeros_like(q))
        assert ((out.double() - ref).abs() <= tol).all() and g.device_status() == 0
    k = torch.randn(1, Hkv, D, device=DEV).half()
    slot = ints([(pages - 1) * S + 5])
    g.paged_norm_rope_append(torch.zeros(1, 8, D, device=DEV).half(), k, k, ints([0]), slot, kp, vp)
    assert torch.equal(kp[-1, :, 5], k[0]) and torch.equal(vp[-1, :, 5], k[0])


@pytest.mark.parametrize("B, n", [(1500, 1), (300, 5), (700, 2), (8192, 1)])
def test_attn_many_requests(B, n):
    rng = np.random.default_rng(B)
    kv = [int(x) for x in rng.integers(n, 60, B)]
    kv[7], kv[B - 1] = 1500, 700
    attn_case([n] * B, kv, 4, 1, 64, 8, "f16", seed=B)


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [40, 9, 1]])
def test_attn_requests_share_pages(q_lens):
    """A common prefix of ten pages: the three tables begin with the same entries."""
    def mess(q, kp, vp, table, cu, kv):
        table[1:, :10] = table[0, :10]
        return q, kp, vp, table, cu, kv
    attn_case(q_lens, [300, 170, 261], 4, 2, 128, 16, "bf16", seed=21, mess=mess)


@pytest.mark.parametrize("q_lens", [[1, 1], [300, 2], [40, 150]])
@pytest.mark.parametrize("pdl", [0, 1])
def test_attn_output_in_place_of_q(q_lens, pdl):
    g.set_option(g.GQAQ_OPT_PDL, pdl)
    try:
        q, kp, vp, table, cu, kv = paged_inputs(q_lens, [1200, 700], 8, 2, 64, 16, torch.float16, 30, DEV)
        ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), 0.125, torch.zeros_like(q))
        assert g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.125, max(q_lens), out=q) is q
        torch.cuda.synchronize()
        assert ((q.double() - ref).abs() <= tol).all() and g.device_status() == 0
    finally:
        g.set_option(g.GQAQ_OPT_PDL, 1)


def test_attn_a_bound_far_above_the_rows():
    attn_case([1, 1, 1], [300, 1, 77], 2, 2, 64, 16, "f16", seed=31, max_q=2 ** 31 - 1)


def test_attn_output_at_16_bytes():
    """An out that is 16-byte but not 32-byte aligned."""
    q, kp, vp, table, cu, kv = paged_inputs([200, 3], [400, 90], 4, 2, 128, 16, torch.bfloat16, 32, DEV)
    room = torch.zeros(q.numel() + 8, dtype=q.dtype, device=DEV)
    out = room[8:].view(q.shape)
    ref, tol = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), 0.09, torch.zeros_like(q))
    g.gqa_paged_attn(q, kp, vp, table, cu, kv, 0.09, 200, out=out)
    torch.cuda.synchronize()
    assert out.data_ptr() % 32 == 16 and ((out.double() - ref).abs() <= tol).all() and int(room[:8].count_nonzero()) == 0


def test_attn_workspace_is_reused_and_left_zero():
    d = g.make_paged_dims(1, 8, 2, 128, 16, 1, 1, 1)
    ws = g.alloc_paged_workspace(d, DEV)
    for ctas in (0, 5):
        g.set_option(g.GQAQ_OPT_MAX_CTAS, ctas)
        for rep in range(2):
            attn_case([1] * 6, [700, 1, 128, 1500, 129, 60], 4, 2, 128, 16, "f16", seed=rep, workspace=ws)
            attn_case([200, 1, 20], [900, 1500, 20], 4, 2, 128, 16, "bf16", seed=rep, workspace=ws)
            attn_case([9, 4], [900, 1500], 4, 2, 64, 16, "f16", seed=rep, workspace=ws)


def test_bindings_check_shapes_and_strides():
    q, kp, vp, table, cu, kv = paged_inputs([2, 3], [40, 50], 4, 2, 64, 16, torch.float16, 1, DEV)
    call = lambda **kw: g.gqa_paged_attn(**{**dict(q=q, k_pages=kp, v_pages=vp, block_table=table, cu_q=cu, kv_len=kv, scale=0.1, max_q_len=3), **kw})  # noqa: E731
    call()
    for bad in (dict(q=q.float()), dict(q=q[:, :, ::2]), dict(k_pages=kp.bfloat16()), dict(v_pages=vp[:-1]), dict(block_table=table.long()),
                dict(cu_q=cu[:-1]), dict(kv_len=kv[:1]), dict(out=q[:1]), dict(block_table=table[:, ::2]), dict(q=q[0])):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    with pytest.raises(g.GqaqError):
        call(max_q_len=0)
    with pytest.raises(g.GqaqError):
        call(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    k, v, pos, slots = q[:, :2].contiguous(), q[:, 2:].contiguous(), ints([0] * 5), ints(list(range(5)))
    app = lambda **kw: g.paged_norm_rope_append(**{**dict(q=q, k=k, v=v, positions=pos, slots=slots, k_pages=kp, v_pages=vp), **kw})  # noqa: E731
    app()
    for bad in (dict(k=q), dict(v=v.bfloat16()), dict(slots=slots[:-1]), dict(q_weight=q[0, 0].float()), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(cos_sin=torch.zeros(4, 64, device=DEV).half()), dict(v_pages=vp[:, :1])):
        with pytest.raises((ValueError, TypeError)):
            app(**bad)
    with pytest.raises(g.GqaqError):
        app(cos_sin=torch.zeros(4, 24, device=DEV))  # not a multiple of 16
    with pytest.raises(ValueError):
        g.paged_build_tables(kv, kv, pos, kv[:1], table[:1], 4)
    with pytest.raises(ValueError):
        g.paged_release_pages(kv, kv[:1], table, pos, kv[:1])
