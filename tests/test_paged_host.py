"""Refusals of the paged calls, without a GPU: every path returns before any CUDA call."""
import ctypes
import os

import pytest
import torch

import gqa_head_folding_gb300 as g
from _paged import counting_case, counting_ref, dominant_case, even_tolerance, ref_attn

FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced
OTHER = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10002)
OFF8 = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(g.LIB_PATH):
        from gqa_head_folding_gb300 import _build
        _build.build()
    return g.lib()


def dims(**kw):
    base = dict(batch=4, num_q_heads=32, num_kv_heads=8, head_dim=64, page_size=16, num_pages=100, max_pages=10, max_tokens=8)
    base.update(kw)
    return g.make_paged_dims(**base)


BAD_TABLES = [(dict(batch=0), 1), (dict(page_size=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(max_tokens=0), 1),
              (dict(page_size=12), 2), (dict(page_size=256), 2), (dict(batch=8193), 2), (dict(max_tokens=(1 << 22) + 1), 2),
              (dict(max_pages=1 << 28), 2), (dict(num_pages=1 << 28), 2), (dict(batch=8192, max_pages=1 << 19), 2)]
BAD_HEADS = BAD_TABLES + [(dict(num_q_heads=0), 1), (dict(num_kv_heads=0), 1), (dict(num_q_heads=30), 1), (dict(head_dim=96), 2),
                          (dict(num_q_heads=24), 2), (dict(num_q_heads=128), 2), (dict(num_pages=1 << 24, page_size=64), 2)]


def tables(L, d, at=None, ptr=None):
    p = [FAKE, FAKE, FAKE, FAKE, FAKE, OTHER, FAKE, FAKE, FAKE, FAKE]
    if at is not None:
        p[at] = ptr
    return L.paged_build_tables(None if d is None else ctypes.byref(d), *p, None)


@pytest.mark.parametrize("kw, status", BAD_TABLES)
def test_table_calls_refuse_dims(L, kw, status):
    assert tables(L, dims(**kw)) == status
    assert L.paged_release_pages(ctypes.byref(dims(**kw)), *[FAKE] * 6, None) == status


def test_table_calls_refuse_pointers(L):
    assert tables(L, None) == g.GQAQ_ERR_INVALID_ARG
    for i in range(10):
        assert tables(L, dims(), i, None) == g.GQAQ_ERR_INVALID_ARG
        assert tables(L, dims(), i, ODD) == g.GQAQ_ERR_INVALID_ARG
    assert tables(L, dims(), 5, FAKE) == g.GQAQ_ERR_INVALID_ARG  # kv_len in the place of cache_len
    for i in range(6):
        p = [FAKE, FAKE, FAKE, OTHER, FAKE, FAKE]
        p[i] = None
        assert L.paged_release_pages(ctypes.byref(dims()), *p, None) == g.GQAQ_ERR_INVALID_ARG
    assert L.paged_release_pages(ctypes.byref(dims()), *[FAKE] * 6, None) == g.GQAQ_ERR_INVALID_ARG  # the table as the list


def append(L, d, q=FAKE, sq=2048, k=FAKE, sk=512, v=FAKE, sv=512, pos=FAKE, slots=FAKE, wq=None, wk=None, eps=1e-6, cs=FAKE, rope=64,
           most=100, q_out=OTHER, kp=FAKE, vp=FAKE):
    return L.paged_norm_rope_append(None if d is None else ctypes.byref(d), q, sq, k, sk, v, sv, pos, slots, wq, wk, eps, cs, rope,
                                    most, 0, q_out, kp, vp, None)


@pytest.mark.parametrize("kw, status", BAD_HEADS)
def test_append_refuses_dims(L, kw, status):
    assert append(L, dims(**kw)) == status


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=OFF8), dict(v=None), dict(pos=None), dict(slots=ODD), dict(q_out=None), dict(kp=OFF8),
                                dict(vp=None), dict(wq=OFF8), dict(wk=OFF8), dict(sq=2047), dict(sq=2052), dict(sk=504), dict(sv=513),
                                dict(rope=8), dict(rope=80), dict(rope=-16), dict(cs=None), dict(cs=OFF8), dict(most=0),
                                dict(eps=float("nan")), dict(eps=-1.0), dict(q_out=FAKE, sq=4096)])
def test_append_refuses_arguments(L, kw):
    assert append(L, dims(), **kw) == g.GQAQ_ERR_INVALID_ARG


def attn(L, d, mq=1, q=FAKE, k=FAKE, v=FAKE, tab=FAKE, cu=FAKE, kv=FAKE, scale=0.1, out=FAKE, ws=FAKE):
    return L.gqa_paged_attn(None if d is None else ctypes.byref(d), mq, q, k, v, tab, cu, kv, scale, out, ws, 1 << 30, None)


@pytest.mark.parametrize("kw, status", BAD_HEADS)
def test_attn_refuses_dims(L, kw, status):
    assert attn(L, dims(**kw)) == status
    assert L.gqaq_paged_workspace_bytes(ctypes.byref(dims(**kw))) == 0


@pytest.mark.parametrize("kw", [dict(mq=0), dict(q=None), dict(k=OFF8), dict(v=None), dict(tab=None), dict(cu=ODD), dict(kv=None),
                                dict(scale=float("inf")), dict(out=OFF8)])
def test_attn_refuses_arguments(L, kw):
    assert attn(L, dims(), **kw) == g.GQAQ_ERR_INVALID_ARG
    assert attn(L, dims(), ws=None) == g.GQAQ_ERR_WORKSPACE
    assert attn(L, dims(), ws=OFF8) == g.GQAQ_ERR_WORKSPACE
    assert attn(L, None) == g.GQAQ_ERR_INVALID_ARG


def test_bindings_refuse_cpu_tensors_and_types():
    i = torch.ones(4, dtype=torch.int32)
    q = torch.zeros(4, 8, 64, dtype=torch.float16)
    kp = torch.zeros(3, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        g.paged_build_tables(i, i, i, i[:1], torch.zeros(4, 3, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        g.paged_release_pages(i, i, torch.zeros(4, 3, dtype=torch.int32), i, i[:1])
    with pytest.raises(ValueError, match="CUDA tensor"):
        g.paged_norm_rope_append(q, q[:, :2], q[:, :2], i, i, kp, kp)
    with pytest.raises(ValueError, match="CUDA tensor"):
        g.gqa_paged_attn(q, kp, kp, torch.zeros(4, 3, dtype=torch.int32), torch.zeros(5, dtype=torch.int32), i, 0.1, 1)
    with pytest.raises(ValueError, match="bfloat16"):
        g.make_paged_dims(1, 8, 2, 64, 16, 10, 10, 1, torch.float32)


@pytest.mark.parametrize("q, kv, status", [(1 << 19, 1 << 18, 1), ((1 << 19) + 2, (1 << 18) + 1, 2), (1 << 23, 1 << 23, 2), (1 << 29, 1 << 26, 2)])
def test_head_counts_are_limited(q, kv, status):
    """2^20 heads in all pass on to the next check (a missing pointer), more do not."""
    d = dims(num_q_heads=q, num_kv_heads=kv, num_pages=1, page_size=8, max_tokens=1)
    assert append(L=g.lib(), d=d, q=None, sq=1 << 40, sk=1 << 40, sv=1 << 40) == status
    assert attn(g.lib(), d, q=None) == status


def test_numbers_past_32_bits_are_refused():
    for kw in (dict(num_pages=2 ** 32 + 4), dict(max_tokens=2 ** 31), dict(page_size=2 ** 32 + 16), dict(max_len=-2 ** 31 - 1)):
        with pytest.raises(ValueError, match=next(iter(kw))):
            dims(**kw)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
def test_long_context_bound_sees_a_lost_page(dtype, D):
    """Leaving out (or counting twice) any page of 40,000 tokens moves an output of the counting case past its bound, a page of
    eight as well as a tile of 128; in fp16 a single key does."""
    L, heads = 39990, 2
    ref = counting_ref(torch.tensor([L]), heads, 1, D)[0]
    tol = even_tolerance(ref, dtype)
    for size in (8, 16, 128) + ((1,) if dtype == torch.float16 else ()):
        first = torch.arange(1, L, size)
        upto = lambda n: counting_ref(n, heads, 1, D) * n[:, None, None]  # noqa: E731
        lost = upto((first + size).clamp(max=L)) - upto(first)
        n = lost.sum(-1, keepdim=True)
        for wrong in ((ref * L - lost) / (L - n), (ref * L + lost) / (L + n)):
            assert ((wrong - ref).abs() > tol).any(-1).all()


def test_long_context_cases_agree_with_the_definition():
    for case in (counting_case, dominant_case):
        for dtype in (torch.float16, torch.bfloat16):
            args = ([1, 5, 40], [700, 23, 301], 4, 2, 64, 16, dtype, 3, "cpu")
            q, kp, vp, table, cu, kv, *scale, ref, tol = case(*args)
            want, _ = ref_attn(q, kp, vp, table, cu.tolist(), kv.tolist(), scale[0] if scale else 0.125, torch.zeros_like(q))
            assert ((want - ref).abs() <= tol).all() and bool((ref.sum(-1) - 1).abs().max() < 1e-9)
