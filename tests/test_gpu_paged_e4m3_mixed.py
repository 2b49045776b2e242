"""Steps over 8-bit pages whose two attention launches run side by side: what an append has just written is read by both."""
import pytest
import torch

import gqa_head_folding_gb300 as g
from _paged import pages_of
from _paged_e4m3 import ref_attn_e4m3

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _clean():
    g.device_status()
    yield
    g.set_option(g.GQAQ_OPT_PDL, 1)


@pytest.mark.parametrize("new, held", [([1, 90, 1, 2], [4000, 2500, 16, 1800]), ([1] * 30 + [40], [37 * i for i in range(30)] + [300]),
                                       ([200, 1], [7, 9000]), ([3, 12, 30, 1], [500, 0, 80, 6000])])
@pytest.mark.parametrize("dtype, D, S", [(torch.float16, 64, 16), (torch.bfloat16, 128, 8)])
def test_attention_reads_the_append_before_it(new, held, dtype, D, S):
    """Append and attention in turn, six times: each append writes the rows, their pages' codes and exponents that the call behind it reads, with
    rows of the output before it. With early launches and without them, and as a graph's nodes, the same bits."""
    Hq, Hkv, B, T = 8, 2, len(new), sum(new)
    gen = torch.Generator(device=DEV).manual_seed(T)
    most = [pages_of(h + n, S) for h, n in zip(held, new)]
    pool = sum(most)
    table = torch.full((B, max(most)), -1, dtype=torch.int32)
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(1)).int()
    for b, n in enumerate(most):
        table[b, :n] = order[sum(most[:b]):sum(most[:b]) + n]
    pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, new)])
    own = torch.cat([torch.full((n,), b) for b, n in enumerate(new)])
    slots = (table[own, pos // S] * S + pos % S).int().to(DEV)
    pos, table = pos.int().to(DEV), table.to(DEV)
    cu = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    kv = torch.tensor([h + n for h, n in zip(held, new)], dtype=torch.int32, device=DEV)
    first = [torch.randint(0, 120, (pool, Hkv, S, D), generator=gen, device=DEV).to(torch.uint8) for _ in range(2)]
    first += [torch.randint(-9, -6, (pool, Hkv), generator=gen, device=DEV).to(torch.int8) for _ in range(2)]
    kp, vp, ke, ve = (t.clone() for t in first)
    x0 = torch.randn(T, Hq, D, generator=gen, device=DEV).to(dtype)
    outs = [torch.zeros(T, Hq, D, dtype=dtype, device=DEV) for _ in range(2)]
    q_out = torch.zeros(T, Hq, D, dtype=dtype, device=DEV)
    ws = g.alloc_paged_workspace(g.paged_dims_of(x0, kp, table), DEV)
    st = torch.cuda.Stream()

    def chain():
        for t, f in zip((kp, vp, ke, ve), first):
            t.copy_(f)
        x = x0
        for i in range(6):
            # rows of the last output as keys and values, so that a key or an exponent read too early shows in the end
            g.paged_norm_rope_append_e4m3(x, x[:, 0:Hkv], x[:, Hkv:2 * Hkv], pos, slots, kp, vp, ke, ve, q_out=q_out)
            x = g.gqa_paged_attn_e4m3(q_out, kp, vp, ke, ve, table, cu, kv, 0.2, max(new), out=outs[i % 2], workspace=ws)
        return x

    torch.cuda.synchronize()
    got = []
    for pdl in (0, 1):
        g.set_option(g.GQAQ_OPT_PDL, pdl)
        with torch.cuda.stream(st):
            for _ in range(3):
                got.append([t.clone() for t in (chain(), kp, vp, ke, ve)])
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=st):
                last = chain()
            for _ in range(3):
                gr.replay()
                got.append([t.clone() for t in (last, kp, vp, ke, ve)])
        st.synchronize()
    for x in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, got[0]))
    assert int(ws[:4096].count_nonzero()) == 0 and g.device_status() == 0
    ref, tol = ref_attn_e4m3(q_out, kp, ke, vp, ve, table, cu.tolist(), kv.tolist(), 0.2, torch.zeros_like(q_out))
    assert ((last.double() - ref).abs() <= tol).all()
