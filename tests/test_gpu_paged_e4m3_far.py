"""Attention over 8-bit pages that lie far apart: an output's channel is as exact as the values that fill it, whatever
other channels of other pages hold."""
import pytest
import torch

import gqa_head_folding_gb300 as g
from _paged import DTYPES, pages_of
from _paged_e4m3 import quantized_inputs
from _paged_e4m3_far import channels_by_level, one_large_channel, ref_far, wide_rows_of_q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# one to four blocks of eight rows in the decode kernel; one row tile and two in the tensor-memory kernel, and single tokens beside
STEPS = [([1, 1], [900, 2500], 4), ([3, 1], [700, 1900], 4), ([5, 4], [900, 2100], 4), ([8, 1], [600, 1300], 4),
         ([40, 1], [800, 1500], 4), ([300, 2], [1500, 700], 1)]


@pytest.fixture(autouse=True)
def _clean():
    g.device_status()
    yield
    g.set_option(g.GQAQ_OPT_MAX_CTAS, 0)


def check(x, scale, channels=slice(None)):
    q, kp, ke, vp, ve, table, cu, kv = x
    ref, tol = ref_far(*x[:6], cu.tolist(), kv.tolist(), scale)
    out = g.gqa_paged_attn_e4m3(q, kp, vp, ke, ve, table, cu, kv, scale, int((cu[1:] - cu[:-1]).max()), out=torch.zeros_like(q))
    err, tol = (out.double() - ref).abs()[..., channels], tol[..., channels]
    assert (err <= tol).all(), f"{(err / tol.clamp(min=1e-300)).max():.3g} of its bound"
    assert g.device_status() == 0
    return out


@pytest.mark.parametrize("far", [5, 6, 7, 8, 12, 16, 20, 24, 30, 57])
@pytest.mark.parametrize("dtype, D, S", [("f16", 64, 16), ("bf16", 128, 8), ("f16", 128, 64)])
def test_one_large_channel(far, dtype, D, S):
    """The other channels do not lose a bit to it."""
    others = [c for c in range(D) if c != 5]
    for i, (q_lens, kv_lens, G) in enumerate(STEPS):
        for where in ("first", "middle", "last"):
            g.set_option(g.GQAQ_OPT_MAX_CTAS, 2 if where == "middle" else 0)
            check(one_large_channel(q_lens, kv_lens, G, D, S, DTYPES[dtype], far, where, i, DEV), D ** -0.5, others)


@pytest.mark.parametrize("ctas", [0, 1])
@pytest.mark.parametrize("dtype, D, S, levels", [("f16", 64, 8, [-14, -11, -7, -4, 0, 4, 6]), ("bf16", 64, 16, [-48, -30, -12, 0, 7, 30, 48]),
                                                 ("bf16", 128, 128, [-48, 48]), ("bf16", 128, 8, [-48, -41, -20, 0, 5, 11, 48])])
def test_channels_of_pages_far_apart(dtype, D, S, levels, ctas):
    g.set_option(g.GQAQ_OPT_MAX_CTAS, ctas)
    for i, (q_lens, kv_lens, G) in enumerate(STEPS):
        check(channels_by_level(q_lens, kv_lens, G, D, S, DTYPES[dtype], levels, i, DEV), D ** -0.5)


@pytest.mark.parametrize("low", [-7, -14, -26, -48])
@pytest.mark.parametrize("D", [64, 128])
def test_half_of_a_small_page(low, D):
    """Equal scores, a page of zeros with a large exponent before one of ones with a small one: half of the latter."""
    for n in (1, 2, 3, 4, 16, 17):
        q = torch.zeros(2 * n, 8, D, dtype=torch.bfloat16, device=DEV)
        kp, vp = (torch.zeros(4, 2, 128, D, dtype=torch.uint8, device=DEV) for _ in range(2))
        ke, ve = (torch.zeros(4, 2, dtype=torch.int8, device=DEV) for _ in range(2))
        vp[1::2] = 0x38  # 1.0
        ve[0::2], ve[1::2] = 48 if low == -48 else 0, low
        table = torch.tensor([[0, 1, 2], [2, 3, 0]], dtype=torch.int32, device=DEV)
        cu, kv = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, n, 2 * n], [256, 256]))
        out = check((q, kp, ke, vp, ve, table, cu, kv), 0.1)
        last = out[[n - 1, 2 * n - 1]].double() * 2.0 ** -low
        assert ((last - 0.5).abs() <= 0.5 * 2.0 ** -8).all()


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_bfloat16_with_unlike_channels(D):
    for i, (q_lens, kv_lens, G) in enumerate(STEPS):
        check(wide_rows_of_q(q_lens, kv_lens, G, D, 16, i, DEV), D ** -0.5)


@pytest.mark.parametrize("size, ke, scale", [(2.0 ** 100, 48, 0.125), (2.0 ** 127, 0, 2.0 ** 20), (-2.0 ** 110, 30, -1.0), (2.0 ** 127, -48, 1.0)])
@pytest.mark.parametrize("q_lens, kv_lens, G", STEPS)
def test_keys_of_zero_meet_huge_queries(size, ke, scale, q_lens, kv_lens, G):
    """A product of zero is zero, however large the factor that it is taken times."""
    x = list(quantized_inputs(q_lens, kv_lens, 2 * G, 2, 64, 16, torch.bfloat16, 3, DEV))
    x[0].fill_(size)
    x[1] = torch.where(x[1] == 127, x[1], torch.zeros_like(x[1]))
    x[2] = torch.where(x[2] == -128, x[2], torch.full_like(x[2], ke))
    check(x, scale)


@pytest.mark.parametrize("D, S", [(64, 16), (128, 8)])
def test_requests_of_unlike_sizes(D, S):
    """Each request's pages are of one size, 2^96 apart from the next one's; so are a request's KV heads."""
    for i, (q_lens, kv_lens, G) in enumerate([([1, 1, 1], [900, 2500, 40], 4), ([5, 4, 2], [900, 30, 2100], 4), ([40, 1, 30, 1], [800, 1500, 50, 3], 4)]):
        x = list(quantized_inputs(q_lens, kv_lens, 2 * G, 2, D, S, torch.bfloat16, i, DEV))
        for b, L in enumerate(kv_lens):
            page = x[5][b, :pages_of(L, S)].long()
            x[4][page, 0], x[4][page, 1] = (-48, 48) if b % 2 else (48, -48)
        check(x, D ** -0.5)


@pytest.mark.parametrize("rows", [1, 70])
def test_wide_offsets_by_channel(rows):
    """Pools of more than 2^32 bytes, their last pages in use; 40,000 tokens, among them pages 20 exponents above the others."""
    Hkv, S, D = 8, 128, 128
    pages, n = 34000, pages_of(40000, 128)  # * 8 * 128 * 128 = 4.4e9
    (kp, ke), (vp, ve) = (g.new_pages_e4m3(pages, Hkv, S, D, DEV) for _ in range(2))
    gen = torch.Generator(device=DEV).manual_seed(rows)
    for codes, e in ((kp, ke), (vp, ve)):
        codes[-n:] = (torch.randn(n, Hkv, S, D, generator=gen, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        e[-n:] = torch.randint(-9, -6, (n, Hkv), generator=gen, device=DEV).to(torch.int8)
    large = torch.randperm(n, generator=gen, device=DEV)[:5] + pages - n
    ve[large] = 12
    vp[large] = 0
    vp[large, :, :, 7] = 0x38  # 1.0
    table = torch.arange(pages - n, pages, dtype=torch.int32, device=DEV).flip(0)[None].contiguous()
    q = torch.randn(rows, 16, D, generator=gen, device=DEV).half()
    cu, kv = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, rows], [39990]))
    out = g.gqa_paged_attn_e4m3(q, kp, vp, ke, ve, table, cu, kv, D ** -0.5, rows)
    here = table - (pages - n)
    ref, tol = ref_far(q, kp[-n:], ke[-n:], vp[-n:], ve[-n:], here, [0, rows], [39990], D ** -0.5)
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), f"{(err / tol).max():.3g} of its bound"
    assert g.device_status() == 0
