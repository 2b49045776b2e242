"""The per-channel bound of tests/test_gpu_paged_e4m3_far.py on the CPU: it lets a softmax pass whose weights are rounded as
the kernels say, and sees one whose weights are rounded relative to 2^exponent."""
import pytest
import torch

from _paged_e4m3 import decode, pow2
from _paged_e4m3_far import softmax_bound


def model(s, codes, e, headroom, spread):
    """out of scores s [tokens] (base 2), E4M3 values codes [tokens, channels] and exponents e [tokens]. Weights 2^(s + e - reference)
    in fp16, the reference `headroom` under the row's largest; of tokens more than `spread` under the largest exponent so far in two
    bfloat16 numbers."""
    top = torch.cummax(e, 0).values
    w = torch.exp2(s + e - (s + e).max() + headroom)
    hi = w.bfloat16().double()
    far = hi + (w - hi).bfloat16().double()
    p = torch.where(top - e > spread, far, w.half().double())
    return p @ codes / (w * torch.exp2(-e)).sum()


@pytest.mark.parametrize("far", [4, 8, 12, 16, 20, 24, 40, 90])
def test_the_bound_sees_weights_relative_to_an_exponent(far):
    gen = torch.Generator().manual_seed(far)
    L, D = 2000, 16
    s = torch.randn(L, generator=gen, dtype=torch.float64) * 1.5
    codes = decode((torch.rand(L, D, generator=gen) * 120).to(torch.uint8))
    e = torch.full((L,), -40.0, dtype=torch.float64)
    codes[:16], e[:16] = 0.0, -40.0 + far
    codes[3, 5] = 448.0
    v = codes * pow2(e)[:, None]
    p = torch.exp2(s - s.max())[None]
    out = p @ v / p.sum()
    bound = softmax_bound(out, p, p.sum(1, keepdim=True), v, 0.0, torch.bfloat16)[0] - 2.0 ** -8 * out[0].abs()  # no rounding of the output here
    others = [c for c in range(D) if c != 5]
    assert ((model(s, codes, e, 6, 6) - out[0]).abs() <= bound)[others].all()
    if far >= 20:  # nearer, what single tokens lose averages out over 2000
        assert ((model(s, codes, e, 0, 200) - out[0]).abs() > bound)[others].any()
