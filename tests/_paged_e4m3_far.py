"""Attention over 8-bit pages against the definition in 64 bits, with a bound for each channel: inputs whose pages lie
far apart, and what the output may be off by in the channels that only the smaller pages fill."""
import torch

from _paged import half_step, pages_of
from _paged_e4m3 import LEAST, MOST, pow2, quantized_inputs, values

P_STEP = 2.0 ** -11   # half a step of fp16, relative
P_LEAST = 2.0 ** -25  # half a step of fp16's smallest numbers


def softmax_bound(out, p, l, v, score_off, dtype):
    """What out = sum p v / l (p: 2^score, the largest 1; [rows, tokens]) may be off by, [rows, channels]. Each p is rounded to
    half a step of fp16, or to half of fp16's smallest step of the row's largest p, whatever the pages' exponents; a score is off by
    score_off, which moves p by as much; in 32 bits an exponential and the factors of moved maxima are off by 2^-20, the sums over L
    tokens by L 2^-24 each. The output is rounded once, in fp16 to half of its smallest step at least."""
    L = v.shape[0]
    size = p @ v.abs() / l
    off = P_STEP + 2 * score_off + 2.0 ** -20 + 2 * L * 2.0 ** -24
    return half_step(dtype) * out.abs() + size * off + P_LEAST * v.abs().sum(0) / l + (P_LEAST if dtype == torch.float16 else 0.0)


def ref_far(q, kp, ke, vp, ve, table, cu, kv_len, scale):
    """(out, bound) of the rows of all requests; others are 0, with a bound of 0. A bfloat16 row of q is taken in fp16 relative
    to its largest channel, which lies in [2^14, 2^15): a channel is off by 2^-25 / 2^14 of it at most."""
    T, Hq, D = q.shape
    Hkv, S = kp.shape[1:3]
    G = Hq // Hkv
    ke, ve = (e.clamp(LEAST, MOST) for e in (ke, ve))
    ref, tol = (torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device) for _ in range(2))
    for b in range(len(kv_len)):
        q0, q1, L = int(cu[b]), int(cu[b + 1]), int(kv_len[b])
        held = table[b, :pages_of(L, S)].long()
        seen = torch.arange(L, device=q.device)[None, :] <= torch.arange(L - q1 + q0, L, device=q.device)[:, None]
        for h in range(Hkv):
            k, v = (values(c[held, h:h + 1], e[held, h:h + 1]).reshape(-1, D)[:L] for c, e in ((kp, ke), (vp, ve)))
            for j in range(h * G, h * G + G):
                x = q[q0:q1, j].double()
                s = torch.where(seen, x @ k.T * scale, -torch.inf)
                p = torch.exp(s - s.amax(1, keepdim=True))
                l = p.sum(1, keepdim=True)
                o = p @ v / l
                off = (D + 3) * 2.0 ** -24 * (x.abs() @ k.abs().T * abs(scale)).amax(1, keepdim=True)
                if q.dtype == torch.bfloat16:
                    off = off + 2.0 ** -39 * x.abs().amax(1, keepdim=True) * k.abs().sum(1).max() * abs(scale)
                ref[q0:q1, j], tol[q0:q1, j] = o, softmax_bound(o, p, l, v, off, q.dtype)
    return ref, tol


def one_large_channel(q_lens, kv_lens, G, D, S, dtype, far, where, seed, device):
    """In each request and KV head one token has one large channel (5) and zeros beside it, on a page of its own kind `far`
    exponents above the others: first, in the middle or last of those that every row sees."""
    x = list(quantized_inputs(q_lens, kv_lens, 2 * G, 2, D, S, dtype, seed, device))
    vp, ve, table = x[3], x[4], x[5]
    ve[ve != -128] = -9
    for b, (n, L) in enumerate(zip(q_lens, kv_lens)):
        most = (L - n) // S  # the pages that every row sees whole
        page = table[b, {"first": 0, "middle": most // 2, "last": most - 1}[where]].long()
        vp[page] = 0
        vp[page, :, S // 2, 5] = 0x7e  # 448
        ve[page] = -9 + far
    return x


def channels_by_level(q_lens, kv_lens, G, D, S, dtype, levels, seed, device):
    """Each page's exponent is one of the levels, and it has values in every len(levels)-th channel only, so that a channel is
    filled by pages of one size."""
    x = list(quantized_inputs(q_lens, kv_lens, 2 * G, 2, D, S, dtype, seed, device))
    vp, ve = x[3], x[4]
    level = torch.randint(0, len(levels), ve.shape, generator=torch.Generator(device=device).manual_seed(seed + 7), device=device)
    mine = torch.arange(D, device=device)[None, None, :] % len(levels) == level[:, :, None]
    keep = mine[:, :, None, :] | (vp == 127)  # stale rows stay NaN
    x[3] = torch.where(keep, vp, torch.zeros_like(vp))
    x[4] = torch.where(ve == -128, ve, torch.tensor(levels, device=device)[level].to(torch.int8))
    return x


def wide_rows_of_q(q_lens, kv_lens, G, D, S, seed, device):
    """bfloat16 rows whose first channels are up to 2^40 times the others, over keys that are zero in those: the small channels
    decide the scores."""
    x = list(quantized_inputs(q_lens, kv_lens, 2 * G, 2, D, S, torch.bfloat16, seed, device))
    q, kp = x[0].float(), x[1]
    q[..., :8] *= pow2(torch.arange(8, device=device) * 5 + 5).float()
    kp[..., :8] = torch.where(kp[..., :8] == 127, kp[..., :8], torch.zeros_like(kp[..., :8]))
    x[0] = q.bfloat16()
    return x
