"""Plain 64-bit definitions of the paged serving operators, and the inputs of their tests."""
import numpy as np
import torch

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def pages_of(n, S):
    return -(-n // S)


# ---------------------------------------------------------------------------
# Tables
# ---------------------------------------------------------------------------
def ref_tables(cache_len, new_len, free, count, table, T, S, num_pages):
    """One request after the other, as the header says. Returns (kv_len, cu, positions, slots, count, table)."""
    B, width = table.shape
    table = table.copy()
    kv, cu = np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    pos, slots = np.zeros(T, np.int64), np.full(T, -1, np.int64)
    rows, taken, full = 0, 0, False
    for b in range(B):
        c, n = int(cache_len[b]), int(new_len[b])
        ok = c >= 0 and n >= 0 and c + n <= width * S
        first = rows
        rows += max(n, 0)
        cu[b + 1] = min(rows, T)
        ok = ok and rows <= T
        if not ok:
            continue
        held, want = pages_of(c, S), pages_of(c + n, S)
        if want > held:
            if full or taken + want - held > count:
                full = True  # the sum with this request's pages is past the free ones for every later one as well
                continue
            for p in range(held, want):
                table[b, p] = free[count - 1 - taken]
                taken += 1
        kv[b] = c + n
        for i in range(n):
            page = table[b, (c + i) // S]
            pos[first + i] = c + i
            slots[first + i] = page * S + (c + i) % S if 0 <= page < num_pages else -1
    return kv, cu, pos, slots, count - taken, table


def ref_release(kv_len, keep_len, free, count, table, S):
    free, width = free.copy(), table.shape[1]
    for b in range(table.shape[0]):
        n, k = int(kv_len[b]), int(keep_len[b])
        if not (0 <= k <= n <= width * S):
            continue
        for p in range(pages_of(k, S), pages_of(n, S)):
            if count < free.size:
                free[count] = table[b, p]
                count += 1
    return free, count


# ---------------------------------------------------------------------------
# Norm, rotation, append
# ---------------------------------------------------------------------------
def angles(positions, R, base=10000.0):
    """The table of cosines and sines [positions, R] in 32 bits, from angles in 64."""
    inv = 1.0 / base ** (np.arange(0, R, 2, dtype=np.float64) / R)
    a = np.arange(positions, dtype=np.float64)[:, None] * inv
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32))


def ref_head_rows(x, weight, eps, cos_sin, positions, inter):
    """x [T,H,D] -> (norm and rotation in 64 bits, the size |a| + |b| of each value's terms)."""
    y = x.double()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    size = y.abs()
    if cos_sin is not None:
        R = cos_sin.shape[1]
        row = cos_sin.double()[positions.long()][:, None]
        cos, sin = row[..., :R // 2], row[..., R // 2:]
        i = torch.arange(R // 2, device=x.device)
        i, j = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
        a, b = y[..., i].clone(), y[..., j].clone()
        size[..., i] = size[..., j] = a.abs() + b.abs()
        y[..., i], y[..., j] = a * cos - b * sin, b * cos + a * sin
    return y, size


def rows_tolerance(ref, size, dtype):
    """One rounding to dtype; before it 32-bit arithmetic: the mean of at most 128 squares (a sum of depth <= 19:
    half of 19 steps after the root), rsqrt (2 units), five products and two additions, each at most 2^-24 of the
    terms' size: below 2^-19 of it. The last term is half a step of fp16's smallest numbers."""
    return half_step(dtype) * ref.abs() + 2.0 ** -19 * size + 2.0 ** -25


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def ref_attn(q, kp, vp, table, cu, kv_len, scale, out, max_q=None):
    """Row by row from the definition, in 64 bits. Returns (out, tolerance): see attn_tolerance."""
    T, Hq, D = q.shape
    num_pages, Hkv, S, _ = kp.shape
    G = Hq // Hkv
    ref, tol = out.double().clone(), torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    u = half_step(q.dtype)
    for b in range(len(kv_len)):
        q0, q1, L = int(cu[b]), int(cu[b + 1]), int(kv_len[b])
        n = q1 - q0
        m = n if max_q is None else min(n, max_q)
        if m <= 0:
            continue
        pg = table[b, :pages_of(L, S)].long()
        bad = (pg < 0) | (pg >= num_pages)
        pg = torch.where(bad, 0, pg)
        pos = torch.arange(m, device=q.device) + (L - n)
        seen = torch.arange(L, device=q.device)[None, :] <= pos[:, None]
        for h in range(Hkv):
            k, v = (torch.where(bad[:, None, None], 0.0, x[pg, h].double()).reshape(-1, D)[:L] for x in (kp, vp))
            for g in range(G):
                x = q[q0:q0 + m, h * G + g].double()
                s = torch.where(seen, x @ k.T * scale, -torch.inf)
                p = torch.exp(s - s.amax(1, keepdim=True).clamp(min=-1e300)) if L else s
                l = p.sum(1, keepdim=True)
                live = l > 0
                p = torch.where(live, p / torch.where(live, l, 1.0), 0.0)
                o = p @ v
                ref[q0:q0 + m, h * G + g] = o
                size = p @ v.abs()
                ds = (x.abs() @ k.abs().T * (scale if scale >= 0 else -scale)).amax(1, keepdim=True) if L else 0.0
                tol[q0:q0 + m, h * G + g] = attn_tolerance(o, size, ds, u, L, D, v.abs().max() if L else 0.0)
    return ref, tol


def attn_tolerance(out, size, score_size, u, L, D, vmax):
    """out = sum p v / l, size = sum p |v|. Each p is rounded once to the dtype (u of it, and half a step 2^-25 of
    fp16's smallest numbers where l >= 1) and so is out. In 32 bits: a score's D products and its scale are off by
    (D + 3) 2^-24 of the sum of their sizes, which moves p by as much; the exponential and the factors of a moved
    maximum by 2^-20; the sums of p and of p v over L tokens by L 2^-24 each."""
    f32 = 2.0 ** -24
    return u * out.abs() + size * (u + 2 * (D + 3) * f32 * score_size + 2.0 ** -20 + 2 * L * f32) + L * 2.0 ** -25 * vmax


def paged_inputs(q_lens, kv_lens, Hq, Hkv, D, S, dtype, seed, device, extra=3, width=None, gap=0, stale_nan=True, rows_behind=0):
    """q, pools, tables of a step. Rows of a page past its request's length, and pages no request holds, are NaN."""
    g = torch.Generator(device=device).manual_seed(seed)
    held = [pages_of(n, S) for n in kv_lens]
    total = sum(held) + extra
    T = gap + sum(q_lens) + rows_behind
    q = torch.randn(max(T, 1), Hq, D, generator=g, device=device).to(dtype)
    kp, vp = (torch.randn(total, Hkv, S, D, generator=g, device=device).to(dtype) for _ in range(2))
    order = torch.randperm(total, generator=g, device=device).to(torch.int32)
    width = max(max(held), 1) if width is None else width
    table = torch.full((len(kv_lens), width), -1, dtype=torch.int32, device=device)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
        if stale_nan and kv_lens[b] % S:
            last = order[at - 1].long()
            kp[last, :, kv_lens[b] % S:] = float("nan")
            vp[last, :, kv_lens[b] % S:] = float("nan")
    if stale_nan:
        kp[order[at:].long()] = float("nan")
        vp[order[at:].long()] = float("nan")
    cu = torch.tensor([gap + sum(q_lens[:i]) for i in range(len(q_lens) + 1)], dtype=torch.int32, device=device)
    kv = torch.tensor(kv_lens, dtype=torch.int32, device=device)
    return q, kp, vp, table, cu, kv


# ---------------------------------------------------------------------------
# Long contexts: inputs whose outputs show the loss of a key
# ---------------------------------------------------------------------------
def counting_ref(seen, heads, G, D):
    """Share of the first seen[t] tokens whose block of eight is channel d's for head h: token j's is (j // 8 + h / G) % D."""
    n, h = seen.double()[:, None, None], torch.arange(heads, device=seen.device)[None, :, None] // G
    e = (torch.arange(D, device=seen.device)[None, None, :] - h) % D
    whole = torch.div(n, 8 * D, rounding_mode="floor")
    return (whole * 8 + (n - whole * 8 * D - 8 * e).clamp(0, 8)) / n


def even_tolerance(ref, dtype):
    """Keys that weigh alike: each P is a power of two in the dtype, so only the sums and weights are off, all of one
    sign: an exponential and two merges (each 2^-22), a division, and sums that are at most 600 additions deep (the tiles
    of one CTA's range, the steps of a tile, warps, parts): 600 * 2^-24 < 2^-14 in all, and one rounding to the dtype."""
    return ref * (half_step(dtype) + 2.0 ** -14)


def _own_rows(q_lens, kv_lens, device):
    """For the token in each row of the step: its request, and the tokens it sees."""
    b = torch.cat([torch.full((n,), i, device=device) for i, n in enumerate(q_lens)])
    seen = torch.cat([torch.arange(L - n + 1, L + 1, device=device) for n, L in zip(q_lens, kv_lens)])
    return b, seen


def counting_case(q_lens, kv_lens, Hq, Hkv, D, S, dtype, seed, device):
    """q = 0, so every key weighs the same, and the values count keys: one that is lost, doubled or taken from
    another place moves a channel by 1 / (kv_len / D) of its value."""
    q, kp, vp, table, cu, kv = paged_inputs(q_lens, kv_lens, Hq, Hkv, D, S, dtype, seed, device)
    q.zero_()
    for b, L in enumerate(kv_lens):
        j, h = torch.arange(L, device=device)[:, None], torch.arange(Hkv, device=device)[None, :]
        one = torch.zeros(L, Hkv, D, dtype=dtype, device=device).scatter_(2, ((j // 8 + h) % D)[..., None], 1.0)
        vp[table[b, j // S].long(), h, j % S] = one
    ref = counting_ref(_own_rows(q_lens, kv_lens, device)[1], Hq, Hq // Hkv, D)
    return q, kp, vp, table, cu, kv, ref, even_tolerance(ref, dtype)


def dominant_case(q_lens, kv_lens, Hq, Hkv, D, S, dtype, seed, device):
    """Up to D keys per request and KV head, one in each stretch of the context, outweigh all others (e^-32 each), and
    each has a channel of its own: one that is not found leaves a channel at 0."""
    q, kp, vp, table, cu, kv = paged_inputs(q_lens, kv_lens, Hq, Hkv, D, S, dtype, seed, device)
    q.fill_(1.0)
    gen = torch.Generator(device=device).manual_seed(seed + 100)
    own, seen = _own_rows(q_lens, kv_lens, device)
    ref = torch.zeros(*q.shape, dtype=torch.float64, device=device)
    h = torch.arange(Hkv, device=device)[:, None]
    for b, L in enumerate(kv_lens):
        j = torch.arange(L, device=device)[:, None]
        kp[table[b, j // S].long(), h.T, j % S] = 0.0
        n = min(D, L)
        edge = torch.arange(n + 1, device=device) * L // n
        at = edge[:-1] + (torch.rand(Hkv, n, generator=gen, device=device) * (edge[1:] - edge[:-1])).long().minimum(edge[1:] - edge[:-1] - 1)
        page = table[b, at // S].long()
        kp[page, h, at % S] = 1.0
        vp[page, h, at % S] = torch.eye(D, dtype=dtype, device=device)[:n].expand(Hkv, n, D)
        rows = own == b
        found = (at[None] < seen[rows][:, None, None]).double()  # [row, KV head, key]
        ref[rows, :, :n] = (found / found.sum(-1, keepdim=True)).repeat_interleave(Hq // Hkv, dim=1)
    tol = even_tolerance(ref, dtype) + max(kv_lens) * 2.0 ** -46 * 8  # the other keys: e^-32 < 2^-46, |v| < 8
    return q, kp, vp, table, cu, kv, 32.0 / D, ref, tol
