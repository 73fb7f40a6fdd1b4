"""Plain 64-bit forms of rotate-and-append, shared-prefix decode, block bounds,
block choice and block-sparse decode, for the tests (CPU tensors, loops)."""
import math

import torch

BS = 16
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HEAD_DIM = {"f32": 64, "f16": 128, "bf16": 128}
# rounding to the type is off by at most this, relative to the value
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def make_cache(lens, hkv, ty, *, seed, spare=3, shared=()):
    """Caches and tables for sequences of these lengths, NaN in every slot without a token.

    shared: (first, last, tokens) sequences first .. last-1 have the same blocks for their first `tokens` tokens."""
    g = torch.Generator().manual_seed(seed)
    d, t = HEAD_DIM[ty], TYPES[ty]
    nblk = [-(-n // BS) for n in lens]
    total = sum(nblk) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    tables = torch.full((len(lens), max([1] + nblk) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = perm[at:at + n]
        at += n
    for first, last, tokens in shared:
        if last > first:
            tables[first:last, :tokens // BS] = tables[first, :tokens // BS].clone()
    k = torch.full((total, BS, hkv, d), float("nan"), dtype=t)
    v = torch.full((total, BS, hkv, d), float("nan"), dtype=t)
    for b, n in enumerate(lens):
        for j in range(nblk[b]):
            live = min(BS, n - j * BS)
            block = int(tables[b, j])
            k[block, :live] = torch.randn((live, hkv, d), generator=g).to(t)
            v[block, :live] = torch.randn((live, hkv, d), generator=g).to(t)
    return k, v, tables, torch.tensor(lens, dtype=torch.int32)


def make_q(n, heads, ty, seed):
    g = torch.Generator().manual_seed(seed + 7919)
    return torch.randn((n, heads, HEAD_DIM[ty]), generator=g).to(TYPES[ty])


def attention(q, k, v, tables, lens, scale, selected=None):
    """(out, weight): softmax attention in 64 bits, and the softmax-weighted mean of |V| (what a relative error of
    the weights is multiplied by)."""
    S, hq, d = q.shape
    hkv = k.shape[2]
    G = hq // hkv
    out = torch.zeros((S, hq, d), dtype=torch.float64)
    weight = torch.zeros((S, hq, d), dtype=torch.float64)
    for b in range(S):
        L = int(lens[b])
        n = -(-L // BS)
        if n == 0:
            continue
        ids = tables[b, :n].long()
        kb = k[ids].reshape(n * BS, hkv, d)[:L].double()
        vb = v[ids].reshape(n * BS, hkv, d)[:L].double()
        for g in range(hkv):
            keep = torch.arange(L)
            if selected is not None:
                chosen = selected[b, g][selected[b, g] >= 0].long()
                keep = (chosen[:, None] * BS + torch.arange(BS)).flatten()
                keep = keep[keep < L]
                if keep.numel() == 0:
                    continue
            p = torch.softmax(scale * (q[b, g * G:(g + 1) * G].double() @ kb[keep, g].T), -1)
            out[b, g * G:(g + 1) * G] = p @ vb[keep, g]
            weight[b, g * G:(g + 1) * G] = p @ vb[keep, g].abs()
    return out, weight


def attention_tolerance(ref, weight, ty, p_bits):
    """Output rounding, plus the weights' relative error times their mean of |V|: P is rounded to p_bits bits; a score
    of magnitude below 16 summed in fp32 over head_dim <= 128 products of N(0, 1) values is off by less than
    128 * 2^-24 * sum |q k| * scale < 2^-14, twice that for the exponential, sum and join."""
    return HALF_STEP[ty] * ref.abs() + (2.0 ** -p_bits + 2.0 ** -13) * weight * (1 + HALF_STEP[ty]) + 1e-7


def rotate(x, positions, cos_sin, interleaved):
    """x [T, H, D] float64 rotated by the table's entries; also the sum of the two products' magnitudes."""
    r = cos_sin.shape[1]
    cs = cos_sin.double()[positions.clamp(min=0)]
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    y, mag = x.clone(), x.abs().clone()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        ia, ib = slice(0, r, 2), slice(1, r, 2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        ia, ib = slice(0, r // 2), slice(r // 2, r)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, mag


def rope_table(max_position, rotary, base):
    p = torch.arange(max_position, dtype=torch.float64)[:, None]
    angle = p * torch.tensor([base ** (-2.0 * i / rotary) for i in range(rotary // 2)], dtype=torch.float64)
    return torch.cat([angle.cos(), angle.sin()], 1)


def block_bounds(k, bounds, tables, lens, new):
    """`bounds` with the touched blocks' entries recomputed (exact: smallest and largest of stored values)."""
    out = bounds.clone()
    for b in range(len(lens)):
        L, n = int(lens[b]), int(new[b])
        if n == 0:
            continue
        for j in range((L - n) // BS, -(-L // BS)):
            block = int(tables[b, j])
            rows = k[block, :min(BS, L - j * BS)].float()
            out[block, 0], out[block, 1] = rows.amin(0).to(k.dtype), rows.amax(0).to(k.dtype)
    return out


def choose(q, bounds, tables, lens, K, sink, recent):
    S, hq, d = q.shape
    hkv = bounds.shape[2]
    G = hq // hkv
    out = torch.full((S, hkv, K), -1, dtype=torch.int32)
    for b in range(S):
        n = -(-int(lens[b]) // BS)
        if n == 0:
            continue
        rows = bounds[tables[b, :n].long()].double()
        for g in range(hkv):
            if n <= K:
                out[b, g, :n] = torch.arange(n, dtype=torch.int32)
                continue
            best = []
            for j in range(n):
                lo, hi = rows[j, 0, g], rows[j, 1, g]
                top = -math.inf
                for h in range(g * G, (g + 1) * G):
                    x = q[b, h].double()
                    s = float((x * torch.where(x >= 0, hi, lo)).sum())
                    top = math.inf if math.isnan(s) or top == math.inf else max(top, s)
                best.append(math.inf if j < sink or j >= n - recent else top)
            # the forced blocks come first, then by score, ties to the lowest index
            order = sorted(range(n), key=lambda j: (not (j < sink or j >= n - recent), -best[j], j))[:K]
            out[b, g] = torch.tensor(sorted(order), dtype=torch.int32)
    return out
