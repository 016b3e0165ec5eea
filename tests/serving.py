"""64-bit references of the rotary, append and shared-prefix tests (no code of the package)."""
import math

import torch


def frequencies(rot, *, base=10000.0, scaling="none", factor=1.0, original_ctx=8192, low=1.0, high=4.0, slow=1.0,
                fast=32.0):
    """Angle per position of each pair, from the definition."""
    res = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" and rot > 2 else base
        f = b ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            turns = original_ctx * f / (2 * math.pi)
            keep = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = keep * f + (1 - keep) * f / factor
        elif scaling == "yarn":
            def corner(n):
                return rot * math.log(original_ctx / (2 * math.pi * n)) / (2 * math.log(base))
            lo, hi = max(math.floor(corner(fast)), 0), min(math.ceil(corner(slow)), rot - 1)
            ramp = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
            f = f * (1 - ramp) + f / factor * ramp
        res.append(f)
    return torch.tensor(res, dtype=torch.float64)


def amplitude(scaling, factor):
    return 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0


def rotate64(x, pos, rot, layout, freq, amp=1.0, transpose=False):
    """x [tokens, heads, d] rotated by the pairs' 2 x 2 matrices, float64."""
    x = x.double().clone()
    ang = pos.double()[:, None] * freq
    c, s = amp * torch.cos(ang)[:, None], amp * torch.sin(ang)[:, None]
    if transpose:
        s = -s
    ia = torch.arange(rot // 2) if layout == "half" else torch.arange(0, rot, 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    return x


def dense64(q, k_cache, v_cache, page_table, seq_lens):
    """Softmax attention of one token per sequence through its own page table, float64 [B, Hq, d]."""
    B, Hq, d = q.shape
    Hkv, ps = k_cache.shape[1], k_cache.shape[2]
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(seq_lens[b])
        if n == 0:
            continue
        pages = page_table[b, :-(-n // ps)].long()
        k, v = (c[pages].double().permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n] for c in (k_cache, v_cache))
        x = q[b].double().view(Hkv, Hq // Hkv, d) @ k.transpose(1, 2) / math.sqrt(d)
        out[b] = (torch.softmax(x, -1) @ v).reshape(Hq, d)
    return out


def shared_batch(sizes, prefixes, own, *, Hq, Hkv, d, ps, dtype, seed=0, spare=2, garbage=float("nan")):
    """A batch of groups over a shuffled page pool. own[b] positions behind (negative: short of) the prefix.

    Rows that belong to no position hold `garbage`."""
    g = torch.Generator().manual_seed(seed)
    B = sum(sizes)
    start = [0]
    for z in sizes:
        start.append(start[-1] + z)
    lens = [max(prefixes[k] + own[b], 0) for k in range(len(sizes)) for b in range(start[k], start[k + 1])]
    max_ctx = max(max(lens), max(prefixes), 1)
    pps = -(-max_ctx // ps)
    table = torch.full((B, pps), -1, dtype=torch.int64)
    n_pages = 0
    content = []  # (page, rows written, copied from page)
    for k in range(len(sizes)):
        if sizes[k] == 0:
            continue
        whole, rest = divmod(prefixes[k], ps)
        first = start[k]
        shared = list(range(n_pages, n_pages + whole))
        n_pages += whole
        content += [(p, ps, None) for p in shared]
        for b in range(first, start[k + 1]):
            # the first sequence of a group lists the whole prefix whatever its length
            n = max(lens[b], prefixes[k]) if b == first else lens[b]
            need = -(-n // ps)
            row = shared[:min(whole, need)]
            for s in range(len(row), need):
                rows = min(ps, n - s * ps)
                copy = int(table[first, s]) if b > first and s == whole and rest else None
                content.append((n_pages, rows, (copy, min(rest, rows)) if copy is not None else None))
                row.append(n_pages)
                n_pages += 1
            table[b, :need] = torch.tensor(row, dtype=torch.int64)
    pool = n_pages + spare
    perm = torch.randperm(pool, generator=g)
    k = torch.full((pool, Hkv, ps, d), garbage)
    v = torch.full((pool, Hkv, ps, d), garbage)
    for page, rows, copy in content:
        k[perm[page], :, :rows] = torch.randn(Hkv, rows, d, generator=g)
        v[perm[page], :, :rows] = torch.randn(Hkv, rows, d, generator=g)
        if copy is not None:
            for c in (k, v):
                c[perm[page], :, :copy[1]] = c[perm[copy[0]], :, :copy[1]]
    table = torch.where(table >= 0, perm[table.clamp_min(0)], table).int()
    q = torch.randn(B, Hq, d, generator=g)
    i32 = dict(dtype=torch.int32)
    return dict(q=q.to(dtype), k_cache=k.to(dtype), v_cache=v.to(dtype), page_table=table,
                seq_lens=torch.tensor(lens, **i32), group_start=torch.tensor(start, **i32),
                prefix_lens=torch.tensor(prefixes, **i32), num_pages=pool, max_ctx=max_ctx)
