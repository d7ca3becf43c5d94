"""Plain fp64 definitions of the paged cache's operators (include/dckv_cache.h), for tests.

Everything is torch float64 on the inputs' device and walks tokens and sequences one by one.
`pool` tensors are [layers, pages, rows, heads, dim]; lens, news and tables are Python lists.
"""
import math

import torch


def rope_freq(rotary, base=1.0e7, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    out = []
    for i in range(rotary // 2):
        if scaling == "ntk":
            f = (base * factor ** (rotary / (rotary - 2))) ** (-2 * i / rotary)
        else:
            f = base ** (-2 * i / rotary)
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            w = (original_len * f / (2 * math.pi) - low) / (high - low)
            w = min(1.0, max(0.0, w))
            f = w * f + (1 - w) * f / factor
        out.append(f)
    return out


def rope(x, positions, freq, layout="half", mode="forward", magnitude=1.0):
    """x [n, heads, dim], positions [n]: (rotated fp64, |a| + |b| of each element's pair times the
    magnitude -- what an error in cos or sin is multiplied by)."""
    x = x.double()
    r = 2 * len(freq)
    ang = positions.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    c, s = torch.cos(ang), torch.sin(ang)
    m = 1.0 / magnitude if mode == "inverse" else magnitude
    if mode != "forward":
        s = -s
    first = list(range(r // 2)) if layout == "half" else list(range(0, r, 2))
    second = [i + r // 2 for i in first] if layout == "half" else [i + 1 for i in first]
    a, b = x[..., first], x[..., second]
    out, size = x.clone(), torch.zeros_like(x)
    out[..., first] = m * (a * c - b * s)
    out[..., second] = m * (b * c + a * s)
    size[..., first] = size[..., second] = m * (a.abs() + b.abs())
    return out, size


def slots(table, count, page_size):
    j = torch.arange(count)
    pages = torch.tensor(table, dtype=torch.int64)
    return pages[j // page_size] if count else pages[:0], j % page_size


def attention(q, k_pool, v_pool, news, lens, tables, scale, causal):
    """q [n, q heads, dim] over one layer's pools [pages, rows, heads, dim].  Returns fp64 out,
    lse, and two sizes for error bounds: mass [n, q heads, dim] = sum of weight |v| and reach
    [n, q heads] = the largest scale * sum |q||k| of the slots a row sees."""
    n, hq, d = q.shape
    g = hq // k_pool.shape[2]
    q = q.double()
    out, mass = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    reach = torch.zeros_like(lse)
    at = 0
    for new, length, table in zip(news, lens, tables):
        pages, rows = slots(table, length, k_pool.shape[1])
        pages, rows = pages.to(q.device), rows.to(q.device)
        k, v = k_pool[pages, rows].double(), v_pool[pages, rows].double()
        for t in range(new):
            seen = length - new + t + 1 if causal else length
            if seen <= 0:
                continue
            for h in range(hq):
                s = scale * (k[:seen, h // g] @ q[at + t, h])
                w = torch.softmax(s, 0)
                out[at + t, h] = w @ v[:seen, h // g]
                mass[at + t, h] = w @ v[:seen, h // g].abs()
                lse[at + t, h] = torch.logsumexp(s, 0)
                reach[at + t, h] = scale * (k[:seen, h // g].abs() @ q[at + t, h].abs()).max()
        at += new
    return out, lse, mass, reach
