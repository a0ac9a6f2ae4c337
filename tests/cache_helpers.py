"""Plain 64-bit forms of the cache operators, on the CPU, for their tests."""
from __future__ import annotations

import math

import torch

PAGE, DV, ROPE, FP8_ROW = 64, 512, 64, 656
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.bfloat16}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # relative, of a rounding to nearest


def rotation_table(n: int, seed: int = 0) -> torch.Tensor:
    half = torch.arange(ROPE // 2, dtype=torch.float64)
    angle = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-half / (ROPE // 2))
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def rotate64(x, cs, interleaved):
    """Rotated columns of x [..., 64] (float64) by cs [..., 64], and per column |a| + |b| of its pair."""
    x = x.double()
    cos, sin = cs[..., :32].double(), cs[..., 32:].double()
    out, size = torch.empty_like(x), torch.empty_like(x)
    for i in range(32):
        i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        a, b = x[..., i0], x[..., i1]
        out[..., i0] = a * cos[..., i] - b * sin[..., i]
        out[..., i1] = b * cos[..., i] + a * sin[..., i]
        size[..., i0] = size[..., i1] = a.abs() + b.abs()
    return out, size


def norm64(x, weight, eps):
    x = x.double()
    if weight is None:
        return x
    return x / torch.sqrt(x.square().sum(-1, keepdim=True) / DV + eps) * weight.double()


def fp8_parts(cache):
    """(codes as values, scales, position columns) of FP8 rows, as float64 on the CPU."""
    c = cache.cpu().reshape(-1, FP8_ROW)
    return (c[:, :DV].contiguous().view(torch.float8_e4m3fn).float().double(),
            c[:, DV:DV + 16].contiguous().view(torch.float32).double(),
            c[:, DV + 16:].contiguous().view(torch.bfloat16).double())


def cache_rows64(cache, fp8: bool):
    """A cache's rows as attention reads them: float64 [rows, d]."""
    if not fp8:
        return cache.cpu().double().reshape(-1, cache.shape[-1])
    codes, scale, rope = fp8_parts(cache)
    lat = (codes.float() * scale.float().repeat_interleave(128, 1)).bfloat16().double()
    return torch.cat([lat, rope], 1)


def random_cache(kind: str, pages: int, d: int = 576, seed: int = 0):
    """A cache of random finite rows (CPU)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(pages * PAGE, d, generator=g)
    if kind != "fp8":
        return x.to(DTYPES[kind]).view(pages, PAGE, 1, d)
    rows = torch.zeros(pages * PAGE, FP8_ROW, dtype=torch.uint8)
    blocks = x[:, :DV].reshape(-1, 4, 128)
    scale = blocks.abs().amax(-1, keepdim=True) / 448
    rows[:, :DV] = (blocks / scale).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1, DV)
    rows[:, DV:DV + 16] = scale.reshape(-1, 4).contiguous().view(torch.uint8)
    rows[:, DV + 16:] = x[:, DV:].bfloat16().contiguous().view(torch.uint8)
    return rows.view(pages, PAGE, 1, FP8_ROW)


def table_of(lengths, seed: int = 0, extra: int = 1, width: int | None = None):
    """(block table of shuffled pages, -1 past a request's pages; number of pages)."""
    need = [-(-n // PAGE) for n in lengths]
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(sum(need) + extra, generator=g).to(torch.int32)
    table = torch.full((len(lengths), max(width or 0, max(need, default=0), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need) + extra


def request_rows(rows64, table, b: int, length: int):
    i = torch.arange(length)
    return rows64[table[b].long()[i // PAGE] * PAGE + i % PAGE]


def attend64(q, kv, n_vis, scale):
    """(o, lse) of query rows q [r, d] over the first n_vis[r] rows of kv, in 64 bits."""
    o = torch.zeros(q.shape[0], DV, dtype=torch.float64)
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    x = q.double() @ kv.T * scale
    hidden = torch.arange(kv.shape[0])[None] >= n_vis[:, None]
    x = x.masked_fill(hidden, -math.inf)
    some = n_vis > 0
    if some.any():
        lse[some] = torch.logsumexp(x[some], -1)
        o[some] = torch.softmax(x[some], -1) @ kv[:, :DV]
    return o, lse
