"""The draft-check operators in 64 bits, written from their definitions with
plain loops over requests (no code of the library), and error bounds."""
import math

import torch

F64 = torch.float64


def scale_of(byte):
    x = torch.exp2(byte.to(F64) - 127)
    return torch.where(byte == 255, torch.full_like(x, math.nan), x)


def cached(x, scale, pages, page_size, lo, hi):
    """Positions lo .. hi-1 of one request: float64 [n, heads, dim]."""
    at = torch.arange(lo, hi, device=x.device)
    p, s = pages[at // page_size].long(), at % page_size
    y = x[p, s].to(F64)
    return y if scale is None else y * scale_of(scale[p, s])[..., None]


def quantise(x):
    """Codes (float64 values on the e4m3 grid) and scale bytes of rows [..., dim]."""
    x = x.to(F64)
    a = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    safe = torch.where(bad | (a == 0), torch.ones_like(a), a)
    e = torch.ceil(torch.log2(safe / 448))
    # log2 rounds: settle the two neighbours by the definition itself
    e = torch.where(safe <= 448 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(safe > 448 * torch.exp2(e), e + 1, e).clamp(-127, 127)
    e = torch.where(a == 0, torch.full_like(e, -127), e)
    y = x * torch.exp2(-e)[..., None]
    grid = torch.tensor([m / 8 * 2.0 ** -6 for m in range(8)] +
                        [(1 + m / 8) * 2.0 ** (b - 7) for b in range(1, 16) for m in range(8)][:-1],
                        dtype=F64, device=x.device)
    mag = torch.nan_to_num(y.abs(), nan=0.0, posinf=448.0)
    hi = torch.searchsorted(grid, mag).clamp(1, len(grid) - 1)
    up, down = grid[hi] - mag, mag - grid[hi - 1]
    code = torch.where((down < up) | ((down == up) & ((hi - 1) % 2 == 0)), grid[hi - 1], grid[hi])
    code = torch.copysign(code, y)
    code = torch.where(bad[..., None], torch.full_like(code, math.nan), code)
    byte = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return code, byte


def attend(q, k, v, ks, vs, pages, page_size, length, first, mask, scale, softcap):
    """(out, lse, weight, sums): float64 results, and for the error bound the rows'
    sum_j p_j |v_j| and the largest sum |q| |k| scale over their visible keys."""
    N, Hq, D = q.shape
    G = Hq // k.shape[2]
    out = torch.full((N, Hq, D), math.nan, dtype=F64, device=q.device)
    lse = torch.full((N, Hq), math.nan, dtype=F64, device=q.device)
    weight, sums = torch.zeros_like(out), torch.zeros_like(lse)
    length, first = length.tolist(), first.tolist()
    for b, n in enumerate(length):
        r0, t = first[b], first[b + 1] - first[b]
        if t == 0:
            continue
        kk = cached(k, ks, pages[b], page_size, 0, n + t)
        vv = cached(v, vs, pages[b], page_size, 0, n + t)
        for i in range(t):
            if mask is None:
                vis = list(range(n + i + 1))
            else:
                words = [int(w) & 0xffffffff for w in mask[r0 + i].tolist()]
                vis = list(range(n)) + [n + j for j in range(t) if words[j // 32] >> (j % 32) & 1]
            if not vis:
                out[r0 + i], lse[r0 + i] = 0.0, -math.inf
                continue
            vis = torch.tensor(vis, device=q.device)
            kv, vvv = kk[vis].transpose(0, 1), vv[vis].transpose(0, 1)       # [Hkv, n, D]
            kv, vvv = kv.repeat_interleave(G, 0), vvv.repeat_interleave(G, 0)
            qq = q[r0 + i].to(F64)
            s = torch.einsum("hd,hnd->hn", qq, kv) * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            p = torch.softmax(s, 1)
            out[r0 + i] = torch.einsum("hn,hnd->hd", p, vvv)
            lse[r0 + i] = torch.logsumexp(s, 1)
            weight[r0 + i] = torch.einsum("hn,hnd->hd", p, vvv.abs())
            sums[r0 + i] = torch.einsum("hd,hnd->hn", qq.abs(), kv.abs()).amax(1) * abs(scale)
    return out, lse, weight, sums


def bounds(out, weight, sums, D, dtype, softcap):
    """What out and lse may be off by, from the formats alone.

    A score: D products added in 32 bits, each addition within 2^-23 (it may
    truncate); the cap adds 2^-21 of it.  A weight e^(s - m): the score's error
    twice (s and m), 2^-21 of the exponential and 2^-22 of its argument; then
    one rounding of the weight to the 16-bit type (half a unit) and one of the
    result."""
    half = torch.finfo(dtype).eps / 2
    score = (D + 4) * 2.0 ** -23 * sums + (softcap or 0.0) * 2.0 ** -21
    top = torch.clamp(sums, max=softcap) if softcap else sums
    p = 2 * score + 2.0 ** -21 + 2.0 ** -22 * top
    tiny = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -120
    tol_out = half * out.abs() + (half * (1 + 2.0 ** -7) + p)[..., None] * weight + tiny
    return tol_out, score + p + 2.0 ** -21
