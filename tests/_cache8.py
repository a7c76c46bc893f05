"""Plain 64-bit forms of the block-scaled 8-bit KV cache's operators (torch, any device), written from
the definitions in include/sgqa.h, and the inputs of their tests."""
from __future__ import annotations

import math

import torch

F8 = torch.float8_e4m3fn


def grid(y):
    """y (fp64) on the E4M3 grid: four significant bits, steps of 2^-9 below 2^-6, ties to even, saturating."""
    fin = torch.where(torch.isfinite(y) & (y != 0), y, 1.0)
    e = torch.frexp(fin.abs()).exponent - 1
    step = torch.ldexp(torch.ones_like(y), e.clamp(min=-6) - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def scale_of(amax):
    """The smallest 2^e, e in [-126, 119], with amax <= 448 * 2^e (fp64)."""
    s = torch.exp2(torch.ceil(torch.log2(torch.clamp(amax, min=2.0 ** -140) / 448.0)))
    s = torch.where(s * 448.0 < amax, s * 2, torch.where(s / 2 * 448.0 >= amax, s / 2, s))
    return s.clamp(2.0 ** -126, 2.0 ** 119)


def encode(y):
    """Codes (uint8) of values that lie on the E4M3 grid."""
    return y.float().to(F8).view(torch.uint8)


def decode(codes):
    return codes.view(F8).double()


def ref_append(cache, block, lens, counts, k_new, v_new):
    """A new cache dict with the tokens appended (fp64 arithmetic, codes as uint8)."""
    out = {n: t.clone() for n, t in cache.items()}
    for codes, scale, x in (("k8", "ks", k_new), ("v8", "vs", v_new)):
        for b, (L, m) in enumerate(zip(lens, counts)):
            for j in range(L // block, -(-(L + m) // block) if m else 0):
                u0, u1 = j * block, min((j + 1) * block, L + m)
                a = max(u0, L)
                new = x[b, a - L:u1 - L].double()
                fin = torch.where(torch.isfinite(new), new, 0.0).abs().amax(dim=(0, 2))
                s = scale_of(fin)
                if u0 < L:
                    old = cache[scale][b, j].double()
                    s = torch.maximum(s, old)
                    grown = (s > old)[None, :, None]
                    held = decode(cache[codes][b, u0:L])
                    held = torch.where(grown, grid(held * (old / s)[None, :, None]), held)
                    out[codes][b, u0:L] = torch.where(grown, encode(held), cache[codes][b, u0:L])
                out[codes][b, a:u1] = encode(grid(new / s[None, :, None]))
                out[scale][b, j] = s.float()
    return out


def values(codes, scale, block):
    """fp64 values of a sequence's rows [n, G, d] given scales [>= ceil(n / block), G]."""
    u = torch.arange(codes.shape[0], device=codes.device)
    return decode(codes) * scale.double()[u // block][:, :, None]


def ref_attend(cache, block, lens, q, gate, weight_in=None, weight_out=None):
    """out (fp64), the bound's ingredient sum p |v| * sigmoid, and weight_out (fp64 or None)."""
    batch, n, Hq, d = q.shape
    G = cache["k8"].shape[2]
    R = Hq // G
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    w = None if weight_out is None else weight_out.double().clone()
    for b, L in enumerate(lens):
        if L == 0:
            continue
        k = values(cache["k8"][b, :L], cache["ks"][b], block)
        v = values(cache["v8"][b, :L], cache["vs"][b], block)
        u = torch.arange(L, device=q.device)
        if w is not None:
            old = torch.zeros((G, L), dtype=torch.float64, device=q.device)
            if weight_in is not None:
                old = torch.where(u < L - n, weight_in[b, :, :L].double(), 0.0)
            w[b, :, :L] = old
        for i in range(n):
            m = L - n + i + 1
            if m <= 0:
                continue
            sig = torch.sigmoid(gate[b, i].double())
            for g in range(G):
                h = slice(g * R, (g + 1) * R)
                z = q[b, i, h].double() @ k[:m, g].T / math.sqrt(d)
                p = torch.softmax(z, -1)
                out[b, i, h] = (p @ v[:m, g]) * sig[h]
                mag[b, i, h] = (p @ v[:m, g].abs()) * sig[h]
                if w is not None:
                    w[b, g, :m] += p.sum(0)
    return out, mag, w


def ref_kept(weight, L, keep, recent):
    """Positions that stay of one (sequence, group): weight [T]."""
    if L <= keep:
        return torch.arange(L, device=weight.device)
    N = L - recent
    w = weight[:N].double()
    w = torch.where(torch.isnan(w), -math.inf, w)
    top = torch.sort(w, descending=True, stable=True).indices[:keep - recent]
    return torch.sort(torch.cat([top, torch.arange(N, L, device=weight.device)])).values


def ref_evict(cache, block, lens, keep, recent, weight, dst):
    """dst: the cache, weight_out, kept and lens_out buffers before the call (a dict); returns them after."""
    out = {n: t.clone() for n, t in dst.items()}
    G = weight.shape[1]
    out["kept"].fill_(-1)
    for b, L in enumerate(lens):
        m = min(L, keep)
        out["lens_out"][b] = m
        for g in range(G):
            rows = ref_kept(weight[b, g], L, keep, recent)
            out["kept"][b, g, :m] = rows.int()
            out["w"][b, g, :m] = weight[b, g][rows]
            for codes, scale in (("k8", "ks"), ("v8", "vs")):
                for j in range(-(-m // block)):
                    r = rows[j * block:min((j + 1) * block, m)]
                    c = cache[codes][b, r, g]
                    s_old = cache[scale][b, :, g].double()[r // block]
                    x = decode(c) * s_old[:, None]
                    s = scale_of(torch.where(torch.isnan(x), 0.0, x).abs().amax())
                    same = (s_old == s)[:, None]
                    out[codes][b, j * block:j * block + len(r), g] = torch.where(same, c, encode(grid(x / s)))
                    out[scale][b, j, g] = s.float()
    return out


def empty_cache(batch, T, G, d, block, device="cuda", code=0x7F, scale=math.nan):
    """A cache of buffers that nothing was stored in: NaN codes and NaN scales."""
    nb = -(-T // block)
    c = {n: torch.full((batch, T, G, d), code, dtype=torch.uint8, device=device) for n in ("k8", "v8")}
    c.update({n: torch.full((batch, nb, G), scale, dtype=torch.float32, device=device) for n in ("ks", "vs")})
    return c


def tokens(gen, batch, n, G, d, spread=1.0):
    """bf16 rows with sizes that differ from token to token by about 2^spread."""
    x = torch.randn((batch, n, G, d), generator=gen)
    return (x * torch.exp2(torch.randn((batch, n, G, 1), generator=gen) * spread)).bfloat16()


def filled_cache(gen, lens, T, G, d, block, spread=1.0):
    """A CPU cache filled at once with lens[b] tokens of every sequence, by the plain form."""
    n = max(max(lens), 1)
    k, v = tokens(gen, len(lens), n, G, d, spread), tokens(gen, len(lens), n, G, d, spread)
    c = empty_cache(len(lens), T, G, d, block, device="cpu")
    return ref_append(c, block, [0] * len(lens), lens, k, v)


def to_cuda(d):
    return {n: t.cuda() for n, t in d.items()}
