"""Attention over the block-scaled 8-bit KV cache where the sizes of V differ inside a tile, against the
64-bit form with a bound of its own for every element.

A row of a tile of 128 tokens (counted from the sequence's first) holds p_u t_u (p the probability, t the
scale of the token's V block) as two E4M3 terms of y = 448 p_u t_u / r. The reference r is at most 16 times
the row's own largest p_u t_u of that tile: 2 times it where the tile's scales differ by more than 2^4 (an
exponent rounded up), else the row's largest p by the tile's largest t. What an element may be off by:
  * a token's p_u t_u by 1/289 of itself (each term at most 1/17 of what it rounds) and 2^-11 of it (fp16
    before them): below 2^-8 + 2^-14; where the terms are subnormal, by half of the second's step 2^-9,
    which counts 1/28: 2^-10 / (28 * 448) r < 2^-23.6 * 16 of the row's largest = 2^-19.6. Times |code_u|,
    summed over the tokens;
  * probabilities below 2^-126 of their tile's largest count nothing (fp32): 2^-126 of that times t |code|
    each; tiles whose largest p t is below 2^-126 of the row's neither: 2^-100 of the row's covers them;
  * the scores: |q| <= 6 and sum |k| <= 1000 put a base-2 exponent off by less than 2^-11.9 from the split
    of q and fp32 (as in test_gpu_cache8.py): 2^-11 of sum p |v| from numerator and denominator together;
    rows that q was made to fit have scores `big` times as large and get `big` times that;
  * the output's own rounding, 2^-8 of its value, and 2^-133 (half of bf16's least step).
"""
import math

import pytest

torch = pytest.importorskip("torch")

import block_sparse_long_kbar_b200 as sg
from tests import _cache8 as c8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attend(c, block, lens, q, gate, **kw):
    batch, n, Hq, d = q.shape
    T, G = c["k8"].shape[1:3]
    dm = sg.sgqa_dims(batch, T, Hq, G, d, 64, 8, 512)
    ws = sg.alloc_workspace(sg.sgqa_cache8_workspace_size(dm, block, n))
    ws[256:].fill_(0xFF)
    out = torch.full_like(q, math.nan)
    sg.sgqa_cache8_attend(dm, block, i32(lens), n, q, gate, c["k8"], c["ks"], c["v8"], c["vs"], out, ws, **kw)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0
    return out


def reference(c, block, lens, q, gate, big=1.0):
    """The 64-bit form and what each of its elements may be off by."""
    batch, n, Hq, d = q.shape
    G = c["k8"].shape[2]
    R = Hq // G
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.full_like(out, 2.0 ** -133)
    for b, L in enumerate(lens):
        k = c8.values(c["k8"][b, :L], c["ks"][b], block)
        t = c["vs"][b].double()[torch.arange(L, device=q.device) // block]  # [L, G]
        code = c8.decode(c["v8"][b, :L])
        for i in range(n):
            m = L - n + i + 1
            if m <= 0:
                continue
            sig = torch.sigmoid(gate[b, i].double())
            for g in range(G):
                h = slice(g * R, (g + 1) * R)
                z = q[b, i, h].double() @ k[:m, g].T / math.sqrt(d)
                pt = torch.softmax(z, -1) * t[:m, g]  # [R, m]
                a = code[:m, g].abs()
                tiles = -(-m // 128)
                of_tile = lambda x: torch.nn.functional.pad(x, (0, tiles * 128 - m)).view(R, tiles, 128).amax(-1)
                step = of_tile(pt).repeat_interleave(128, 1)[:, :m] * 2.0 ** -19.6
                none = of_tile(pt / t[:m, g]).repeat_interleave(128, 1)[:, :m] * t[:m, g] * 2.0 ** -126
                o = (pt @ code[:m, g]) * sig[h]
                e = (pt * (2.0 ** -8 + 2.0 ** -14 + big * 2.0 ** -11) + step + none) @ a + 2.0 ** -100 * pt.amax(-1, True)
                out[b, i, h] = o
                tol[b, i, h] += e * sig[h] + o.abs() * 2.0 ** -8
    return out, tol


def check(c, block, lens, q, gate, big=1.0):
    ref, tol = reference(c, block, lens, q, gate, big)
    got = attend(c, block, lens, q, gate)
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (float((err / tol).nan_to_num(nan=math.inf).max()), int(bad.sum()), bad.nonzero()[:4].tolist())
    return got, ref, tol


def queries(gen, batch, n, Hq, d):
    return (torch.randn(batch, n, Hq, d, generator=gen).clamp(-6, 6).bfloat16().cuda(),
            torch.randn(batch, n, Hq, d, generator=gen).bfloat16().cuda())


def filled(k, v, T, block):
    batch, L, G, d = k.shape
    c = c8.empty_cache(batch, T, G, d, block, device="cpu")
    return c8.to_cuda(c8.ref_append(c, block, [0] * batch, [L] * batch, k, v))


@pytest.mark.parametrize("d,R", [(64, 4), (64, 12), (128, 4), (128, 16)])
@pytest.mark.parametrize("down", [5, 12, 17, 24, 30, 60, 90])
def test_the_heaviest_token_has_the_smallest_value(d, R, down):
    """A token that takes nearly all attention, with a V block 2^-down of its tile's others."""
    gen = torch.Generator().manual_seed(d + R + down)
    L, G, block = 200, 1, 8
    k, v = c8.tokens(gen, 1, L, G, d, 0.0), c8.tokens(gen, 1, L, G, d, 0.0)
    q, gate = queries(gen, 1, 1, R, d)
    q = (q[:, :, :1] + q * 0.125).bfloat16()  # rows alike, so that one token is the heaviest of all
    x = q[0, 0, 0].float().cpu()
    k[0, 3, 0] = (x * (1.45 * (down + 40) * math.sqrt(d) / float(x @ x))).bfloat16()
    v[0, :8] *= 2.0 ** -down
    check(filled(k, v, L, block), block, [L], q, gate, big=(down + 40) / 8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [8, 32])
def test_values_that_only_later_rows_see(d, block):
    """The last tokens' V is 2^40 of the others': what the rows before them see keeps its digits."""
    gen = torch.Generator().manual_seed(d + block)
    lens, G, n = [97, 161, 257], 2, 3  # the last token has a block of its own
    L = max(lens)
    k, v = c8.tokens(gen, 3, L, G, d, 0.0), c8.tokens(gen, 3, L, G, d, 0.0)
    for b, x in enumerate(lens):
        v[b, x - 1:] *= 2.0 ** 40
    q, gate = queries(gen, 3, n, 8, d)
    check(filled(k, v, L, block), block, lens, q, gate)


@pytest.mark.parametrize("batch,L", [(1, 700), (160, 300)])
@pytest.mark.parametrize("d,R,n", [(64, 8, 1), (128, 4, 1), (128, 16, 4), (128, 8, 4)])
def test_scales_far_apart_from_tile_to_tile(batch, L, d, R, n):
    """Tiles, and blocks within them, at both ends of the scales: an early one near the largest with next to
    no attention, the rest 2^-100 and less of it; a CTA has one tile of them or several."""
    gen = torch.Generator().manual_seed(batch + d + R)
    G, block = 1, 32
    k, v = c8.tokens(gen, batch, L, G, d, 0.0), c8.tokens(gen, batch, L, G, d, 0.0)
    x = torch.randn(1, 1, 1, d, generator=gen)
    q = (x + 0.25 * torch.randn(batch, n, R, d, generator=gen)).clamp(-6, 6).bfloat16().cuda()
    gate = torch.randn(batch, n, R, d, generator=gen).bfloat16().cuda()
    u = x[0, 0, 0]
    away = (-150 * math.sqrt(d) / float(u @ u)) * u
    k[:, :128, 0] = (0.1 * k[:, :128, 0].float() + away).bfloat16()
    c = filled(k, v, L, block)
    for j in range(c["vs"].shape[1]):
        c["vs"][:, j] = 2.0 ** (110 if j < 4 else -20 - 13 * (j % 5))
    check(c, block, [L] * batch, q, gate, big=12.0)


@pytest.mark.parametrize("d,R,n", [(64, 2, 2), (128, 4, 4), (128, 16, 1), (64, 16, 2)])
def test_blocks_of_many_sizes(d, R, n):
    gen = torch.Generator().manual_seed(d + R)
    lens, G, block = [513, 90, 128, 1], 2, 8
    c = c8.to_cuda(c8.filled_cache(gen, lens, 520, G, d, block))
    q, gate = queries(gen, 4, n, G * R, d)
    for spread in (1, 3, 10, 30):
        s = {**c, "vs": c["vs"].clone()}
        for j in range(s["vs"].shape[1]):
            s["vs"][:, j] *= 2.0 ** (spread * (j * 7 % 5 - 2))
        check(s, block, lens, q, gate)


def test_alone_and_in_a_batch():
    """A sequence by itself and among others: the same within both calls' bounds (bits may differ, since the
    tiles of all sequences are cut into equal pieces)."""
    gen = torch.Generator().manual_seed(14)
    lens, G, d, block, T = [3000, 17, 901, 1400], 2, 128, 64, 3001
    c = c8.to_cuda(c8.filled_cache(gen, lens, T, G, d, block))
    q, gate = queries(gen, 4, 2, 16, d)
    got, _, tol = check(c, block, lens, q, gate)
    for b, L in enumerate(lens):
        one = {n: t[b:b + 1].clone() for n, t in c.items()}
        alone = attend(one, block, [L], q[b:b + 1].clone(), gate[b:b + 1].clone())
        assert bool(((alone.double() - got[b:b + 1].double()).abs() <= 2 * tol[b:b + 1]).all())
        again = attend(one, block, [L], q[b:b + 1].clone(), gate[b:b + 1].clone())
        assert torch.equal(alone, again)
