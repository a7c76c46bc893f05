"""The block-scaled 8-bit KV cache on the GPU (sgqa_cache8_append, _attend, _evict) against the plain
64-bit forms of tests/_cache8.py.

Tolerances. Codes, scales, positions and moved weights are compared exactly. An output element is
off by at most
  * the rounding of the probabilities to two E4M3 terms. Rounding to four significant bits is off by
    at most 1/17 of a value (half a step of 1/8 at 17/16), so the two by 1/289 of p; the fp16 step
    before them by 2^-11 of it: together below 2^-8 + 2^-14 of p and hence of sum p |v|. Where the terms
    are subnormal: the second is 28 times the first's rest and its half step 2^-10, with 448 for the
    largest p v-scale, so 2^-10 / (28 * 448) = 2^-23.6 of that; over a tile's 128 tokens 2^-16 of the
    largest |v|;
  * the scores' error: q as two E4M3 terms keeps 2^-22 of its row's largest element and products are
    summed in fp32, so with |q| <= 6 and sum |k| <= 1000 a base-2 exponent is off by less than
    2^-22 * 6 * 1000 * log2(e) / 8 < 2^-11.9, and by 2^-24 of itself from fp32; numerator and denominator
    by 0.7 times that each in relative terms: with the 2^-14 above below 2^-11;
  * the output's own rounding, 2^-8 of its value (bf16).
A received weight is a sum of fp32 probabilities: each off by 2^-11 of itself at most by the same bound,
and 2^-24 of the total by each fp32 addition (at most 66 of them).
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


def dims(batch, T, Hq, G, d):
    return sg.sgqa_dims(batch, T, Hq, G, d, 64, 8, 512)


def workspace(dm, block, n_new=1):
    ws = sg.alloc_workspace(sg.sgqa_cache8_workspace_size(dm, block, n_new))
    ws[256:].fill_(0xFF)  # all but the status word: whatever was in the memory
    return ws


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache_args(c):
    return c["k8"], c["ks"], c["v8"], c["vs"]


def same(a, b):
    """Equal, NaN where NaN."""
    if a.dtype.is_floating_point:
        return torch.equal(torch.nan_to_num(a, nan=12345.0), torch.nan_to_num(b, nan=12345.0))
    return torch.equal(a, b)


def run_append(cache, block, lens, k, v, counts=None):
    batch, n_t, G, d = k.shape
    T = cache["k8"].shape[1]
    dm = dims(batch, T, G, G, d)
    ws = workspace(dm, block)
    sg.sgqa_cache8_append(dm, block, i32(lens), n_t, k, v, *cache_args(cache), ws,
                          counts=None if counts is None else i32(counts))
    torch.cuda.synchronize()
    return sg.sgqa_get_device_status(ws)


def check_append(cache_cpu, block, lens, counts, k, v):
    want = c8.ref_append(cache_cpu, block, lens, counts, k, v)
    got = c8.to_cuda(cache_cpu)
    ragged = any(m != k.shape[1] for m in counts)
    for _ in range(2):  # repeating an append gives the same bits
        assert run_append(got, block, lens, k.cuda(), v.cuda(), counts if ragged else None) == 0
        for n in want:
            assert same(got[n].cpu(), want[n]), n
    return want


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [8, 16, 32, 64, 128])
def test_append(d, block):
    gen = torch.Generator().manual_seed(block + d)
    lens, counts, n_t, G, T = [0, 1, block - 1, block, 130, 261], [300, 17, 1, 0, 299, 39], 300, 4, 501
    c = c8.filled_cache(gen, lens, T, G, d, block)
    k, v = c8.tokens(gen, 6, n_t, G, d), c8.tokens(gen, 6, n_t, G, d, 3.0)
    check_append(c, block, lens, counts, k, v)


@pytest.mark.parametrize("n_t", [1, 4, 7])
def test_append_step_by_step_grows_blocks(n_t):
    gen = torch.Generator().manual_seed(n_t)
    G, d, block, T, lens = 1, 128, 32, 96, [0, 30, 31]
    c = c8.filled_cache(gen, lens, T, G, d, block, spread=0.0)
    for step in range(8):
        k, v = c8.tokens(gen, 3, n_t, G, d, 2.0), c8.tokens(gen, 3, n_t, G, d, 2.0) * 2.0 ** (step - 4)
        c = check_append(c, block, lens, [n_t] * 3, k, v.bfloat16())
        lens = [x + n_t for x in lens]


def test_append_to_the_last_row_and_into_one_block():
    gen = torch.Generator().manual_seed(3)
    c = c8.filled_cache(gen, [45, 0], 50, 2, 64, 64)
    check_append(c, 64, [45, 0], [5, 5], c8.tokens(gen, 2, 5, 2, 64), c8.tokens(gen, 2, 5, 2, 64))


def test_append_special_values():
    gen = torch.Generator().manual_seed(4)
    k, v = c8.tokens(gen, 1, 40, 1, 64), c8.tokens(gen, 1, 40, 1, 64)
    k[0, 3, 0, 5] = math.inf
    k[0, 4, 0, 6] = -math.inf
    k[0, 5, 0, 7] = math.nan
    k[0, 8:16] = 0.0                       # a block of zeros
    k[0, 16:24] *= 2.0 ** -126             # bf16 subnormals
    k[0, 24:32] *= 2.0 ** 124
    k[0, 33] = 2.0 ** -60                  # far below its block's step
    v[0, 0] = math.nan                     # a row of NaN does not touch its neighbours
    v[0, 8:16] = math.nan
    check_append(c8.empty_cache(1, 64, 1, 64, 8, device="cpu"), 8, [0], [40], k, v)
    check_append(c8.empty_cache(1, 64, 1, 64, 64, device="cpu"), 64, [0], [40], k, v)


def test_append_refuses_lengths_that_do_not_fit():
    gen = torch.Generator().manual_seed(5)
    G, d, block, T = 2, 128, 16, 64
    c = c8.to_cuda(c8.filled_cache(gen, [10] * 5, T, G, d, block))
    before = {n: t.clone() for n, t in c.items()}
    k, v = c8.tokens(gen, 5, 4, G, d).cuda(), c8.tokens(gen, 5, 4, G, d).cuda()
    assert run_append(c, block, [-1, 61, 10, 2 ** 31 - 2, 10], k, v, [4, 4, 5, 4, -1]) == 6
    for n in before:
        assert same(c[n], before[n])
    assert run_append(c, block, [-1, 10, 10, 10, 10], k, v) == 6  # the others are appended
    want = c8.ref_append({n: t.cpu() for n, t in before.items()}, block, [10] * 5, [0, 4, 4, 4, 4], k.cpu(), v.cpu())
    for n in want:
        assert same(c[n].cpu(), want[n])


# ---- attend ----------------------------------------------------------------------------------------
def close(got, ref, mag, vmax, extra=0.0):
    err = (got.double() - ref).abs()
    tol = mag * (2.0 ** -8 + 2.0 ** -11 + extra) + ref.abs() * 2.0 ** -8 + 2.0 ** -16 * vmax + 1e-30
    bad = err > tol
    assert not bool(bad.any()) and bool(torch.isfinite(got).all()), (float((err / tol).max()), int(bad.sum()))


def close_weight(got, want, lens, batch_rows, untouched):
    for b, L in enumerate(lens):
        w, g = want[b, :, :L], got[b, :, :L].double()
        assert bool(((g - w).abs() <= 2.0 ** -11 * w.clamp(max=batch_rows) + 66 * 2.0 ** -24 * w).all())
        assert same(got[b, :, L:], untouched[b, :, L:])


def check_attend(cache, block, lens, q, gate, weight=True, w_in=None, alias=False, extra=0.0):
    batch, n, Hq, d = q.shape
    T, G = cache["k8"].shape[1:3]
    dm = dims(batch, T, Hq, G, d)
    ws = workspace(dm, block, n)
    out = torch.full_like(q, math.nan)
    w_out = torch.full((batch, G, T), -7.0, device="cuda") if weight else None
    w_ref_in = None if w_in is None else w_in.clone()
    if alias:
        w_out = w_in
    untouched = None if w_out is None else w_out.clone()
    ref, mag, w = c8.ref_attend(cache, block, lens, q, gate, w_ref_in, w_out)
    sg.sgqa_cache8_attend(dm, block, i32(lens), n, q, gate, *cache_args(cache), out, ws, weight_in=w_in, weight_out=w_out)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0
    vmax = max([float(c8.values(cache["v8"][b, :L], cache["vs"][b], block).abs().max()) for b, L in enumerate(lens) if L] + [0.0])
    close(out, ref, mag, vmax, extra)
    if weight:
        close_weight(w_out, w, lens, n * Hq // G, untouched)
    return out, w_out


def queries(gen, batch, n, Hq, d, size=1.0):
    return ((torch.randn(batch, n, Hq, d, generator=gen) * size).bfloat16().cuda(),
            torch.randn(batch, n, Hq, d, generator=gen).bfloat16().cuda())


LENS = [0, 1, 2, 5, 127, 128, 129, 255, 256, 257, 383, 700]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("R,n_new", [(1, 1), (1, 3), (2, 2), (3, 5), (8, 1), (8, 4), (5, 12), (16, 4), (1, 64)])
def test_attend(d, R, n_new):
    gen = torch.Generator().manual_seed(100 * R + n_new + d)
    G, block = 2, (8, 16, 32, 64, 128)[(R + n_new) % 5]
    c = c8.to_cuda(c8.filled_cache(gen, LENS, 701, G, d, block))
    q, gate = queries(gen, len(LENS), n_new, G * R, d)
    w_in = torch.rand((len(LENS), G, 701), generator=gen).cuda() * 3
    check_attend(c, block, LENS, q, gate, True, w_in)
    check_attend(c, block, LENS, q, gate, False)


@pytest.mark.parametrize("block", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_attend_blocks_and_groups(block, G):
    gen = torch.Generator().manual_seed(block * G)
    lens = [block - 1, block, block + 1, 333]
    c = c8.to_cuda(c8.filled_cache(gen, lens, 333, G, 128, block, spread=2.0))
    q, gate = queries(gen, 4, 2, 4 * G, 128)
    check_attend(c, block, lens, q, gate)


def test_attend_weight_in_place_and_without_a_past():
    gen = torch.Generator().manual_seed(9)
    lens = [300, 4, 0, 2]
    c = c8.to_cuda(c8.filled_cache(gen, lens, 310, 2, 128, 32))
    q, gate = queries(gen, 4, 4, 16, 128)
    w = torch.rand((4, 2, 310), generator=gen).cuda()
    check_attend(c, 32, lens, q, gate, True, w, alias=True)
    check_attend(c, 32, lens, q, gate, True, None)


def test_attend_nan_behind_the_last_token_and_in_masked_ones():
    gen = torch.Generator().manual_seed(10)
    lens, G, d, block, T = [130, 40], 2, 128, 16, 200
    c = c8.filled_cache(gen, lens, T, G, d, block)
    clean = c8.to_cuda(c)
    q, gate = queries(gen, 2, 3, 8, d)
    base, _ = check_attend(clean, block, lens, q, gate, False)
    # the last token is NaN in a K dim of group 0 and in a V dim of group 1: only the last query sees it
    for b, L in enumerate(lens):
        c["k8"][b, L - 1, 0, 7] = 0x7F
        c["v8"][b, L - 1, 1, 9] = 0xFF
    c = c8.to_cuda(c)
    dm = dims(2, T, 8, G, d)
    ws, out = workspace(dm, block, 3), torch.zeros_like(q)
    sg.sgqa_cache8_attend(dm, block, i32(lens), 3, q, gate, *cache_args(c), out, ws)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0
    assert torch.equal(out[:, :2], base[:, :2])
    assert bool(torch.isnan(out[:, 2, :4]).all()), "every dim of a row with a NaN score"
    assert bool(torch.isnan(out[:, 2, 4:, 9]).all()), "the NaN dim of V"
    others = torch.arange(d, device="cuda") != 9
    assert torch.equal(out[:, 2, 4:][..., others], base[:, 2, 4:][..., others])


def test_attend_sharp_and_flat_rows():
    """Scores of hundreds (one token takes all) and of zero (all take the same), scales far apart."""
    gen = torch.Generator().manual_seed(11)
    lens, G, d, block = [513, 90], 2, 128, 32
    c = c8.filled_cache(gen, lens, 520, G, d, block)
    q, gate = queries(gen, 2, 2, 8, d, size=0.0)
    check_attend(c8.to_cuda(c), block, lens, q, gate)
    # with |q| up to 200 the exponents' error bound grows by 200 / 6: 2^-11 * 34 < 2^-5
    q, gate = queries(gen, 2, 2, 8, d, size=40.0)
    check_attend(c8.to_cuda(c), block, lens, q, gate, False, extra=2.0 ** -5)
    # V blocks whose sizes differ by 2^40 inside a tile, K blocks by 2^12
    for j in range(c["vs"].shape[1]):
        c["vs"][:, j] *= 2.0 ** (10 * (j % 5) - 20)
        c["ks"][:, j] *= 2.0 ** (-3 * (j % 5))
    q, gate = queries(gen, 2, 2, 8, d)
    check_attend(c8.to_cuda(c), block, lens, q, gate)


def test_attend_first_tokens_carry_most_weight_and_least_value():
    """A token that takes nearly all attention with a V block 2^30 smaller than its neighbours'."""
    gen = torch.Generator().manual_seed(12)
    L, G, d, block = 200, 1, 128, 8
    k, v = c8.tokens(gen, 1, L, G, d, 0.0), c8.tokens(gen, 1, L, G, d, 0.0)
    q, gate = queries(gen, 1, 1, 4, d)
    k[0, 0, 0] = (q[0, 0].float().sum(0) * 8).cpu().bfloat16()
    v[0, :8] *= 2.0 ** -30
    c = c8.to_cuda(c8.ref_append(c8.empty_cache(1, L, G, d, block, device="cpu"), block, [0], [L], k, v))
    check_attend(c, block, [L], q, gate, False, extra=2.0 ** -8)


def test_attend_refuses_lengths_that_do_not_fit():
    gen = torch.Generator().manual_seed(13)
    lens, T = [50, 60, 64], 64
    c = c8.to_cuda(c8.filled_cache(gen, lens, T, 2, 64, 16))
    q, gate = queries(gen, 3, 2, 8, 64)
    good, _ = check_attend(c, 16, lens, q, gate, False)
    dm = dims(3, T, 8, 2, 64)
    ws, out = workspace(dm, 16, 2), torch.full_like(q, math.nan)
    w = torch.full((3, 2, T), -1.0, device="cuda")
    sg.sgqa_cache8_attend(dm, 16, i32([-5, 60, 65]), 2, q, gate, *cache_args(c), out, ws, weight_out=w)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 6
    assert bool((out[0] == 0).all()) and bool((out[2] == 0).all()) and torch.equal(out[1], good[1])
    assert bool((w[0] == -1).all()) and bool((w[2] == -1).all()) and bool((w[1, :, :60] >= 0).all())


def test_attend_is_deterministic_and_independent_of_the_batch():
    gen = torch.Generator().manual_seed(14)
    lens, G, d, block, T = [3000, 17, 901], 2, 128, 64, 3001
    c = c8.to_cuda(c8.filled_cache(gen, lens, T, G, d, block))
    q, gate = queries(gen, 3, 2, 16, d)
    outs = [check_attend(c, block, lens, q, gate) for _ in range(3)]
    for o, w in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(w, outs[0][1])


def test_attend_many_sequences():
    gen = torch.Generator().manual_seed(15)
    lens = [int(x) for x in torch.randint(0, 140, (1500,), generator=gen)]
    c = c8.to_cuda(c8.filled_cache(gen, lens, 140, 1, 64, 16))
    q, gate = queries(gen, 1500, 1, 2, 64)
    check_attend(c, 16, lens, q, gate)


@pytest.mark.slow
def test_attend_offsets_beyond_32_bits():
    """8.5 million tokens of four groups: 4.35 GB of K codes and of V codes."""
    T, G, d, block, Hq = 8500003, 4, 128, 128, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    c = {}
    for n in ("k8", "v8"):
        c[n] = torch.randint(0, 256, (1, T, G, d), generator=g, dtype=torch.uint8, device="cuda")
        c[n][(c[n] & 0x7F) == 0x7F] = 0
    for n in ("ks", "vs"):
        c[n] = torch.full((1, -(-T // block), G), 2.0 ** -9, device="cuda")
    q = torch.randn((1, 1, Hq, d), generator=g, device="cuda").bfloat16()
    gate = torch.randn((1, 1, Hq, d), generator=g, device="cuda").bfloat16()
    dm = dims(1, T, Hq, G, d)
    ws, out = workspace(dm, block), torch.zeros_like(q)
    w = torch.zeros((1, G, T), device="cuda")
    sg.sgqa_cache8_attend(dm, block, i32([T]), 1, q, gate, *cache_args(c), out, ws, weight_out=w)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0
    for h in range(G):
        z = torch.cat([(c8.decode(c["k8"][0, a:a + 1000000, h]) * 2.0 ** -9) @ q[0, 0, h].double() for a in range(0, T, 1000000)])
        p = torch.softmax(z / math.sqrt(d), 0)
        o = sum(p[a:a + 1000000] @ (c8.decode(c["v8"][0, a:a + 1000000, h]) * 2.0 ** -9) for a in range(0, T, 1000000))
        m = sum(p[a:a + 1000000] @ (c8.decode(c["v8"][0, a:a + 1000000, h]).abs() * 2.0 ** -9) for a in range(0, T, 1000000))
        sig = torch.sigmoid(gate[0, 0, h].double())
        # 2^-20 of sum p |v| more: a million partial sums in fp32, each off by 2^-24, of random sign
        close(out[0, 0, h], o * sig, m * sig, 448 * 2.0 ** -9 * 2.0 ** -7, extra=2.0 ** -20)
        assert bool(((w[0, h].double() - p).abs() <= 2.0 ** -11 * p + 1e-12).all())


def nan_rows(out, want):
    """Where a plain form gives NaN the kernel does, and nowhere else."""
    assert torch.equal(torch.isnan(out), torch.isnan(want))


@pytest.mark.parametrize("n_new,L", [(64, 130), (64, 64), (40, 300), (64, 257), (17, 9)])
def test_attend_nan_values_over_two_tiles_of_new_tokens(n_new, L):
    """NaN V codes among the new tokens: the rows before them are as without, those that see one are NaN in its dim."""
    gen = torch.Generator().manual_seed(n_new + L)
    G, d, block = 2, 64, 8
    c = c8.filled_cache(gen, [L, L], L + 3, G, d, block)
    q, gate = queries(gen, 2, n_new, G, d)
    base, _ = check_attend(c8.to_cuda(c), block, [L, L], q, gate, False)
    want = base.clone()
    for b, (u, g, x) in enumerate([(L - 1, 0, 3), (max(0, L - n_new // 2), 1, 63)]):
        c["v8"][b, u, g, x] = 0x7F if b else 0xFF
        c["v8"][b, u, g, 0] = 0x7F
        first = max(0, u - (L - n_new))  # the first row that sees token u
        want[b, first:, g, x] = math.nan
        want[b, first:, g, 0] = math.nan
    dm = dims(2, L + 3, G, G, d)
    ws, out = workspace(dm, block, n_new), torch.zeros_like(q)
    c = c8.to_cuda(c)
    sg.sgqa_cache8_attend(dm, block, i32([L, L]), n_new, q, gate, *cache_args(c), out, ws)
    torch.cuda.synchronize()
    nan_rows(out, want)
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))


@pytest.mark.parametrize("d,R", [(64, 2), (128, 2), (128, 12)])
def test_attend_nan_values_of_many_short_sequences(d, R):
    """Every other of 1800 short sequences has a NaN in the V of its last token, each at its own length and dim."""
    gen = torch.Generator().manual_seed(d + R)
    batch, n, block, T = 1800, 2, 32, 96
    lens = [2 + int(x) for x in torch.randint(0, T - 2, (batch,), generator=gen)]
    c = c8.filled_cache(gen, lens, T, 1, d, block)
    q, gate = queries(gen, batch, n, R, d)
    base, _ = check_attend(c8.to_cuda(c), block, lens, q, gate, False)
    want = base.clone()
    for b in range(0, batch, 2):
        c["v8"][b, lens[b] - 1, 0, (7 * b) % d] = 0x7F
        want[b, 1, :, (7 * b) % d] = math.nan
    c, dm = c8.to_cuda(c), dims(batch, T, R, 1, d)
    ws = workspace(dm, block, n)
    for _ in range(3):
        out = torch.zeros_like(q)
        sg.sgqa_cache8_attend(dm, block, i32(lens), n, q, gate, *cache_args(c), out, ws)
        torch.cuda.synchronize()
        nan_rows(out, want)
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))


@pytest.mark.parametrize("d", [64, 128])
def test_attend_rows_of_nan_and_infinity(d):
    """A query with a NaN or an infinity gives NaN, its neighbours what they give without it."""
    gen = torch.Generator().manual_seed(d)
    lens, G, block = [300, 129], 2, 32
    c = c8.to_cuda(c8.filled_cache(gen, lens, 300, G, d, block))
    q, gate = queries(gen, 2, 2, 16, d)
    base, base_w = check_attend(c, block, lens, q, gate)
    q[0, 1, 3, 5], q[1, 0, 9, d - 1], q[1, 1, 0, 0] = math.nan, math.inf, -math.inf
    dm = dims(2, 300, 16, G, d)
    ws, out, w = workspace(dm, block, 2), torch.zeros_like(q), torch.full((2, G, 300), -7.0, device="cuda")
    sg.sgqa_cache8_attend(dm, block, i32(lens), 2, q, gate, *cache_args(c), out, ws, weight_out=w)
    torch.cuda.synchronize()
    bad = torch.zeros(2, 2, 16, dtype=torch.bool, device="cuda")
    bad[0, 1, 3] = bad[1, 0, 9] = bad[1, 1, 0] = True
    assert bool(torch.isnan(out[bad]).all()) and torch.equal(out[~bad], base[~bad])
    # group 1 of sequence 0 has none of those rows
    assert torch.equal(w[0, 1], base_w[0, 1]) and bool(torch.isnan(w[0, 0, :300]).all())
    # row 0 of sequence 1 does not see the last token
    assert bool(torch.isnan(w[1, 1, :128]).all()) and torch.equal(w[1, 1, 128:], base_w[1, 1, 128:])


def test_attend_extreme_scales():
    """V blocks at both ends of the scales' range, and a token of nearly all weight whose V block is all zero."""
    gen = torch.Generator().manual_seed(16)
    L, G, d, block = 400, 1, 128, 16
    c = c8.filled_cache(gen, [L], L, G, d, block)
    q, gate = queries(gen, 1, 1, 4, d)
    for top in (2.0 ** 119, 2.0 ** -100):
        c["vs"][:] = top
        c["vs"][0, ::3] = 2.0 ** -126
        check_attend(c8.to_cuda(c), block, [L], q, gate)
    k, v = c8.tokens(gen, 1, L, G, d, 0.0), c8.tokens(gen, 1, L, G, d, 0.0)
    k[0, 0, 0] = (q[0, 0].float().sum(0) * 4).cpu().bfloat16()
    v[0, :block] = 0.0
    c = c8.ref_append(c8.empty_cache(1, L, G, d, block, device="cpu"), block, [0], [L], k, v)
    check_attend(c8.to_cuda(c), block, [L], q, gate)


def test_attend_more_rows_than_one_unit_holds_over_many_ctas():
    gen = torch.Generator().manual_seed(17)
    lens, G, block = [6000, 0, 3], 1, 64
    for d, R, n in ((128, 16, 4), (64, 11, 3)):
        c = c8.to_cuda(c8.filled_cache(gen, lens, 6001, G, d, block))
        q, gate = queries(gen, 3, n, G * R, d)
        check_attend(c, block, lens, q, gate)


def test_calls_refuse_tensors_elsewhere():
    gen = torch.Generator().manual_seed(18)
    c = c8.to_cuda(c8.filled_cache(gen, [20], 32, 1, 64, 8))
    dm = dims(1, 32, 1, 1, 64)
    ws, (q, gate) = workspace(dm, 8), queries(gen, 1, 1, 1, 64)
    with pytest.raises(ValueError):
        sg.sgqa_cache8_attend(dm, 8, torch.tensor([20], dtype=torch.int32), 1, q, gate, *cache_args(c), torch.zeros_like(q), ws)
    with pytest.raises(ValueError):
        wide = torch.zeros((1, 1, 1, 128), dtype=torch.bfloat16, device="cuda")
        sg.sgqa_cache8_attend(dm, 8, i32([20]), 1, wide[..., ::2], gate, *cache_args(c), torch.zeros_like(q), ws)
    with pytest.raises(sg.SgqaError):
        sg.sgqa_cache8_attend(dm, 8, i32([20]), 1, q, gate, *cache_args(c), torch.zeros_like(q), ws[256:512])


def test_a_wait_that_runs_out_ends_the_call():
    """One CTA issues no loads (the hook's flag that nothing sets): the call ends with the status recorded,
    the next one stops at once and writes nothing, and after a reset all is as before."""
    gen = torch.Generator().manual_seed(19)
    lens, G, d, block = [900, 500], 2, 128, 32
    c = c8.to_cuda(c8.filled_cache(gen, lens, 900, G, d, block))
    q, gate = queries(gen, 2, 4, 16, d)
    base, base_w = check_attend(c, block, lens, q, gate)
    dm = dims(2, 900, 16, G, d)
    ws = workspace(dm, block, 4)
    out, w = torch.full_like(q, math.nan), torch.full((2, G, 900), -7.0, device="cuda")
    call = lambda: sg.sgqa_cache8_attend(dm, block, i32(lens), 4, q, gate, *cache_args(c), out, ws, weight_out=w)
    sg.sgqa_test_stall_decode_cta(1)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        sg.sgqa_test_stall_decode_cta(-1)
    assert sg.sgqa_get_device_status(ws) == 5
    for _ in range(2):
        call()
        torch.cuda.synchronize()
        assert sg.sgqa_get_device_status(ws) == 5
        assert bool(torch.isnan(out).all()) and bool((w == -7).all())
    sg.sgqa_reset_device_status(ws)
    call()
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0 and torch.equal(out, base) and torch.equal(w, base_w)


# ---- evict -----------------------------------------------------------------------------------------
def run_evict(cache, block, lens, keep, recent, weight, T_out):
    batch, T, G, d = cache["k8"].shape
    dst = c8.empty_cache(batch, T_out, G, d, block, code=0xAB, scale=-3.0)
    dst["w"] = torch.full((batch, G, T_out), -5.0, device="cuda")
    dst["kept"] = torch.full((batch, G, keep), 99, dtype=torch.int32, device="cuda")
    dst["lens_out"] = i32([-9] * batch)
    before = {n: t.clone() for n, t in dst.items()}
    dm = dims(batch, T, G, G, d)
    ws = workspace(dm, block)
    sg.sgqa_cache8_evict(dm, block, i32(lens), keep, recent, T_out, weight, *cache_args(cache), *cache_args(dst), dst["w"],
                         dst["kept"], dst["lens_out"], ws)
    torch.cuda.synchronize()
    return dst, before, sg.sgqa_get_device_status(ws)


def check_evict(cache, block, lens, keep, recent, weight, T_out):
    got, before, status = run_evict(cache, block, lens, keep, recent, weight, T_out)
    assert status == 0
    want = c8.ref_evict({n: t.cpu() for n, t in cache.items()}, block, lens, keep, recent, weight.cpu(),
                        {n: t.cpu() for n, t in before.items()})
    for n in want:
        assert same(got[n].cpu(), want[n]), n


@pytest.mark.parametrize("d,block", [(64, 8), (128, 8), (64, 16), (128, 16), (128, 32), (64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("keep,recent,T_out", [(150, 30, 151), (1, 0, 1), (1, 1, 40), (129, 129, 129), (300, 0, 500)])
def test_evict(d, block, keep, recent, T_out):
    gen = torch.Generator().manual_seed(block + keep)
    lens, G = [0, 1, keep, keep + 1, 401, 77], 2
    c = c8.to_cuda(c8.filled_cache(gen, lens, 403, G, d, block, spread=3.0))
    w = torch.exp2(torch.randn((6, G, 403), generator=gen) * 4)
    w[:, :, ::3] = w[:, :, :1]                                # many equal
    check_evict(c, block, lens, keep, recent, w.cuda(), T_out)


def test_evict_odd_weights():
    gen = torch.Generator().manual_seed(2)
    lens, G, T = [257, 400, 256, 300], 1, 400
    c = c8.to_cuda(c8.filled_cache(gen, lens, T, G, 64, 16, spread=12.0))
    w = torch.randn((4, G, T), generator=gen)
    w[0] = 0.0
    w[0, :, ::2] = -0.0                                       # one value: the lowest positions stay
    w[1, :, 5:200:7] = math.nan
    w[1, :, 6:200:7] = -math.inf
    w[1, :, 7:200:7] = math.inf
    w[2] = math.nan
    w[3] = torch.where(torch.rand((G, T), generator=gen) < 0.5, 1.0, 1.0 + 2.0 ** -23)  # neighbours in fp32
    w[3, :, 10] = 1e-45                                       # subnormal
    check_evict(c, 16, lens, 100, 7, w.cuda(), 100)
    check_evict(c, 16, lens, 255, 0, w.cuda(), 300)


def test_evict_keeps_nan_codes_and_odd_scales():
    gen = torch.Generator().manual_seed(6)
    c = c8.filled_cache(gen, [200], 200, 1, 128, 16)
    c["k8"][0, 3::9, 0, 4] = 0x7F
    c["v8"][0, 5::9, 0] = 0xFF                                # whole rows of NaN
    c["ks"][0, ::3] = 2.0 ** 119
    c["ks"][0, 1::3] = 2.0 ** -126
    c["vs"][0, ::2] *= 2.0 ** 20
    w = torch.rand((1, 1, 200), generator=gen).cuda()
    got, before, status = run_evict(c8.to_cuda(c), 16, [200], 90, 10, w, 90)
    want = c8.ref_evict(c, 16, [200], 90, 10, w.cpu(), {n: t.cpu() for n, t in before.items()})
    assert status == 0
    for n in ("k8", "v8"):  # NaN by NaN (its sign is not kept when a row is rescaled), the rest by code
        a, b = got[n].cpu(), want[n]
        nan = (b & 0x7F) == 0x7F
        assert torch.equal((a & 0x7F) == 0x7F, nan) and torch.equal(a[~nan] & 0x7F, b[~nan] & 0x7F)
        assert torch.equal(c8.decode(a[~nan]), c8.decode(b[~nan]))
    for n in ("ks", "vs", "w", "kept"):
        assert same(got[n].cpu(), want[n]), n


def test_evict_refuses_lengths_that_do_not_fit():
    gen = torch.Generator().manual_seed(7)
    c = c8.to_cuda(c8.filled_cache(gen, [40, 40, 40], 40, 2, 64, 8))
    w = torch.rand((3, 2, 40), generator=gen).cuda()
    got, before, status = run_evict(c, 8, [41, 40, -1], 20, 5, w, 25)
    assert status == 6 and got["lens_out"].tolist() == [0, 20, 0]
    assert bool((got["kept"][0] == -1).all()) and bool((got["kept"][2] == -1).all())
    for n in ("k8", "ks", "v8", "vs", "w"):
        assert same(got[n][0], before[n][0]) and same(got[n][2], before[n][2])


def test_evict_long():
    gen = torch.Generator().manual_seed(8)
    T, lens = 300001, [300001, 70000]
    c = {n: torch.randint(0, 0x7F, (2, T, 1, 64), generator=gen, dtype=torch.uint8).cuda() for n in ("k8", "v8")}
    c.update({n: torch.exp2(torch.randint(-9, -5, (2, -(-T // 32), 1), generator=gen).float()).cuda() for n in ("ks", "vs")})
    w = torch.exp2(torch.randn((2, 1, T), generator=gen) * 3).cuda()
    w[0, 0, 1000:50000] = w[0, 0, 777]
    got, before, status = run_evict(c, 32, lens, 65537, 100, w, 70001)
    assert status == 0
    for b, L in enumerate(lens):
        rows = c8.ref_kept(w[b, 0], L, 65537, 100)
        assert torch.equal(got["kept"][b, 0].long(), rows)
        assert torch.equal(got["w"][b, 0, :65537], w[b, 0][rows])
        for codes, scale in (("k8", "ks"), ("v8", "vs")):
            x = c8.decode(c[codes][b, rows, 0]) * c[scale][b, rows // 32, 0].double()[:, None]
            xb = torch.nn.functional.pad(x, (0, 0, 0, 31)).view(-1, 32, 64)
            s = c8.scale_of(xb.abs().amax(dim=(1, 2)))
            want = (c8.grid(xb / s[:, None, None]) * s[:, None, None]).view(-1, 64)[:65537]
            assert torch.equal(got[scale][b, :len(s), 0].double(), s)
            assert torch.equal(c8.values(got[codes][b, :65537], got[scale][b], 32)[:, 0], want)


def random_codes(gen, batch, T, G, d, block):
    """A cache of random codes, made on the GPU (the ordinary one's plain form is slow)."""
    c = {n: torch.randint(0, 0x7F, (batch, T, G, d), generator=gen, dtype=torch.uint8, device="cuda") for n in ("k8", "v8")}
    c.update({n: torch.exp2(torch.randint(-9, -5, (batch, -(-T // block), G), generator=gen, device="cuda").float())
              for n in ("ks", "vs")})
    return c


def same_eviction(got, c, w, lens, keep, recent, block):
    """Positions, weights and values of an eviction, a (sequence, group) at a time."""
    batch, T, G, d = c["k8"].shape
    for b, L in enumerate(lens):
        for g in range(G):
            rows = c8.ref_kept(w[b, g], L, keep, recent)
            m = len(rows)
            assert torch.equal(got["kept"][b, g, :m].long(), rows) and bool((got["kept"][b, g, m:] == -1).all())
            assert same(got["w"][b, g, :m], w[b, g][rows])
            for codes, scale in (("k8", "ks"), ("v8", "vs")):
                x = c8.decode(c[codes][b, rows, g]) * c[scale][b, rows // block, g].double()[:, None]
                xb = torch.nn.functional.pad(x, (0, 0, 0, -m % block)).view(-1, block, d)
                s = c8.scale_of(xb.abs().amax(dim=(1, 2)))
                assert torch.equal(got[scale][b, :len(s), g].double(), s)
                want = c8.grid(xb / s[:, None, None]).view(-1, d)[:m]
                assert torch.equal(c8.decode(got[codes][b, :m, g]), want)


# one CTA per (sequence, group) with 1, 2, 4 and 8 loads a lane; clusters of 2, 4, 8; of 16; the whole GPU
@pytest.mark.parametrize("batch,G,T,keep,recent", [
    (1, 1, 1, 1, 0), (80, 1, 2041, 500, 0), (60, 2, 4096, 1000, 3), (80, 1, 8191, 4000, 0), (75, 1, 16380, 8000, 100),
    (75, 1, 16381, 700, 1), (1, 2, 5003, 1234, 17), (2, 1, 9002, 8999, 2), (1, 1, 20001, 333, 333), (1, 1, 131071, 60000, 5),
    (5, 2, 140003, 70001, 1000), (3, 1, 131073, 1, 0), (1, 1, 500002, 1000, 0)])
def test_evict_every_selection(batch, G, T, keep, recent):
    gen = torch.Generator(device="cuda").manual_seed(T)
    c = random_codes(gen, batch, T, G, 64, 32)
    w = torch.exp2(torch.randn((batch, G, T), generator=gen, device="cuda") * 3)
    w[:, :, 5:T // 2:3] = 0.75  # many equal, of which some stay
    w[:, :, T // 3:T // 3 + 40] = math.nan
    lens = [T if b % 3 == 0 else T - (b * 37) % (T // 2 + 1) for b in range(batch)]
    got, _, status = run_evict(c, 32, lens, keep, recent, w, keep + 5)
    assert status == 0
    same_eviction(got, c, w, lens, keep, recent, 32)


# many groups; one token; lengths of as many sequences as one warp or one CTA reads, and one more
@pytest.mark.parametrize("batch,G,d,R,n_new,T", [
    (2, 128, 128, 16, 4, 200), (2, 128, 64, 1, 1, 200), (1, 64, 128, 3, 2, 300), (1, 1, 64, 1, 1, 1), (3, 4, 128, 8, 4, 1),
    (256, 2, 64, 4, 2, 150), (257, 1, 128, 8, 4, 130), (512, 1, 128, 4, 1, 140), (513, 2, 64, 1, 1, 129), (641, 1, 64, 2, 1, 150)])
def test_attend_shapes_at_the_limits(batch, G, d, R, n_new, T):
    gen = torch.Generator(device="cuda").manual_seed(batch + G)
    cpu, block = torch.Generator().manual_seed(T), 16
    lens = [int(x) for x in torch.randint(0, T + 1, (batch,), generator=cpu)]
    lens[-1] = T
    c = random_codes(gen, batch, T, G, d, block)
    for n in ("k8", "v8"):
        c[n] = torch.where(c[n] >= 0x50, c[n] & 0x9F | 0x80, c[n])  # both signs, magnitudes below 2
        for b, L in enumerate(lens):
            c[n][b, L:] = 0x7F
    q, gate = queries(cpu, batch, n_new, G * R, d)
    w = torch.rand((batch, G, T), generator=gen, device="cuda")
    check_attend(c, block, lens, q, gate, True, w)


@pytest.mark.parametrize("T,keep", [(3000, 500), (150000, 9000)])
def test_a_captured_eviction_serves_every_length(T, keep):
    gen = torch.Generator(device="cuda").manual_seed(T + 1)
    c = random_codes(gen, 2, T, 1, 64, 64)
    w = torch.rand((2, 1, T), generator=gen, device="cuda")
    dst = c8.empty_cache(2, keep, 1, 64, 64)
    dst.update(w=torch.zeros((2, 1, keep), device="cuda"), kept=torch.zeros((2, 1, keep), dtype=torch.int32, device="cuda"))
    dm, lens, lens_out = dims(2, T, 1, 1, 64), i32([0, 0]), i32([0, 0])
    ws = workspace(dm, 64)
    call = lambda: sg.sgqa_cache8_evict(dm, 64, lens, keep, 7, keep, w, *cache_args(c), *cache_args(dst), dst["w"], dst["kept"],
                                        lens_out, ws)
    call()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call()
    for ls in ([T, keep + 1], [keep, 0], [T - 5, T]):
        lens.copy_(i32(ls))
        w.copy_(torch.rand(w.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert sg.sgqa_get_device_status(ws) == 0 and lens_out.tolist() == [min(x, keep) for x in ls]
        same_eviction(dst, c, w, ls, keep, 7, 64)


# ---- together, streams, graphs ----------------------------------------------------------------------
class Session:
    """A serving session's buffers: prompt, steps with received weights, an eviction, further steps."""

    def __init__(self, batch, T, Hq, G, d, block, n_new):
        self.dm, self.block, self.n_new = dims(batch, T, Hq, G, d), block, n_new
        self.ws = workspace(self.dm, block, n_new)
        self.c = [c8.empty_cache(batch, T, G, d, block) for _ in range(2)]
        self.w = [torch.full((batch, G, T), math.nan, device="cuda") for _ in range(2)]
        self.lens = [torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.k, self.v = (torch.zeros((batch, n_new, G, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.q, self.gate, self.out = (torch.zeros((batch, n_new, Hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(3))
        self.kept = None
        self.at = 0

    def prompt(self, k, v, counts):
        sg.sgqa_cache8_append(self.dm, self.block, self.lens[self.at], k.shape[1], k, v, *cache_args(self.c[self.at]), self.ws,
                              counts=counts)
        self.lens[self.at] += counts

    def step(self):
        a = self.at
        sg.sgqa_cache8_append(self.dm, self.block, self.lens[a], self.n_new, self.k, self.v, *cache_args(self.c[a]), self.ws)
        self.lens[a] += self.n_new
        sg.sgqa_cache8_attend(self.dm, self.block, self.lens[a], self.n_new, self.q, self.gate, *cache_args(self.c[a]), self.out,
                              self.ws, weight_in=self.w[a], weight_out=self.w[a])

    def evict(self, keep, recent):
        a, b = self.at, 1 - self.at
        self.kept = torch.zeros((self.dm.batch, self.dm.G, keep), dtype=torch.int32, device="cuda")
        sg.sgqa_cache8_evict(self.dm, self.block, self.lens[a], keep, recent, self.dm.T, self.w[a], *cache_args(self.c[a]),
                             *cache_args(self.c[b]), self.w[b], self.kept, self.lens[b], self.ws)
        self.at = b


def test_prompt_steps_eviction_and_on():
    gen = torch.Generator().manual_seed(20)
    batch, T, Hq, G, d, block, n = 3, 400, 8, 2, 128, 16, 2
    s = Session(batch, T, Hq, G, d, block, n)
    ref = c8.empty_cache(batch, T, G, d, block, device="cpu")
    counts = [200, 0, 117]
    k, v = c8.tokens(gen, batch, 200, G, d), c8.tokens(gen, batch, 200, G, d)
    s.w[0].zero_()
    s.prompt(k.cuda(), v.cuda(), i32(counts))
    ref = c8.ref_append(ref, block, [0] * 3, counts, k, v)
    lens = counts
    for step in range(12):
        for t in (s.k, s.v):
            t.copy_(c8.tokens(gen, batch, n, G, d))
        for t in (s.q, s.gate):
            t.copy_(torch.randn(t.shape, generator=gen))
        w_in = s.w[s.at].clone()
        s.step()
        ref = c8.ref_append(ref, block, lens, [n] * 3, s.k.cpu(), s.v.cpu())
        lens = [x + n for x in lens]
        torch.cuda.synchronize()
        c = s.c[s.at]
        for b, L in enumerate(lens):
            for name in ("k8", "v8"):
                assert torch.equal(c[name][b, :L].cpu(), ref[name][b, :L]), (step, name)
        out, mag, w = c8.ref_attend(c8.to_cuda(ref), block, lens, s.q, s.gate, w_in, s.w[s.at])
        close(s.out, out, mag, 64.0)
        close_weight(s.w[s.at], w, lens, n * Hq // G, s.w[s.at])
        if step in (5, 9):
            keep, recent = (64, 8) if step == 5 else (50, 3)
            w, a = s.w[s.at].cpu(), s.at
            s.evict(keep, recent)
            torch.cuda.synchronize()
            dst = c8.empty_cache(batch, T, G, d, block, device="cpu")
            dst.update(w=torch.zeros((batch, G, T)), kept=s.kept.cpu() * 0, lens_out=torch.zeros(batch, dtype=torch.int32))
            ref = c8.ref_evict(ref, block, lens, keep, recent, w, dst)
            lens = ref["lens_out"].tolist()
            assert s.lens[s.at].tolist() == lens and torch.equal(s.kept.cpu(), ref["kept"])
            ref = {x: ref[x] for x in ("k8", "ks", "v8", "vs")}
    assert sg.sgqa_get_device_status(s.ws) == 0


def test_a_captured_step_serves_every_length():
    gen = torch.Generator().manual_seed(21)
    make = lambda: Session(2, 600, 8, 2, 64, 32, 2)
    a, b = make(), make()
    k, v = c8.tokens(gen, 2, 120, 2, 64).cuda(), c8.tokens(gen, 2, 120, 2, 64).cuda()
    for s in (a, b):
        s.w[0].zero_()
        s.prompt(k, v, i32([120, 31]))
    steps = [(c8.tokens(gen, 2, 2, 2, 64), c8.tokens(gen, 2, 2, 2, 64), torch.randn(2, 2, 8, 64, generator=gen),
              torch.randn(2, 2, 8, 64, generator=gen)) for _ in range(60)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        b.step()
    for x in steps:
        for s in (a, b):
            for t, y in zip((s.k, s.v, s.q, s.gate), x):
                t.copy_(y)
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, b.out) and torch.equal(a.lens[0], b.lens[0])
    for i, L in enumerate(a.lens[0].tolist()):
        assert torch.equal(a.w[0][i, :, :L], b.w[0][i, :, :L])
        assert torch.equal(a.c[0]["k8"][i, :L], b.c[0]["k8"][i, :L])
    assert sg.sgqa_get_device_status(a.ws) == 0 and sg.sgqa_get_device_status(b.ws) == 0


def test_two_sessions_on_two_streams():
    gen = torch.Generator().manual_seed(22)
    sessions = [Session(2, 2000, 16, 2, 128, 64, 1) for _ in range(3)]
    k, v = c8.tokens(gen, 2, 1500, 2, 128).cuda(), c8.tokens(gen, 2, 1500, 2, 128).cuda()
    q = torch.randn(2, 1, 16, 128, generator=gen).cuda()
    for s in sessions:
        s.w[0].zero_()
        s.prompt(k, v, i32([1500, 700]))
        s.q.copy_(q)
        s.k.copy_(k[:, :1])
    for _ in range(20):
        sessions[0].step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, st in zip(sessions[1:], streams):
            with torch.cuda.stream(st):
                s.step()
    torch.cuda.synchronize()
    for s in sessions[1:]:
        assert torch.equal(s.out, sessions[0].out) and torch.equal(s.lens[0], sessions[0].lens[0])
        assert sg.sgqa_get_device_status(s.ws) == 0


def test_nothing_is_written_outside():
    """Buffers lie between guard bytes; rows behind a sequence's tokens keep what they held."""
    gen = torch.Generator().manual_seed(23)
    batch, T, Hq, G, d, block, n = 2, 203, 6, 2, 64, 16, 3
    guard = 4096

    def guarded(shape, dtype):
        nbytes = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((nbytes + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
        return raw, raw[guard:guard + nbytes].view(dtype).view(shape)

    nb = -(-T // block)
    shapes = dict(k8=((batch, T, G, d), torch.uint8), ks=((batch, nb, G), torch.float32), v8=((batch, T, G, d), torch.uint8),
                  vs=((batch, nb, G), torch.float32), out=((batch, n, Hq, d), torch.bfloat16),
                  w=((batch, G, T), torch.float32), k8o=((batch, 90, G, d), torch.uint8), kso=((batch, 6, G), torch.float32),
                  v8o=((batch, 90, G, d), torch.uint8), vso=((batch, 6, G), torch.float32), wo=((batch, G, 90), torch.float32),
                  kept=((batch, G, 77), torch.int32), lo=((batch,), torch.int32))
    raw, t = {}, {}
    for name, (shape, dtype) in shapes.items():
        raw[name], t[name] = guarded(shape, dtype)
    dm = dims(batch, T, Hq, G, d)
    ws = workspace(dm, block, n)
    lens = i32([0, 0])
    k, v = c8.tokens(gen, batch, 200, G, d).cuda(), c8.tokens(gen, batch, 200, G, d).cuda()
    cache = (t["k8"], t["ks"], t["v8"], t["vs"])
    sg.sgqa_cache8_append(dm, block, lens, 200, k, v, *cache, ws, counts=i32([200, 90]))
    lens = i32([200, 90])
    q, gate = queries(gen, batch, n, Hq, d)
    sg.sgqa_cache8_attend(dm, block, lens, n, q, gate, *cache, t["out"], ws, weight_out=t["w"])
    sg.sgqa_cache8_evict(dm, block, lens, 77, 9, 90, t["w"], *cache, t["k8o"], t["kso"], t["v8o"], t["vso"], t["wo"], t["kept"],
                         t["lo"], ws)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0
    for name, r in raw.items():
        assert bool((r[:guard] == 0xA5).all()) and bool((r[-guard:] == 0xA5).all()), name
    canary = lambda x: bool((x.contiguous().view(torch.uint8) == 0xA5).all())
    for b, L in enumerate((200, 90)):
        assert canary(t["k8"][b, L:]) and canary(t["v8"][b, L:]) and canary(t["w"][b, :, L:])
        assert canary(t["ks"][b, -(-L // block):]) and canary(t["vs"][b, -(-L // block):])
        assert canary(t["k8o"][b, 77:]) and canary(t["v8o"][b, 77:]) and canary(t["wo"][b, :, 77:])
        assert canary(t["kso"][b, 5:]) and canary(t["vso"][b, 5:])
