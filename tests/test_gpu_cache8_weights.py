"""What the received weights of sgqa_cache8_attend keep of their digits.

Queries are multiples of 1/16 of eight bits and keys small whole numbers (times their block's scale), so that both
E4M3 terms of q, all products and their sums are exact in any order: below 2^17 in multiples of 2^-4. With z the
base-2 exponent, |z| <= 32 and |z - log2 sum| <= 64, what is left is fp32's rounding:
  * z: the factor log2(e) / sqrt(d) (three roundings: constant, root, quotient) and two products, 2^-24 of z
    each: 5 * 32 * 2^-24; the same in a row's maximum and through its denominator (an average over its tokens);
  * the denominator: differences to the maximum (64 * 2^-24) and the base-2 exponential (2^-22) of every token, at
    most 30 additions on the way from a token to the row's sum (4 tokens of a lane, 3 halvings, 4 warps, the tiles of
    a piece, the pieces), and a logarithm (2^-22 and half a step of a number below 64, 2^-19 in all);
  * the probability: a difference (64 * 2^-24) and an exponential (2^-22).
Exponents count ln 2 times in a probability: ln 2 (160 + 160 + 64 + 64 + 32) 2^-24 + (2 * 4 + 30 + 4) 2^-24 < 375 * 2^-24
< 2^-15.4; the sum over up to 64 rows adds 66 * 2^-24. Below 2^-15 together. What a token had received before is only
added to: 2^-24 of the total.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import block_sparse_long_kbar_b200 as sg
from tests import _cache8 as c8

pytestmark = pytest.mark.gpu


def exact_inputs(gen, batch, T, G, R, d, block, n):
    k = torch.randint(-2, 3, (batch, T, G, d), generator=gen).double()
    c = c8.empty_cache(batch, T, G, d, block, device="cpu")
    c["k8"] = c8.encode(k)
    c["v8"] = torch.randint(0, 0x50, (batch, T, G, d), generator=gen, dtype=torch.uint8)
    c["ks"] = torch.exp2(-torch.randint(2, 5, c["ks"].shape, generator=gen).float())
    c["vs"] = torch.ones_like(c["vs"])
    q = (torch.randint(16, 256, (batch, n, G * R, d), generator=gen) * (torch.randint(0, 2, (batch, n, G * R, d), generator=gen) * 2 - 1)) / 16
    assert torch.equal(q.bfloat16().double(), q.double())
    return c8.to_cuda(c), q.bfloat16().cuda(), torch.randn(batch, n, G * R, d, generator=gen).bfloat16().cuda()


@pytest.mark.parametrize("d,R,n,block", [(64, 1, 1, 8), (64, 3, 5, 64), (128, 4, 1, 16), (128, 8, 4, 32), (128, 16, 4, 128), (64, 12, 3, 16)])
@pytest.mark.parametrize("past", [0.0, 1.0, 3000.0])
def test_received_weights_keep_their_digits(d, R, n, block, past):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gen = torch.Generator().manual_seed(d + R + n)
    lens, G, T = [900, 129, 70, 2, 0], 2, 903
    c, q, gate = exact_inputs(gen, len(lens), T, G, R, d, block, n)
    w_in = ((torch.rand((len(lens), G, T), generator=gen) + 0.5) * past).cuda()
    dm = sg.sgqa_dims(len(lens), T, G * R, G, d, 64, 8, 512)
    ws, out, w = sg.alloc_workspace(sg.sgqa_cache8_workspace_size(dm, block, n)), torch.zeros_like(q), torch.full_like(w_in, -7.0)
    sg.sgqa_cache8_attend(dm, block, torch.tensor(lens, dtype=torch.int32, device="cuda"), n, q, gate, c["k8"], c["ks"], c["v8"], c["vs"],
                          out, ws, weight_in=w_in, weight_out=w)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0
    for b, L in enumerate(lens):
        assert bool((w[b, :, L:] == -7.0).all())
        if not L:
            continue
        k = c8.values(c["k8"][b, :L], c["ks"][b], block)
        fresh = torch.zeros((G, L), dtype=torch.float64, device="cuda")
        for i in range(n):
            m = L - n + i + 1
            for g in range(G if m > 0 else 0):
                z = q[b, i, g * R:(g + 1) * R].double() @ k[:m, g].T / math.sqrt(d)
                assert float(z.abs().max()) * math.log2(math.e) <= 32
                fresh[g, :m] += torch.softmax(z, -1).sum(0)
        old = torch.where(torch.arange(L, device="cuda") < L - n, w_in[b, :, :L].double(), 0.0)
        err = (w[b, :, :L].double() - (old + fresh)).abs()
        assert bool((err <= 2.0 ** -15 * fresh + 2.0 ** -24 * (old + fresh)).all()), float((err / (2.0 ** -15 * fresh)).max())
