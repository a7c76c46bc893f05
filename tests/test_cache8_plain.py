"""The plain forms that the block-scaled 8-bit cache's GPU tests compare with, and the argument checks of
its entry points, on the CPU."""
import ctypes
import math

import pytest
import torch

import block_sparse_long_kbar_b200 as sg
from block_sparse_long_kbar_b200 import build as sg_build
from tests import _cache8 as c8


@pytest.fixture(scope="module")
def lib():
    sg_build.build()
    return sg.load_library()


def test_grid_is_the_e4m3_cast():
    x = torch.randn(20000, dtype=torch.float64) * torch.exp2(torch.rand(20000, dtype=torch.float64) * 22 - 14)
    x = torch.cat([x, torch.tensor([0.0, 448.0, -448.0, 460.0, 1e9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 17.0, 19.0])])
    want = x.clamp(-448, 448).float().to(c8.F8).double()  # the fp32 step rounds none of these to a tie
    near = (x.float().double() != x)
    got = c8.grid(x.float().double())
    assert torch.equal(got[~near], want[~near])
    assert torch.equal(got, x.float().double().clamp(-448, 448).float().to(c8.F8).double())


def test_scale_is_the_smallest_that_holds():
    a = torch.tensor([0.0, 2.0 ** -140, 1.0, 448.0, 449.0, 447.0, 1.75, 1.76, 3.3e38, 2.0 ** -118, 448 * 2.0 ** -126])
    s = c8.scale_of(a.double())
    for x, y in zip(a.double().tolist(), s.tolist()):
        e = math.log2(y)
        assert e == int(e) and -126 <= e <= 119
        assert x <= 448 * y or e == 119
        assert e == -126 or x > 448 * (y / 2)


def test_quantize_agrees_with_the_row_format(oracle_lib):
    """A block of one token and one group is the (token, group) row format, for ordinary magnitudes."""
    import numpy as np
    x = (torch.randn(64, 128) * torch.exp2(torch.randint(-20, 20, (64, 1)).float())).bfloat16()
    s = c8.scale_of(x.double().abs().amax(1))
    codes = c8.encode(c8.grid(x.double() / s[:, None]))
    q, so = oracle_lib.quantize_fp8(x.view(torch.int16).numpy().view(np.uint16))
    np.testing.assert_array_equal(codes.numpy(), q.reshape(64, 128))
    np.testing.assert_array_equal(s.numpy(), np.asarray(so).reshape(64))


def test_plain_attention_is_sdpa():
    gen = torch.Generator().manual_seed(0)
    lens, n, G, R, d, block = [5, 40], 3, 2, 3, 64, 16
    c = c8.filled_cache(gen, lens, 64, G, d, block)
    q, gate = torch.randn(2, n, G * R, d, generator=gen).bfloat16(), torch.randn(2, n, G * R, d, generator=gen).bfloat16()
    out, _, w = c8.ref_attend(c, block, lens, q, gate, None, torch.full((2, G, 64), -1.0))
    for b, L in enumerate(lens):
        k = c8.values(c["k8"][b, :L], c["ks"][b], block).repeat_interleave(R, 1).permute(1, 0, 2)
        v = c8.values(c["v8"][b, :L], c["vs"][b], block).repeat_interleave(R, 1).permute(1, 0, 2)
        mask = torch.arange(L)[None, :] <= (L - n + torch.arange(n))[:, None]
        o = torch.nn.functional.scaled_dot_product_attention(q[b].double().permute(1, 0, 2), k, v, attn_mask=mask)
        want = o.permute(1, 0, 2) * torch.sigmoid(gate[b].double())
        assert torch.allclose(out[b], want, rtol=1e-12, atol=1e-12)
        assert torch.allclose(w[b, :, :L].sum(-1), torch.full((G,), float(n * R), dtype=torch.float64))
        assert (w[b, :, L:] == -1).all()


def test_plain_eviction_keeps_the_heaviest_and_the_last():
    w = torch.tensor([3.0, math.nan, 0.0, -0.0, 5.0, 5.0, 1.0, math.inf, -math.inf, 2.0])
    assert c8.ref_kept(w, 10, 5, 1).tolist() == [0, 4, 5, 7, 9]
    assert c8.ref_kept(w, 9, 7, 0).tolist() == [0, 2, 3, 4, 5, 6, 7]
    assert c8.ref_kept(w, 9, 8, 0).tolist() == [0, 1, 2, 3, 4, 5, 6, 7]  # NaN ties with -infinity: lower position
    assert c8.ref_kept(w, 4, 5, 5).tolist() == [0, 1, 2, 3]
    assert c8.ref_kept(w, 9, 3, 3).tolist() == [6, 7, 8]


# ---- refusals (host checks: the pointers are never dereferenced) ------------------------------------
def D(**kw):
    base = dict(batch=2, T=512, Hq=8, G=2, d=64, d_idx=32, B=8, k=512)
    base.update(kw)
    return sg.sgqa_dims(*[base[n] for n in ("batch", "T", "Hq", "G", "d", "d_idx", "B", "k")])


GOOD = 0x7F0000000000
P = ctypes.c_void_p


def append(lib, dims=None, block=16, n_t=4, ws_bytes=1 << 20, **ptr):
    p = {n: P(ptr.get(n, GOOD)) for n in ("lens", "counts", "k", "v", "k8", "ks", "v8", "vs", "ws")}
    return lib.sgqa_cache8_append(ctypes.byref(dims or D()), block, p["lens"], p["counts"], n_t, p["k"], p["v"], p["k8"],
                                  p["ks"], p["v8"], p["vs"], p["ws"], ws_bytes, None)


def attend(lib, dims=None, block=16, n_new=4, ws_bytes=1 << 28, **ptr):
    names = ("lens", "q", "gate", "k8", "ks", "v8", "vs", "out", "w_in", "w_out", "ws")
    p = {n: P(ptr.get(n, GOOD)) for n in names}
    return lib.sgqa_cache8_attend(ctypes.byref(dims or D()), block, p["lens"], n_new, p["q"], p["gate"], p["k8"], p["ks"],
                                  p["v8"], p["vs"], p["out"], p["w_in"], p["w_out"], p["ws"], ws_bytes, None)


def evict(lib, dims=None, block=16, keep=100, recent=10, T_out=512, ws_bytes=1 << 28, **ptr):
    names = ("lens", "w", "k8", "ks", "v8", "vs", "k8o", "kso", "v8o", "vso", "wo", "kept", "lo", "ws")
    far = {n: GOOD + (i << 40) for i, n in enumerate(("k8o", "v8o", "wo", "lo"), 1)}
    p = {n: P(ptr.get(n, far.get(n, GOOD))) for n in names}
    return lib.sgqa_cache8_evict(ctypes.byref(dims or D()), block, p["lens"], keep, recent, T_out,
                                 *[p[n] for n in names[1:]], ws_bytes, None)


@pytest.mark.parametrize("call,pointers", [
    (append, ("lens", "k", "v", "k8", "ks", "v8", "vs")),
    (attend, ("lens", "q", "gate", "k8", "ks", "v8", "vs", "out")),
    (evict, ("lens", "w", "k8", "ks", "v8", "vs", "k8o", "kso", "v8o", "vso", "wo", "kept", "lo")),
])
def test_refusals_common(lib, call, pointers):
    for n in pointers:
        assert call(lib, **{n: 0}) == 1, n
        assert call(lib, **{n: GOOD + 8}) == 1, n
    assert call(lib, D(T=0)) == 1
    assert call(lib, D(d=96)) == 2
    for block in (0, -8, 4, 12, 24, 256):
        assert call(lib, block=block) == 2, block
    assert call(lib, ws=0) == 3
    assert call(lib, ws=GOOD + 16) == 3
    assert call(lib, ws_bytes=255) == 3


def test_refusals_append(lib):
    assert append(lib, n_t=-1) == 1
    assert append(lib, n_t=513) == 1
    assert append(lib, counts=GOOD + 4) == 1
    assert append(lib, n_t=0, counts=0, k=0, v=0) == 0  # nothing to do, nothing launched


def test_refusals_attend(lib):
    assert attend(lib, n_new=0) == 1
    assert attend(lib, n_new=-1) == 1
    assert attend(lib, w_out=0) == 1                     # weight_in without weight_out
    assert attend(lib, w_in=GOOD + 4) == 1
    assert attend(lib, w_out=GOOD + 4) == 1
    assert attend(lib, n_new=17) == 2                    # 17 * 4 heads per group > 64 rows
    need = sg.sgqa_cache8_workspace_size(D(), 16, 4)
    assert need > 0 and attend(lib, ws_bytes=need - 1) == 3
    assert sg.sgqa_cache8_workspace_size(D(), 16, 0) == 0
    assert sg.sgqa_cache8_workspace_size(D(), 16, 17) == 0
    assert sg.sgqa_cache8_workspace_size(D(), 16, 16) > 0
    assert sg.sgqa_cache8_workspace_size(D(), 24, 4) == 0
    assert sg.sgqa_cache8_workspace_size(D(T=0), 16, 4) == 0


def test_refusals_evict(lib):
    assert evict(lib, keep=0) == 1
    assert evict(lib, recent=-1) == 1
    assert evict(lib, recent=101) == 1
    assert evict(lib, T_out=99) == 1
    assert evict(lib, k8o=GOOD) == 1                     # onto itself
    assert evict(lib, v8o=GOOD) == 1
    assert evict(lib, wo=GOOD) == 1
    assert evict(lib, lo=GOOD) == 1
    assert evict(lib, T_out=1 << 28) == 1
    assert evict(lib, D(batch=64), T_out=1 << 27) == 2   # 2^34 rows in all
    long = D(batch=1, T=200000)                          # a selection with histograms in the workspace
    assert evict(lib, long, ws_bytes=256) == 3 and sg.sgqa_cache8_workspace_size(long, 16, 1) > 256


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(16)
    with pytest.raises(ValueError):
        sg.sgqa_cache8_append(D(), 16, x, 1, x, x, x, x, x, x, x)
    with pytest.raises(ValueError):
        sg.sgqa_cache8_attend(D(), 16, x, 1, x, x, x, x, x, x, x, x)
    with pytest.raises(ValueError):
        sg.sgqa_cache8_evict(D(), 16, x, 1, 0, 1, x, x, x, x, x, x, x, x, x, x, x, x, x)
