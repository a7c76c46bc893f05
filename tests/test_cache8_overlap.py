"""Tensors of the block-scaled 8-bit cache's calls that share memory, refused on the host (the pointers are never
dereferenced), and those that may."""
import ctypes

import pytest
import torch

import block_sparse_long_kbar_b200 as sg
from block_sparse_long_kbar_b200 import build as sg_build

BATCH, T, HQ, G, D, BLOCK, N, KEEP, T_OUT = 2, 512, 8, 2, 64, 16, 4, 100, 256
CODES, SCALES, NEW, QS, W = BATCH * T * G * D, BATCH * T // BLOCK * G * 4, BATCH * N * G * D * 2, BATCH * N * HQ * D * 2, BATCH * G * T * 4
CODES_OUT, SCALES_OUT, W_OUT = BATCH * T_OUT * G * D, BATCH * T_OUT // BLOCK * G * 4, BATCH * G * T_OUT * 4
INPUTS = {
    "append": dict(lens=8, counts=8, k=NEW, v=NEW),
    "attend": dict(lens=8, q=QS, gate=QS, k8=CODES, ks=SCALES, v8=CODES, vs=SCALES, w_in=W),
    "evict": dict(lens=8, w=W, k8=CODES, ks=SCALES, v8=CODES, vs=SCALES),
}
OUTPUTS = {
    "append": dict(k8=CODES, ks=SCALES, v8=CODES, vs=SCALES, ws=256),
    "attend": dict(out=QS, w_out=W, ws=256),
    "evict": dict(k8o=CODES_OUT, kso=SCALES_OUT, v8o=CODES_OUT, vso=SCALES_OUT, wo=W_OUT, kept=BATCH * G * KEEP * 4, lo=8, ws=256),
}
MAY = {("attend", "out", "gate"), ("attend", "w_out", "w_in")}  # the same tensor
MAY_OR_BESIDE = {"append": [("k8", "k"), ("v8", "k8"), ("ks", "v8")], "attend": [("out", "gate"), ("w_out", "w_in"), ("out", "q")],
                 "evict": [("k8o", "k8"), ("vso", "vs"), ("wo", "kept")]}


@pytest.fixture(scope="module")
def lib():
    sg_build.build()
    return sg.load_library()


def call(lib, name, at):
    P = lambda *n: [ctypes.c_void_p(at[x]) for x in n]
    dm = ctypes.byref(sg.sgqa_dims(BATCH, T, HQ, G, D, 32, 8, 512))
    if name == "append":
        return lib.sgqa_cache8_append(dm, BLOCK, *P("lens", "counts"), N, *P("k", "v", "k8", "ks", "v8", "vs", "ws"), 1 << 28, None)
    if name == "attend":
        return lib.sgqa_cache8_attend(dm, BLOCK, *P("lens"), N, *P("q", "gate", "k8", "ks", "v8", "vs", "out", "w_in", "w_out", "ws"),
                                      1 << 28, None)
    return lib.sgqa_cache8_evict(dm, BLOCK, *P("lens"), KEEP, 10, T_OUT, *P("w", "k8", "ks", "v8", "vs", "k8o", "kso", "v8o", "vso",
                                                                          "wo", "kept", "lo", "ws"), 1 << 28, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: for a machine without a GPU")
@pytest.mark.parametrize("name", list(INPUTS))
def test_an_output_over_another_tensor_is_refused(lib, name):
    sizes = {**INPUTS[name], **OUTPUTS[name]}
    if name == "attend":
        sizes["ws"] = sg.sgqa_cache8_workspace_size(sg.sgqa_dims(BATCH, T, HQ, G, D, 32, 8, 512), BLOCK, N)
    apart = {n: (i + 1) << 40 for i, n in enumerate(sizes)}
    assert call(lib, name, apart) == 4  # gets as far as the launch, which has no GPU
    for o in OUTPUTS[name]:
        for x in sizes:
            if x == o:
                continue
            # the same address; the output's end in the other's start; its start in the other's end (addresses of
            # ws are multiples of 256, all others of 16)
            for shift in {0, -(sizes[o] - 1) // 256 * 256 + 256, (sizes[x] - 1) // 256 * 256}:
                if shift <= -sizes[o] or (shift == 0 and {(name, o, x), (name, x, o)} & MAY):
                    continue
                assert call(lib, name, {**apart, o: apart[x] + shift}) == 1, (o, x, shift)
    for o, x in MAY_OR_BESIDE[name]:
        assert call(lib, name, {**apart, o: apart[x] + (0 if (name, o, x) in MAY else sizes[x])}) == 4, (o, x)
        if (name, o, x) in MAY:
            assert call(lib, name, {**apart, o: apart[x] + 256}) == 1, "moved against it"


@pytest.mark.gpu
def test_out_over_gate_and_weights_in_place():
    """What may be the same tensor gives what separate ones do."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for batch, T, R, d, n in ((3, 700, 4, 64, 2), (1, 9000, 16, 128, 4), (300, 90, 2, 64, 1)):
        k8 = torch.randint(0, 0x50, (batch, T, 2, d), generator=gen, dtype=torch.uint8, device="cuda")
        v8, ks = k8.flip(1).contiguous(), torch.full((batch, -(-T // 16), 2), 2.0 ** -5, device="cuda")
        q, gate = (torch.randn(batch, n, 2 * R, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
        w = torch.rand(batch, 2, T, generator=gen, device="cuda")
        lens = torch.randint(0, T + 1, (batch,), generator=gen, device="cuda").int()
        dm = sg.sgqa_dims(batch, T, 2 * R, 2, d, 64, 8, 512)
        ws = sg.alloc_workspace(sg.sgqa_cache8_workspace_size(dm, 16, n))
        out, w_out = torch.zeros_like(q), w.clone()
        sg.sgqa_cache8_attend(dm, 16, lens, n, q, gate, k8, ks, v8, ks, out, ws, weight_in=w, weight_out=w_out)
        sg.sgqa_cache8_attend(dm, 16, lens, n, q, gate, k8, ks, v8, ks, gate, ws, weight_in=w, weight_out=w)
        torch.cuda.synchronize()
        assert sg.sgqa_get_device_status(ws) == 0 and torch.equal(gate, out) and torch.equal(w, w_out)
        for bad in (q, k8.view(torch.bfloat16).flatten()[:q.numel()] if k8.numel() >= 2 * q.numel() else q):
            with pytest.raises(sg.SgqaError):
                sg.sgqa_cache8_attend(dm, 16, lens, n, q, gate, k8, ks, v8, ks, bad, ws)


@pytest.mark.parametrize("R,d", [(1, 64), (3, 128), (8, 128), (11, 64), (16, 128)])
def test_a_workspace_for_more_new_tokens_holds_fewer(lib, R, d):
    sizes = [sg.sgqa_cache8_workspace_size(sg.sgqa_dims(3, 4000, 4 * R, 4, d, 32, 8, 512), 16, n) for n in range(1, 64 // R + 1)]
    assert sizes == sorted(sizes) and sizes[0] > 0
