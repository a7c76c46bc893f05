"""The block-scaled 8-bit cache at the limits of its arguments: the most sequences, large queries, captured calls
that share a workspace, a captured eviction by clusters of 16."""
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


def workspace(dm, block, n=1):
    ws = sg.alloc_workspace(sg.sgqa_cache8_workspace_size(dm, block, n))
    ws[256:].fill_(0xFF)
    return ws


def test_the_most_sequences():
    """65535 sequences of up to 5 tokens: append, attend, evict. Bounds as in test_gpu_cache8_bounds.py, with p = 1 and
    a code of 448 in the floor that each token adds."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    batch, T, G, R, d, block, n, keep = 65535, 5, 1, 2, 64, 8, 2, 3
    dm = dims(batch, T, R, G, d)
    ws = workspace(dm, block, n)
    lens = torch.randint(0, T + 1, (batch,), generator=gen, device="cuda").int()
    lens[-1] = T
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    k, v = new(batch, T, G, d), new(batch, T, G, d)
    c = c8.empty_cache(batch, T, G, d, block)
    a = (c["k8"], c["ks"], c["v8"], c["vs"])
    sg.sgqa_cache8_append(dm, block, torch.zeros_like(lens), T, k, v, *a, ws, counts=lens)
    live = torch.arange(T, device="cuda") < lens[:, None]
    vals = {}
    for name, x, codes, scale in (("k", k, c["k8"], c["ks"]), ("v", v, c["v8"], c["vs"])):
        y = torch.where(live[:, :, None, None], x.double(), 0.0)
        s = c8.scale_of(y.abs().amax(dim=(1, 3)))
        some = lens > 0
        assert torch.equal(scale[:, 0][some].double(), s[some])
        want = c8.grid(y / s[:, None, :, None])
        assert torch.equal(torch.where(live[:, :, None, None], c8.decode(codes), 0.0).nan_to_num(nan=9e9), want)
        assert bool((codes[~live] == 0x7F).all())
        vals[name] = want * s[:, None, :, None]
        vals["s"] = s
    q, gate = new(batch, n, R, d), new(batch, n, R, d)
    out, w = torch.zeros_like(q), torch.full((batch, G, T), -7.0, device="cuda")
    sg.sgqa_cache8_attend(dm, block, lens, n, q, gate, *a, out, ws, weight_out=w)
    z = torch.einsum("bnhd,btd->bnht", q.double(), vals["k"][:, :, 0]) / math.sqrt(d)
    pos = lens[:, None] - n + torch.arange(n, device="cuda")
    sees = (torch.arange(T, device="cuda") <= pos[:, :, None])[:, :, None]
    p = torch.softmax(torch.where(sees, z, -math.inf), -1).nan_to_num(nan=0.0)
    sig = torch.sigmoid(gate.double())
    ref = torch.einsum("bnht,btd->bnhd", p, vals["v"][:, :, 0]) * sig
    tol = torch.einsum("bnht,btd->bnhd", p, vals["v"][:, :, 0].abs()) * sig * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14) + ref.abs() * 2.0 ** -8
    tol += T * 2.0 ** -19.6 * 448 * vals["s"][:, :, None, None] + 2.0 ** -133
    assert bool(((out.double() - ref).abs() <= tol).all())
    assert bool((((w[:, 0].double() - p.sum((1, 2))).abs() <= 2.0 ** -10) | ~live).all()) and bool((w[:, 0][~live] == -7).all())
    d8 = c8.empty_cache(batch, keep, G, d, block)
    w2, kept = torch.zeros((batch, G, keep), device="cuda"), torch.zeros((batch, G, keep), dtype=torch.int32, device="cuda")
    l2 = torch.zeros_like(lens)
    sg.sgqa_cache8_evict(dm, block, lens, keep, 1, keep, w, *a, d8["k8"], d8["ks"], d8["v8"], d8["vs"], w2, kept, l2, ws)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0 and torch.equal(l2, lens.clamp(max=keep))
    # of 5 tokens the last stays and the two heaviest of the others
    old = torch.where(torch.arange(T, device="cuda") < lens[:, None] - 1, w[:, 0], -1.0)
    top = torch.sort(torch.sort(old, dim=1, descending=True, stable=True).indices[:, :keep - 1], dim=1).values
    long = lens > keep
    assert torch.equal(kept[long, 0, :2].long(), top[long]) and torch.equal(kept[long, 0, 2], lens[long] - 1)
    u = torch.arange(keep, device="cuda").int()
    assert torch.equal(kept[~long, 0], torch.where(u < lens[~long, None], u, -1))


@pytest.mark.parametrize("d", [64, 128])
def test_large_queries_on_small_keys(d):
    """Queries near 2^111 on keys as small: the scores are ordinary ones, and so is the result."""
    gen = torch.Generator().manual_seed(d)
    L, G, R, block = 300, 1, 4, 16
    k, v = c8.tokens(gen, 1, L, G, d, 0.0), c8.tokens(gen, 1, L, G, d, 0.0)
    q = torch.randn(1, 2, R, d, generator=gen).clamp(-4, 4).bfloat16()
    gate = torch.randn(1, 2, R, d, generator=gen).bfloat16().cuda()
    outs = []
    for up in (0, 109):
        c = c8.to_cuda(c8.ref_append(c8.empty_cache(1, L, G, d, block, device="cpu"), block, [0], [L], k * 2.0 ** -up, v))
        dm = dims(1, L, R, G, d)
        ws, out, w = workspace(dm, block, 2), torch.zeros_like(gate), torch.zeros((1, G, L), device="cuda")
        sg.sgqa_cache8_attend(dm, block, torch.tensor([L], dtype=torch.int32, device="cuda"), 2, (q * 2.0 ** up).cuda(), gate, c["k8"],
                              c["ks"], c["v8"], c["vs"], out, ws, weight_out=w)
        torch.cuda.synchronize()
        assert sg.sgqa_get_device_status(ws) == 0
        outs.append((out, w))
    # powers of two change no digit
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert bool(torch.isfinite(outs[1][0]).all()) and bool((outs[1][0] != 0).any())


def test_a_captured_eviction_by_clusters_of_16():
    gen = torch.Generator(device="cuda").manual_seed(5)
    batch, T, keep, recent, block = 11, 140003, 900, 10, 64
    dm = dims(batch, T, 1, 1, 64)
    c = {n: torch.randint(0, 0x7F, (batch, T, 1, 64), generator=gen, dtype=torch.uint8, device="cuda") for n in ("k8", "v8")}
    c.update({n: torch.ones((batch, -(-T // block), 1), device="cuda") for n in ("ks", "vs")})
    w = torch.rand((batch, 1, T), generator=gen, device="cuda")
    dst = c8.empty_cache(batch, keep, 1, 64, block)
    w2, kept = torch.zeros((batch, 1, keep), device="cuda"), torch.zeros((batch, 1, keep), dtype=torch.int32, device="cuda")
    lens, l2 = torch.full((batch,), T, dtype=torch.int32, device="cuda"), torch.zeros(batch, dtype=torch.int32, device="cuda")
    ws = workspace(dm, block)
    call = lambda: sg.sgqa_cache8_evict(dm, block, lens, keep, recent, keep, w, c["k8"], c["ks"], c["v8"], c["vs"], dst["k8"], dst["ks"],
                                        dst["v8"], dst["vs"], w2, kept, l2, ws)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):  # the first call of the process may be a captured one
        call()
    for less in (0, 7, 100):
        lens.copy_(T - less - torch.arange(batch, device="cuda") * less)
        w.copy_(torch.rand(w.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert sg.sgqa_get_device_status(ws) == 0
        for b, L in enumerate(lens.tolist()):
            rows = c8.ref_kept(w[b, 0], L, keep, recent)
            assert torch.equal(kept[b, 0].long(), rows) and torch.equal(w2[b, 0], w[b, 0][rows])
            assert torch.equal(dst["k8"][b, :, 0][:5] & 0x80, c["k8"][b, rows[:5], 0] & 0x80)


def test_graphs_of_two_sizes_share_a_workspace():
    """A workspace made for the longest step serves shorter ones, and captured calls that share it take turns."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    batch, T, G, R, d, block = 4, 3000, 2, 4, 128, 32
    dm = dims(batch, T, G * R, G, d)
    ws = workspace(dm, block, 16)
    c = {n: torch.randint(0, 0x50, (batch, T, G, d), generator=gen, dtype=torch.uint8, device="cuda") for n in ("k8", "v8")}
    c.update({n: torch.full((batch, -(-T // block), G), 2.0 ** -5, device="cuda") for n in ("ks", "vs")})
    lens = torch.tensor([T, 17, 2222, 1], dtype=torch.int32, device="cuda")
    calls, alone = [], []
    for n in (1, 16, 4, 9):
        q, gate = (torch.randn(batch, n, G * R, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
        out, w = torch.zeros_like(q), torch.zeros((batch, G, T), device="cuda")
        call = lambda n=n, q=q, gate=gate, out=out, w=w, ws=ws: sg.sgqa_cache8_attend(
            dm, block, lens, n, q, gate, c["k8"], c["ks"], c["v8"], c["vs"], out, ws, weight_out=w)
        call(ws=workspace(dm, block, n))
        torch.cuda.synchronize()
        alone.append((out.clone(), w.clone()))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        calls.append((graph, out, w, q, gate))  # (a captured call reads q and gate where they are)
    for _ in range(3):
        for graph, out, w, *_ in calls:
            out.zero_()
            w.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for (graph, out, w, *_), (o, x) in zip(calls, alone):
            assert torch.equal(out, o) and torch.equal(w, x)
    assert sg.sgqa_get_device_status(ws) == 0
