"""Appending to and evicting from caches of more than 2^32 bytes of codes (attention: test_gpu_cache8.py)."""
import pytest

torch = pytest.importorskip("torch")

import block_sparse_long_kbar_b200 as sg
from tests import _cache8 as c8

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

T, G, D, BLOCK = 8500003, 4, 128, 128
STEP = 1000 * BLOCK


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache(T):
    nb = -(-T // BLOCK)
    c = [torch.full((1, T, G, D), 0x7F, dtype=torch.uint8, device="cuda") if i % 2 == 0 else
         torch.full((1, nb, G), -3.0, device="cuda") for i in range(4)]
    return c


def rounded(x):
    """Codes and scales of rows [n, G, D] (fp64), n from a block's first token on."""
    n = x.shape[0]
    xb = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -n % BLOCK)).view(-1, BLOCK, G, D)
    s = c8.scale_of(xb.abs().amax(dim=(1, 3)))
    return c8.encode(c8.grid(xb / s[:, None, :, None]).view(-1, G, D)[:n]), s.float()


def dims(T):
    return sg.sgqa_dims(1, T, G, G, D, 64, 8, 512)


@pytest.fixture(autouse=True)
def room():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_append_beyond_32_bits():
    """A prompt of 8.5M tokens (4.35 GB of K codes, 8.7 GB of K), then a step at its end."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = T - 5
    k = torch.empty((1, n, G, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    v = torch.empty((1, n, G, D), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    c, ws = cache(T), sg.alloc_workspace(sg.sgqa_cache8_workspace_size(dims(T), BLOCK, 1))
    sg.sgqa_cache8_append(dims(T), BLOCK, i32([0]), n, k, v, *c, ws)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0
    for x, codes, scale in ((k, c[0], c[1]), (v, c[2], c[3])):
        for a in range(0, n, STEP):
            want, s = rounded(x[0, a:a + STEP].double())
            assert torch.equal(codes[0, a:a + STEP][:len(want)], want), a
            assert torch.equal(scale[0, a // BLOCK:a // BLOCK + len(s)], s), a
        assert bool((codes[0, n:] == 0x7F).all())
    a = n // BLOCK * BLOCK
    held = [t[:, a:].clone() if i % 2 == 0 else t[:, a // BLOCK:].clone() for i, t in enumerate(c)]
    k4, v4 = (torch.randn((1, 5, G, D), generator=gen, device="cuda").bfloat16() * 3 for _ in range(2))
    sg.sgqa_cache8_append(dims(T), BLOCK, i32([n]), 5, k4, v4, *c, ws)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0
    want = c8.ref_append(dict(zip(("k8", "ks", "v8", "vs"), (t.cpu() for t in held))), BLOCK, [n - a], [5], k4.cpu(), v4.cpu())
    for i, (name, t) in enumerate(zip(("k8", "ks", "v8", "vs"), c)):
        assert torch.equal((t[:, a:] if i % 2 == 0 else t[:, a // BLOCK:]).cpu(), want[name]), name


def test_evict_beyond_32_bits():
    """Nearly all of 8.5M tokens of four groups move to another cache of that size."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    keep, recent = 8450001, 1000
    src = cache(T)
    for t in (src[0], src[2]):
        t.random_(0, 0x7F, generator=gen)
    for t in (src[1], src[3]):
        t.copy_(torch.exp2(torch.randint(-9, -5, t.shape, generator=gen, device="cuda").float()))
    w = torch.rand((1, G, T), generator=gen, device="cuda")
    dst, w_out = cache(T), torch.full((1, G, T), -5.0, device="cuda")
    kept, lens_out = torch.zeros((1, G, keep), dtype=torch.int32, device="cuda"), i32([0])
    ws = sg.alloc_workspace(sg.sgqa_cache8_workspace_size(dims(T), BLOCK, 1))
    sg.sgqa_cache8_evict(dims(T), BLOCK, i32([T]), keep, recent, T, w, *src, *dst, w_out, kept, lens_out, ws)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0 and lens_out.tolist() == [keep]
    for g in range(G):
        rows = c8.ref_kept(w[0, g], T, keep, recent)
        assert torch.equal(kept[0, g].long(), rows)
        assert torch.equal(w_out[0, g, :keep], w[0, g][rows]) and bool((w_out[0, g, keep:] == -5).all())
        for codes, scale, to, to_scale in ((src[0], src[1], dst[0], dst[1]), (src[2], src[3], dst[2], dst[3])):
            for a in range(0, keep, STEP):
                r = rows[a:a + STEP]
                x = c8.decode(codes[0, r, g]) * scale[0, r // BLOCK, g].double()[:, None]
                xb = torch.nn.functional.pad(x, (0, 0, 0, -len(r) % BLOCK)).view(-1, BLOCK, D)
                s = c8.scale_of(xb.abs().amax(dim=(1, 2)))
                want = c8.grid(xb / s[:, None, None]).view(-1, D)[:len(r)]
                assert torch.equal(c8.decode(to[0, a:a + len(r), g]), want), (g, a)
                assert torch.equal(to_scale[0, a // BLOCK:a // BLOCK + len(s), g].double(), s), (g, a)
            assert bool((to[0, keep:, g] == 0x7F).all())
