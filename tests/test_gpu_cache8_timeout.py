"""sgqa_cache8_attend when a wait of its pass for the received weights runs out."""
import pytest

torch = pytest.importorskip("torch")

import block_sparse_long_kbar_b200 as sg
from tests import _cache8 as c8

pytestmark = pytest.mark.gpu

STALL_WEIGHTS = 1 << 20


@pytest.mark.parametrize("d,R,n", [(64, 2, 1), (128, 8, 4), (128, 16, 4)])
def test_weights_are_as_they_were_or_complete(d, R, n):
    """One CTA of the pass issues no loads (the hook): the call ends with the timeout recorded, `out` is whole, and
    of weights that are added up in place each is the one before the call or the one after a good call."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gen = torch.Generator(device="cuda").manual_seed(d + R)
    batch, T, G, block = 2, 13000, 2, 64
    c = {x: torch.randint(0, 0x50, (batch, T, G, d), generator=gen, dtype=torch.uint8, device="cuda") for x in ("k8", "v8")}
    c.update({x: torch.full((batch, -(-T // block), G), 2.0 ** -5, device="cuda") for x in ("ks", "vs")})
    q, gate = (torch.randn(batch, n, G * R, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    past = torch.rand((batch, G, T), generator=gen, device="cuda")
    lens = torch.tensor([T, 11111], dtype=torch.int32, device="cuda")
    dm = sg.sgqa_dims(batch, T, G * R, G, d, 64, 8, 512)
    ws = sg.alloc_workspace(sg.sgqa_cache8_workspace_size(dm, block, n))

    def call(w):
        out = torch.zeros_like(q)
        sg.sgqa_cache8_attend(dm, block, lens, n, q, gate, c["k8"], c["ks"], c["v8"], c["vs"], out, ws, weight_in=w, weight_out=w)
        torch.cuda.synchronize()
        return out, sg.sgqa_get_device_status(ws)

    whole = past.clone()
    out, status = call(whole)
    assert status == 0
    for cta in (0, 77, 147):
        w = past.clone()
        sg.sgqa_test_stall_decode_cta(STALL_WEIGHTS + cta)
        try:
            got, status = call(w)
        finally:
            sg.sgqa_test_stall_decode_cta(-1)
        assert status == 5 and torch.equal(got, out)
        old, new = w == past, w == whole
        assert bool((old | new).all()), int((~(old | new)).sum())
        assert bool((old & ~new).any()) and bool((new & ~old).any())
        sg.sgqa_reset_device_status(ws)
    w = past.clone()
    got, status = call(w)
    assert status == 0 and torch.equal(got, out) and torch.equal(w, whole)
