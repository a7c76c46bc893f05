"""The block-scaled 8-bit cache under the bounds-checking debug build (libsgqa_checks.so): its kernels test the
indices they get from lengths, pieces of tiles and selections before they use them. The cache's tests run with it in
a child process, where a check that fires shows in a status they require to be clean, and its results are the
normal build's bit for bit."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu

RUN = """
import sys, torch
import block_sparse_long_kbar_b200 as sg
out = {}
for batch, T, G, R, d, block, n, keep in ((5, 1000, 2, 4, 128, 16, 3, 300), (1, 200000, 2, 16, 64, 64, 4, 60001),
                                          (300, 130, 1, 2, 64, 8, 1, 50), (11, 135000, 1, 1, 64, 128, 1, 9000)):
    gen = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    dm = sg.sgqa_dims(batch, T, G * R, G, d, 64, 8, 512)
    ws = sg.alloc_workspace(sg.sgqa_cache8_workspace_size(dm, block, n))
    new = lambda t: (*(torch.zeros(batch, t, G, d, dtype=torch.uint8, device="cuda") if i % 2 == 0 else
                       torch.ones(batch, -(-t // block), G, device="cuda") for i in range(4)),)
    c, c2 = new(T), new(keep + 7)
    lens = torch.randint(0, T - 99, (batch,), generator=gen, device="cuda").int()
    lens[-1] = T - 100
    sg.sgqa_cache8_append(dm, block, torch.zeros_like(lens), T - 100, rand(batch, T - 100, G, d), rand(batch, T - 100, G, d), *c, ws,
                          counts=lens)
    sg.sgqa_cache8_append(dm, block, lens, n, rand(batch, n, G, d), rand(batch, n, G, d), *c, ws)
    lens += n
    o, w = rand(batch, n, G * R, d), torch.zeros(batch, G, T, device="cuda")
    sg.sgqa_cache8_attend(dm, block, lens, n, rand(batch, n, G * R, d), rand(batch, n, G * R, d), *c, o, ws, weight_out=w)
    w2, kept = torch.zeros(batch, G, keep + 7, device="cuda"), torch.zeros(batch, G, keep, dtype=torch.int32, device="cuda")
    l2 = torch.zeros_like(lens)
    sg.sgqa_cache8_evict(dm, block, lens, keep, 20, keep + 7, w, *c, *c2, w2, kept, l2, ws)
    torch.cuda.synchronize()
    assert sg.sgqa_get_device_status(ws) == 0
    out[T] = [x.cpu() for x in (*c, o, w, *c2, w2, kept, l2)]
torch.save((sg.SO_PATH, out), sys.argv[1])
"""


def env(checks):
    e = dict(os.environ, PYTHONPATH=ROOT)
    e.pop("SGQA_LIBRARY", None)
    if checks:
        e["SGQA_LIBRARY"] = "checks"
    return e


def test_the_caches_tests_under_bounds_checks():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cmd = [sys.executable, "-m", "pytest", "tests/test_gpu_cache8.py", "tests/test_gpu_cache8_bounds.py", "-m", "gpu", "-q", "-x", "-p",
           "no:cacheprovider", "-k", "not beyond_32_bits"]
    r = subprocess.run(cmd, cwd=ROOT, env=env(True), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout


def test_the_checks_change_no_result(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    got = []
    for checks in (False, True):
        p = str(tmp_path / f"{checks}.pt")
        r = subprocess.run([sys.executable, "-c", RUN, p], cwd=ROOT, env=env(checks), capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
        got.append(torch.load(p))
    (so, a), (so_checks, b) = got
    assert so.endswith("libsgqa.so") and so_checks.endswith("libsgqa_checks.so")
    for T in a:
        for i, (x, y) in enumerate(zip(a[T], b[T])):
            assert torch.equal(x, y), (T, i)
