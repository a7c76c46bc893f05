"""What the binding of the block-scaled 8-bit cache refuses before the library is called: tensors of another type,
or of other sizes than dims, would be read as they lie. On the CPU, with stand-ins for device tensors."""
import math

import pytest
import torch

import block_sparse_long_kbar_b200 as sg

U8, F32, I32, BF16 = torch.uint8, torch.float32, torch.int32, torch.bfloat16
B, T, HQ, G, D, BLOCK, N = 3, 50, 8, 2, 64, 16, 4
NB, KEEP, T_OUT = -(-T // BLOCK), 20, 33
NB_OUT = -(-T_OUT // BLOCK)


class Tensor:
    """What the binding asks of a device tensor."""

    def __init__(self, shape, dtype, device=0, contiguous=True):
        self.shape, self.dtype, self.device_index, self.contiguous = torch.Size(shape), dtype, device, contiguous

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return math.prod(self.shape)

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 0x7F0000000000


class Library:
    calls = 0

    def __getattr__(self, name):
        def call(*args):
            Library.calls += 1
            return 0
        return call


@pytest.fixture(autouse=True)
def fake(monkeypatch):
    monkeypatch.setattr(sg, "load_library", lambda lib=Library(): lib)
    monkeypatch.setattr(sg, "_current_device", lambda: 0)
    monkeypatch.setattr(sg, "_current_stream", lambda device: 0)


def calls_of(f, **kw):
    before = Library.calls
    f(**kw)
    return Library.calls - before


def dims():
    return sg.sgqa_dims(B, T, HQ, G, D, 64, 8, 512)


CACHE = dict(k8=((B, T, G, D), U8), k_scale=((B, NB, G), F32), v8=((B, T, G, D), U8), v_scale=((B, NB, G), F32))
CALLS = {
    "append": (lambda **t: sg.sgqa_cache8_append(dims(), BLOCK, n_t=N, **t),
               dict(lens=((B,), I32), counts=((B,), I32), k_new=((B, N, G, D), BF16), v_new=((B, N, G, D), BF16), **CACHE)),
    "attend": (lambda **t: sg.sgqa_cache8_attend(dims(), BLOCK, n_new=N, **t),
               dict(lens=((B,), I32), q=((B, N, HQ, D), BF16), gate=((B, N, HQ, D), BF16), out=((B, N, HQ, D), BF16),
                    weight_in=((B, G, T), F32), weight_out=((B, G, T), F32), **CACHE)),
    "evict": (lambda **t: sg.sgqa_cache8_evict(dims(), BLOCK, keep=KEEP, recent=5, T_out=T_OUT, **t),
              dict(lens=((B,), I32), weight=((B, G, T), F32), k8_out=((B, T_OUT, G, D), U8), k_scale_out=((B, NB_OUT, G), F32),
                   v8_out=((B, T_OUT, G, D), U8), v_scale_out=((B, NB_OUT, G), F32), weight_out=((B, G, T_OUT), F32),
                   kept=((B, G, KEEP), I32), lens_out=((B,), I32), **CACHE)),
}
EACH = [(call, name) for call, (_, t) in CALLS.items() for name in t]


def tensors(call):
    return {n: Tensor(*x) for n, x in CALLS[call][1].items()} | {"ws": Tensor((1 << 20,), U8)}


@pytest.mark.parametrize("call", CALLS)
def test_what_fits_reaches_the_library(call):
    f, spec = CALLS[call]
    t = tensors(call)
    assert calls_of(f, **t) == 1
    for name, (shape, dtype) in spec.items():
        for other in ((math.prod(shape),), (shape[0] + 2, *shape[1:])):  # flat; sequences behind the batch's
            assert calls_of(f, **{**t, name: Tensor(other, dtype)}) == 1, (name, other)
        if dtype is BF16:
            assert calls_of(f, **{**t, name: Tensor(shape, torch.uint16)}) == 1
        if dtype is U8:
            assert calls_of(f, **{**t, name: Tensor(shape, torch.float8_e4m3fn)}) == 1


@pytest.mark.parametrize("call,name", EACH)
def test_refuses_other_types(call, name):
    f, spec = CALLS[call]
    shape, dtype = spec[name]
    for other in (torch.int64, torch.float16, torch.float64, torch.bool, U8, F32, I32, BF16):
        if other is not dtype:
            with pytest.raises(ValueError, match=name):
                f(**{**tensors(call), name: Tensor(shape, other)})


@pytest.mark.parametrize("call,name", EACH)
def test_refuses_other_sizes(call, name):
    f, spec = CALLS[call]
    shape, dtype = spec[name]
    others = [(shape[0] - 1, *shape[1:]), (math.prod(shape) - 1,), (math.prod(shape) + 1,), ()]
    others += [shape[:i] + (shape[i] + x,) + shape[i + 1:] for i in range(1, len(shape)) for x in (-1, 1)]
    for other in others:
        if len(shape) == 1 and len(other) == 1 and other[0] > shape[0]:
            continue  # sequences behind the batch's
        with pytest.raises(ValueError, match=name):
            f(**{**tensors(call), name: Tensor(other, dtype)})


@pytest.mark.parametrize("call,name", EACH + [(c, "ws") for c in CALLS])
def test_refuses_other_devices_and_strides(call, name):
    f, spec = CALLS[call]
    shape, dtype = spec.get(name, ((1 << 20,), U8))
    for bad in (Tensor(shape, dtype, device=-1), Tensor(shape, dtype, device=1), Tensor(shape, dtype, contiguous=False)):
        with pytest.raises(ValueError):
            f(**{**tensors(call), name: bad})


def test_what_the_library_refuses_by_itself_reaches_it():
    """Sizes and blocks that no cache has: the library's own status says so."""
    t = tensors("append")
    for kw in (dict(block=0, n_t=N), dict(block=24, n_t=N), dict(block=BLOCK, n_t=-1), dict(block=BLOCK, n_t=0)):
        assert calls_of(sg.sgqa_cache8_append, dims=dims(), **kw, **t) == 1
    t = tensors("attend")
    for kw in (dict(block=7, n_new=N), dict(block=BLOCK, n_new=0)):
        assert calls_of(sg.sgqa_cache8_attend, dims=dims(), **kw, **t) == 1
    t = tensors("evict")
    for kw in (dict(block=4, keep=KEEP, T_out=T_OUT), dict(block=BLOCK, keep=0, T_out=T_OUT), dict(block=BLOCK, keep=KEEP, T_out=-1)):
        assert calls_of(sg.sgqa_cache8_evict, dims=dims(), recent=0, **kw, **t) == 1
