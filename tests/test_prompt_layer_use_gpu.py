"""PromptLayer as a program uses it: weights that are parameters, grad and inference modes."""

import pytest
import torch

from mla_latent_kv_45_b200 import _lib as L
from mla_latent_kv_45_b200 import build, synth
from mla_latent_kv_45_b200.layer import DecodeLayer, PromptLayer
from mla_testlib import dev, dev_weights, lib_dims

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    L.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


SIZES = {
    "fp32": synth.TINY,
    "bf16": synth.reduced(synth.V2_STEP128, "prompt", 94, 1, 0, 0, d_model=1024, d_q=512),
}
N = 20


def case(name):
    wl = SIZES[name]
    dims, Wd = lib_dims(wl), dev_weights(synth.make_weights(wl), wl)
    ps = wl.page_size
    pages = -(-(N + 1) // ps)
    pool = torch.zeros(pages, ps, wl.row, dtype=dims.torch_dtype, device="cuda")
    cache = L.PagedCache(pool, i32([list(range(pages))]), None)
    return wl, dims, Wd, cache, dev(synth.make_hidden(wl, n=N), wl)


def prompt(dims, W, cache, h):
    layer = PromptLayer(dims, W, 1, N, N)
    out = layer.step(cache, h, i32([0, N]), None, i32([0, N])).clone()
    assert layer.device_error() == 0
    return layer, out


@pytest.mark.parametrize("name", SIZES)
def test_weights_and_inputs_that_require_a_gradient(name):
    """The layer takes a model's parameters as DecodeLayer does, and records nothing."""
    wl, dims, Wd, cache, h = case(name)
    _, want = prompt(dims, Wd, cache, h)
    params = {k: None if v is None else torch.nn.Parameter(v.clone()) for k, v in Wd.items()}
    layer, out = prompt(dims, params, cache, h.clone().requires_grad_())
    assert torch.equal(out, want) and not layer.step(cache, h, i32([0, N]), None, i32([0, N])).requires_grad
    g = layer.capture(cache, h, i32([0, N]), None, i32([0, N]))
    layer.out.zero_()
    assert torch.equal(g.replay(), want)
    cache.seq_lens = i32([N + 1])
    dec = DecodeLayer(dims, params, 1)
    assert torch.isfinite(dec.step(cache, h[-1:].contiguous(), i32([N]))).all()


@pytest.mark.parametrize("made,used", [(False, True), (True, False), (True, True)])
def test_inference_mode(made, used):
    wl, dims, Wd, cache, h = case("bf16")
    _, want = prompt(dims, Wd, cache, h)
    with torch.inference_mode(made):
        layer = PromptLayer(dims, {k: None if v is None else v.clone() for k, v in Wd.items()}, 1, N, N)
    with torch.inference_mode(used):
        out = layer.step(cache, h, i32([0, N]), None, i32([0, N]))
        assert torch.equal(out, want)
    assert layer.device_error() == 0


def test_error_of_a_step_on_another_stream():
    """The status is that of all steps, those that other streams have not come to as well."""
    wl, dims, Wd, cache, h = case("fp32")
    layer = PromptLayer(dims, Wd, 1, N, N)
    side = torch.cuda.Stream()
    cu, bad = i32([0, N]), i32([0, N + 1])
    torch.cuda.synchronize()
    for offsets, want in ((bad, 6), (cu, 0), (bad, 6)):
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)      # about a tenth of a second
        layer.step(cache, h, cu, None, offsets, side)
        assert layer.device_error() == want
    g = layer.capture(cache, h, cu, None, bad)
    assert layer.device_error() == 6
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        g.replay()
    assert layer.device_error() == 6


def test_what_uses_the_current_device_does_so_on_the_layers(monkeypatch):
    """One GPU stands for several here: the layer makes its own device current wherever it or
    the binding asks for the current stream."""
    wl, dims, Wd, cache, h = case("fp32")
    inside = []

    class Device(torch.cuda.device):
        def __enter__(self):
            inside.append(self.idx)
            return super().__enter__()

        def __exit__(self, *a):
            inside.pop()
            return super().__exit__(*a)

    seen = []

    def noted(name, f):
        def g(*a, **k):
            seen.append((name, inside[-1:] == [0]))
            return f(*a, **k)
        return g

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(L, "mla_workspace_init", noted("init", L.mla_workspace_init))
    monkeypatch.setattr(L, "mla_get_device_error", noted("error", L.mla_get_device_error))
    monkeypatch.setattr(torch.cuda, "synchronize", noted("synchronize", torch.cuda.synchronize))
    monkeypatch.setattr(torch.cuda, "CUDAGraph", noted("graph", torch.cuda.CUDAGraph))
    layer = PromptLayer(dims, Wd, 1, N, N)
    g = layer.capture(cache, h, i32([0, N]), None, i32([0, N]))
    g.replay()
    assert layer.device_error() == 0
    assert {n for n, _ in seen} == {"init", "error", "synchronize", "graph"}
    assert all(ok for _, ok in seen), seen
