"""A tensor that is not where x is, or an x that is on no GPU, is refused before the library
is called: it takes bare addresses, and one of host memory would fault the GPU."""

import pytest
import torch


class Refusing:
    """No entry point of the library may be reached."""

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *shape: 4096
        return lambda *args: pytest.fail(f"{name} was called")


@pytest.fixture
def w(monkeypatch):
    import w4a16_int4_weight_amd as m
    monkeypatch.setattr(m, "_lib", Refusing())
    m._need.cache_clear()
    yield m
    m._need.cache_clear()


def tensors():
    t = {"x": torch.zeros((4, 256), dtype=torch.bfloat16), "packed": torch.zeros(1 << 15, dtype=torch.uint8),
         "dy": torch.zeros((4, 64), dtype=torch.bfloat16), "labels": torch.zeros(4, dtype=torch.int32),
         "top_ids": torch.zeros((4, 3), dtype=torch.int32), "top_logits": torch.zeros((4, 3)),
         "workspace": torch.zeros(4096, dtype=torch.uint8), "h": torch.zeros((4, 64), dtype=torch.bfloat16),
         "dx": torch.zeros((4, 256), dtype=torch.bfloat16), "loss": torch.zeros(4), "lse": torch.zeros(4),
         "dloss": torch.ones(4)}
    t["dh"] = t["dy"]
    return t


CALLS = {
    "w4a16_gemm_grad": ("dy", ["packed", "dx", "workspace"],
                        lambda w, t: w.w4a16_gemm_grad(t["dy"], t["packed"], 256, dx=t["dx"], workspace=t["workspace"])),
    "w4a16_gated": ("x", ["packed", "h", "workspace"],
                    lambda w, t: w.w4a16_gated(t["x"], t["packed"], 64, h=t["h"], workspace=t["workspace"])),
    "w4a16_gated_grad": ("x", ["dh", "packed", "dx", "workspace"],
                         lambda w, t: w.w4a16_gated_grad(t["x"], t["dh"], t["packed"], 64, dx=t["dx"],
                                                         workspace=t["workspace"])),
    "w4a16_cross_entropy": ("x", ["labels", "packed", "dloss", "loss", "lse", "dx", "workspace"],
                            lambda w, t: w.w4a16_cross_entropy(t["x"], t["labels"], t["packed"], 1000, dloss=t["dloss"], grad=True,
                                                               loss=t["loss"], lse=t["lse"], dx=t["dx"], workspace=t["workspace"])),
    "w4a16_distill": ("x", ["top_ids", "top_logits", "packed", "dloss", "loss", "lse", "dx", "workspace"],
                      lambda w, t: w.w4a16_distill(t["x"], t["top_ids"], t["top_logits"], t["packed"], 1000, dloss=t["dloss"],
                                                   grad=True, loss=t["loss"], lse=t["lse"], dx=t["dx"], workspace=t["workspace"])),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_a_tensor_elsewhere(w, name):
    _, others, call = CALLS[name]
    for n in others:
        t = tensors()
        t[n] = t[n].to("meta")
        with pytest.raises(ValueError, match=f"^{n} must be on cpu, not on meta"):
            call(w, t)


@pytest.mark.parametrize("name", list(CALLS))
def test_everything_on_the_host(w, name):
    class Stream:
        cuda_stream = 0

    _, _, call = CALLS[name]
    with pytest.raises(ValueError, match="on a GPU"):
        call(w, tensors())
    with pytest.raises(ValueError, match="on a GPU"):
        w._launch(name, (), None, 0, torch.device("cpu"), Stream())
