"""The layer example: generation on pools after a prefill against one prefill of everything, and the gradients of
its three operators together by differences."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_generation_continues_the_prefill():
    from examples import generate
    off, grads = generate.run()
    assert off < 1e-2   # the chunked form's budget
    assert all(torch.isfinite(t).all() for t in grads.values())


def test_gradients_of_the_layer_by_differences():
    """The derivative of sum(o do) along the weights of the norm, from the layer's backward and from two forwards with the
    weights moved: the difference quotient's own error is the outputs' rounding (2^-9 each, of random sign) over the step."""
    import numpy as np
    from examples import generate
    layer = generate.Layer(H=2, HV=4, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    T, cu = 96, np.array([0, 40, 96], np.int32)
    rows = torch.randn((T, layer.C), generator=gen, device="cuda").to(torch.bfloat16)
    g = torch.nn.functional.logsigmoid(2 + 4 * torch.rand((T, layer.HV), generator=gen, device="cuda"))
    beta = torch.rand((T, layer.HV), generator=gen, device="cuda")
    o = layer.prefill(rows, g, beta, cu)
    do = torch.randn(o.shape, generator=gen, device="cuda").to(torch.bfloat16)
    grads = layer.backward(do)
    for name in ("wq", "wk"):
        w = getattr(layer, name)
        way = torch.randn(w.shape, generator=gen, device="cuda")
        along = float((grads[name].double() * way.double()).sum())
        ends = []
        for h in (0.05, -0.05):
            setattr(layer, name, w + h * way)
            ends.append(float((layer.prefill(rows, g, beta, cu).double() * do.double()).sum()))
        setattr(layer, name, w)
        quotient = (ends[0] - ends[1]) / 0.1
        noise = 2 ** -8 * float((o.double() * do.double()).norm()) / 0.1
        assert abs(along - quotient) < 6 * noise + 0.02 * abs(quotient), (name, along, quotient, noise)
