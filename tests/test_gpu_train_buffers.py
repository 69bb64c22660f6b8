"""A layer's own output buffers handed back to it (needs a B200)."""
import pytest
import torch

from test_gpu_train_layer import _cfg, _layer

pytestmark = pytest.mark.gpu


def test_forward_train_refuses_its_backward_s_output():
    """backward() writes dx before it last reads x, so x must not be that buffer:
    refused before anything is computed, not after half of the gradients."""
    inp, layer = _layer(_cfg("tiny"))
    layer.forward_train(inp.x)
    dx = layer.backward(inp.x, layer.grad_buffers())
    before = dx.clone()
    with pytest.raises(ValueError, match="backward overwrites"):
        layer.forward_train(dx)
    with pytest.raises(ValueError, match="backward overwrites"):
        layer.forward_train(dx[:3])
    assert torch.equal(dx, before)


@pytest.mark.parametrize("name", ["tiny", "noshared", "wide"])
def test_own_buffers_as_the_gradient(name):
    """y, and an earlier dx, may be dy (the gradient of sum(y^2) / 2 is y)."""
    inp, layer = _layer(_cfg(name))
    y = layer.forward_train(inp.x)
    grads, want = layer.grad_buffers(), layer.grad_buffers()
    dx = layer.backward(y, grads).clone()
    layer.forward_train(inp.x)
    assert torch.equal(layer.backward(y.clone(), want), dx)
    for k in want:
        assert torch.equal(grads[k], want[k])
    layer.forward_train(inp.x)
    got = layer.backward(layer._train["dx"], grads).clone()
    layer.forward_train(inp.x)
    assert torch.equal(layer.backward(dx, want), got)
    for k in want:
        assert torch.equal(grads[k], want[k])


def test_a_permutation_ends_forward_train_s_claim():
    """permute() on its own (a stage of the forward) writes over the rows that
    backward() needs."""
    inp, layer = _layer(_cfg("tiny"))
    layer.forward_train(inp.x)
    layer.permute((inp.x * 2).contiguous(), inp.x.shape[0])
    with pytest.raises(ValueError, match="without forward_train"):
        layer.backward(inp.x, layer.grad_buffers())
