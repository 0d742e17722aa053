"""What the binding says about arguments that are no GPU tensors. No GPU is
needed: nothing here reaches the library."""
import pytest
import torch

from zero_sharded_mixed_pad_amd import binding


class OnGpu(torch.Tensor):
    """A host tensor that passes for one on the GPU: the buffers before the bad
    one are good."""
    is_cuda = True


def grad(n=8, dtype=torch.float32):
    return torch.zeros(n, dtype=dtype).as_subclass(OnGpu)


def test_gradient_arrays():
    g = [grad(), grad(9)]
    arr, code = binding._grad_array(g, 2, 8)
    assert list(arr) == [x.data_ptr() for x in g] and code == binding.F32
    assert binding._grad_array([grad(dtype=torch.bfloat16)], 1)[1] == binding.BF16


@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("bad", [None, 3, "g", [1.0]])
def test_a_gradient_that_is_no_tensor_is_named(bad, at):
    g = [grad(), grad(), grad()]
    g[at] = bad
    with pytest.raises(TypeError, match=rf"^grads\[{at}\] must be a torch tensor$"):
        binding._grad_array(g, 3, 8)


@pytest.mark.parametrize("bad,kind,says", [
    (grad(7), ValueError, r"grads\[1\] holds 7 elements; this layout reads 8"),
    (grad(16)[::2], ValueError, r"grads\[1\] must be contiguous"),
    (grad(dtype=torch.bfloat16), TypeError, r"grads\[1\] must be torch.float32"),
    (torch.zeros(8), ValueError, r"grads\[1\] must be on the GPU"),
])
def test_a_gradient_that_does_not_fit_is_named(bad, kind, says):
    with pytest.raises(kind, match=says):
        binding._grad_array([grad(), bad], 2, 8)


@pytest.mark.parametrize("bad", [None, 3, [1.0, 2.0]])
def test_a_record_that_is_no_tensor_is_named(bad):
    with pytest.raises(TypeError, match="^clip must be a torch tensor$"):
        binding._rec(bad, "clip")
    with pytest.raises(TypeError, match="^parts must be a torch tensor$"):
        binding.zsp_clip_combine(bad, torch.zeros(1, 2, dtype=torch.float64))


@pytest.mark.parametrize("bad,kind,says", [
    (torch.zeros(1, 2), TypeError, "clip must be torch.float64"),
    (torch.zeros(2, 2, dtype=torch.float64).t(), ValueError, "clip must be contiguous"),
    (torch.zeros(1, 2, dtype=torch.float64), ValueError, "clip must be on the GPU"),
])
def test_a_record_that_does_not_fit_is_named(bad, kind, says, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(kind, match=says):
        binding._rec(bad, "clip")
