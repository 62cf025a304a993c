"""What is no dense tensor in a list of gradients is named in the refusal."""
import pytest
import torch

import transformer_reduce_gb300 as L


@pytest.mark.parametrize("entry", [None, 1.0, [1.0]])
def test_entries_that_are_no_tensors_are_refused(entry):
    g = torch.zeros(4)
    for call in (lambda x: L.grad_norm(x), lambda x: L.grad_clip(x, 1.0)):
        with pytest.raises(TypeError, match=r"grads\[1\] is no tensor"):
            call([g, entry, g])
    with pytest.raises(TypeError, match=r"grads\[0\] is no tensor"):
        L.grad_norm([entry])


def test_outputs_that_are_no_tensors_are_refused():
    class OnGpu:
        """A tensor that says it is on a GPU, for the checks of the outputs."""
        is_cuda = True

        def __init__(self):
            self.t = torch.zeros(4)

        def __getattr__(self, name):
            return getattr(self.t, name)

    g = OnGpu()
    with pytest.raises(TypeError, match=r"out\[1\] is no tensor"):
        L.grad_clip([g, g], 1.0, out=[g, None])
