"""The layer operators' binding without a GPU, at the ends of its arguments'
ranges."""
import torch

from delta_rule_linear_kla_b200 import autograd


def test_gradients_are_laid_out_for_the_library():
    """Autograd's view of a part of a concatenation is contiguous at any
    element: what the library gets is aligned and equal."""
    x = torch.randn(1, 5, 3, requires_grad=True)
    got = []
    x.register_hook(got.append)
    (torch.cat([torch.zeros(1, 5, 3), x], 1) * torch.randn(1, 10, 3)).sum().backward()
    g = got[0]
    assert g.is_contiguous() and g.data_ptr() % 16 == 12
    for dtype in (torch.float32, torch.bfloat16):
        a = autograd._given(g, dtype)
        assert a.is_contiguous() and a.data_ptr() % 16 == 0 and torch.equal(a, g.to(dtype))
    t = torch.randn(4, 6)
    assert autograd._given(t, torch.float32) is t and autograd._given(None, t.dtype) is None
    assert torch.equal(autograd._given(t.mT, t.dtype), t.mT)
