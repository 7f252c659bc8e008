"""What the Python binding of the calls around the cache refuses before it calls the
library (no GPU needed)."""
import math

import pytest

from tests.test_abi import K  # noqa: F401


def test_binding_refuses_host_tensors(K):
    import torch
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        K.norm_rope(x)
    with pytest.raises(ValueError):
        K.Norm(torch.ones(64))
    with pytest.raises(ValueError):
        K.Rope([1.0, 0.5], axes=[0])
    with pytest.raises(K.KvqError):
        K.Rope([math.nan])
    with pytest.raises(ValueError):
        K.diff_heads(x, torch.zeros(1))
    with pytest.raises(TypeError):
        K.norm_rope([1.0])


def test_module_refuses_wrong_calls(K):
    m = K.calls()
    for call in (lambda: m.norm_rope(1), lambda: m.load(None), lambda: m.init(1, 2), lambda: m.init((1, 2), None)):
        with pytest.raises(TypeError):
            call()
