"""What the Python binding of the calls over several sequences refuses before it calls the
library (no GPU needed)."""
import pytest

from tests.test_abi import K  # noqa: F401


def test_binding_refuses(K):
    import torch
    q = torch.zeros(2, 4, 64)
    ints = torch.zeros(2, dtype=torch.int32)
    cache = type("C", (), {"handle": (1, 0)})()
    with pytest.raises(ValueError):  # on the host
        K.decode_local(cache, q, ints, ints.reshape(2, 1), 1, 1.0, 0)
    with pytest.raises(ValueError):
        K.attn_seqs(cache, q, torch.zeros(3, dtype=torch.int32), ints, ints.reshape(2, 1), 1, 1, 1.0)
    with pytest.raises(TypeError):
        K.decode_local(cache, [1.0], ints, ints.reshape(2, 1), 1, 1.0, 0)
    with pytest.raises(ValueError):
        K.decode_local(cache, q[0], ints, ints.reshape(2, 1), 1, 1.0, 0)
