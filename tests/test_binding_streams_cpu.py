"""Which streams the binding hands to the library, without a GPU."""
import os
from types import SimpleNamespace

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_stream_of_another_device_is_refused():
    """Tensors on one device, work put on another's stream: the kernels would run there."""
    if not os.path.exists(os.path.join(ROOT, "balanced_token_dispatch_amd", "libmoe.so")):
        pytest.skip("libmoe.so not built")
    import balanced_token_dispatch_amd as m
    assert m._on(1, SimpleNamespace(device_index=1, cuda_stream=77)) == 77
    for dev, of in ((0, 1), (1, 0)):
        with pytest.raises(m.MoeError, match="stream"):
            m._on(dev, SimpleNamespace(device_index=of, cuda_stream=77))
