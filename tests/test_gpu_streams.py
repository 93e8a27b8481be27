"""The binding's stream is the current one of a tensor's device, by either of
the two lookups."""

import pytest
import torch

from bit_nf4_quantized_absmax_amd import ops
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def test_stream_lookups(monkeypatch):
    t = torch.zeros(4, device=DEV)
    s = torch.cuda.Stream()
    handles = []
    for _ in range(2):
        handles.append(ops._stream(t))
        with torch.cuda.stream(s):
            assert ops._stream(t) == s.cuda_stream
        monkeypatch.setattr(ops, "_raw_stream", None)
    assert handles[0] == handles[1] == torch.cuda.current_stream().cuda_stream
    with pytest.raises(ValueError):
        ops._stream(t.cpu())
