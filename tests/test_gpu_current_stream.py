"""A call without a stream goes to the current one, with or without torch's short way to its handle."""
import pytest
import torch

from combine_ep_route_amd import ep as binding
from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("short", [True, False])
def test_current_stream(short, monkeypatch):
    need_gpu()
    say(f"current stream, {'torch._C' if short else 'torch.cuda'}")
    if not short:
        monkeypatch.setattr(binding, "_raw_stream", None)
    assert binding._stream(None) == torch.cuda.current_stream().cuda_stream
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert binding._stream(None) == s.cuda_stream
    assert binding._stream(s) == s.cuda_stream
    assert binding._stream(None) == torch.cuda.current_stream().cuda_stream
