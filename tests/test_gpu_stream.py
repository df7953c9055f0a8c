"""The stream that the binding hands to the library is torch's current one."""

import pytest
import torch

from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu


def test_stream_is_torchs_current_one():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = torch.zeros(1, device="cuda")

    def check():
        assert av._stream() == torch.cuda.current_stream().cuda_stream
        assert av._stream_on(x) == torch.cuda.current_stream().cuda_stream
    check()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        check()
        with torch.cuda.stream(b):
            check()
            with torch.cuda.device(0):
                check()
        check()
    with torch.cuda.device(0):
        check()
        with torch.cuda.stream(b):
            check()
    check()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        check()                    # the capture's own stream
        x.zero_()
    with pytest.raises(ValueError, match="current GPU"):
        av._stream_on(torch.zeros(1))
