"""An explicit stream of the segmented products has to be on the operands' GPU
(no GPU is needed: the refusal comes before any call)."""
import types

import pytest
import torch

from dense_fp16_gemm_f16_amd import segments


@pytest.mark.parametrize("index", [1, 7])
def test_a_stream_of_another_gpu_is_refused(index):
    other = types.SimpleNamespace(device=torch.device("cuda", index), cuda_stream=0x1234)
    called = []
    with pytest.raises(ValueError, match="stream"):
        segments._launch(torch.device("cuda", 0), other, called.append)
    assert not called
