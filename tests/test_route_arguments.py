"""Numbers that the binding of route must not pass on: no result is allocated for them, and none
becomes another one in 32 bits.  No GPU is needed."""
import pytest
import torch

import dense_fp16_gemm_f16_amd as g


@pytest.mark.parametrize("fan,how", [
    (0, {}), (-1, {}), (33, {}), (1 << 40, {}), ((1 << 64) + 2, {}),
    (2, {"groups": 0}), (2, {"groups": 65}), (2, {"groups": (1 << 32) + 2}), (2, {"groups": -(1 << 32) + 2}),
    (2, {"groups": 4, "top_groups": 0}), (2, {"groups": 4, "top_groups": (1 << 32) + 1}),
    (2, {"groups": 4, "group_top": 3}), (2, {"groups": 4, "group_top": (1 << 32) + 2}),
])
def test_numbers_out_of_range_are_refused(fan, how):
    with pytest.raises(g.GemmError) as e:
        g.route(torch.zeros(4, 64), fan, **how)
    assert e.value.status == g.EINVAL
