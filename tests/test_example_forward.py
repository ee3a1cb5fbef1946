"""Which forward of the layer the example model scores with."""

import pytest

from mixture_experts_layer_deepseekmoe_amd import binding as moe
from mixture_experts_layer_deepseekmoe_amd import example as X


@pytest.mark.parametrize("T,kw,few", [(0, {}, True), (1, {}, True), (48, {}, True), (49, {}, False), (64, {}, False), (4096, {}, False),
                                      (1, dict(inter=32768), True), (1, dict(inter=32832), False)])
def test_scoring_takes_the_faster_call(T, kw, few):
    s = X.ModelShape(**kw)
    assert X.layer_forward(s, T) is (moe.moe_forward_few if few else moe.moe_forward)
    if few:   # it is within the call's limits
        assert moe.few_workspace_size(s.layer(T)) >= 0
