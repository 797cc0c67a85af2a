"""What a refused size is told, of the layer and of calls with other rules."""
import pytest
import torch

import mxfp8_mxfp4_moe_gb300 as K


def test_the_text_of_a_refused_size_does_not_give_the_layers_rule_to_every_call():
    text = K.kmoe_status_string(2)
    assert "the layer: H and I must be multiples of 128" in text and "other calls: see their declaration" in text
    # widths of a product are multiples of 16, of the moves of 8
    lib = K.lib()
    assert lib.kmoe_permute(4096, 4096, 4, 60, 2, 0, 4096, None) == 2
    assert lib.kmoe_gemm_fp8(4096, 4096, 4096, 4096, None, 4, 40, 32, 1, 0, 4096, 4096, 256, None) == 2
    with pytest.raises(K.KmoeError, match="other calls: see their declaration"):
        raise K.KmoeError("kmoe_gemm_fp8", 2, lib)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):  # (before the sizes, in the binding)
        K.kmoe_permute(torch.zeros(4, 60, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32))
