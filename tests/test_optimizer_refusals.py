"""block.AdamW on the CPU: a step that is refused is not counted."""

import pytest
import torch


def test_a_refused_step_is_not_counted():
    from mixture_experts_layer_pft_gb300 import block, build

    build.build()
    p = [torch.zeros(300), torch.zeros(8, dtype=torch.bfloat16)]
    for bits in (32, 8):
        o = block.AdamW(p, [torch.zeros_like(t) for t in p], lr=1e-3, bits=bits)
        for _ in range(2):
            with pytest.raises(ValueError):  # not on a CUDA device
                o.step()
        assert int(o.step_count) == 0
