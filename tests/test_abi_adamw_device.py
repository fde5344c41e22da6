"""CPU check of the device that the optimizer step's table is written to: nothing but a GPU is taken, whatever memory
the tensors are in, before any of it is allocated."""

import pytest
import torch


@pytest.mark.parametrize("device", ["cpu", "cpu:0", "meta", torch.device("cpu"), torch.device("cpu", 0)])
@pytest.mark.parametrize("eight", [True, False])
def test_the_table_is_written_to_a_gpu_only(device, eight):
    import bit_quantized_fine_qlora_amd as Q
    f, g = torch.zeros(256), torch.zeros(256, dtype=torch.bfloat16)
    mv = [Q.alloc_moment8(256, signed, device="cpu") for signed in (True, False)] if eight else [f.clone(), f.clone()]
    with pytest.raises(ValueError, match="device: must be a GPU"):
        Q.AdamWStep([(f, None, g, *mv)], device=device)
