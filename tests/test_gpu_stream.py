"""The stream that calls are launched on is the device's current one, also
with a torch that lacks the undocumented function for it."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("documented", [False, True])
def test_current_stream(documented, monkeypatch):
    import bit_quantized_fine_qlora_amd as Q
    from bit_quantized_fine_qlora_amd import api
    print(f"[case] current stream, documented interface only {documented}", flush=True)
    assert hasattr(api, "_raw_stream")
    if documented:
        monkeypatch.setattr(api, "_raw_stream", None)
    x = torch.randn((64, 256), device="cuda").to(torch.bfloat16)
    want = Q.checkpoint_pack(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            for device in (None, x.device, torch.device("cuda")):
                assert api._stream(device) == stream.cuda_stream
            got = Q.checkpoint_pack(x)
        torch.cuda.current_stream().wait_stream(stream)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
