"""Calls that the documentation allows in forms that users meet: other dtypes of a
buffer, the first call of a process inside a capture, and so on."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_e4m3_codes_into_torch_s_own_type(cuda_lib):
    csd = cuda_lib
    x = torch.randn((2, 3, 64, 128), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    pos = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    want, want_scale = csd.csa_head_norm_rope_e4m3(x, pos)
    codes = torch.empty((2, 3, 64, 128), dtype=torch.float8_e4m3fn, device="cuda")
    got, scale = csd.csa_head_norm_rope_e4m3(x, pos, codes=codes)
    assert got is codes and torch.equal(got.view(torch.uint8), want) and torch.equal(scale, want_scale)
    with pytest.raises(ValueError, match="codes"):
        csd.csa_head_norm_rope_e4m3(x, pos, codes=torch.empty((2, 3, 64, 128), dtype=torch.int8, device="cuda"))
