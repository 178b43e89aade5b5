"""The group of quantised weights: that of the tiles given, or the one asked for."""
import pytest
import torch

import bloom_decoder_token_gb300 as bg


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("has", [32, 64, 128])
@pytest.mark.parametrize("asked", [32, 64, 128, 16, 0])
def test_another_group_than_that_of_the_tiles_is_refused(has, asked):
    w, out = torch.zeros(48, 512, dtype=torch.bfloat16), bg.W4.empty(48, 512, has, "cpu")
    # host tensors are refused too, behind this
    with pytest.raises(bg.BloomError, match="group" if asked != has else "CUDA device"):
        bg.op_w4_quantize(w, asked, out)


@pytest.mark.gpu
@pytest.mark.parametrize("has", [32, 64, 128])
def test_groups_of_the_tiles(has):
    w = torch.randn(48, 520, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    want = bg.op_w4_read(bg.op_w4_quantize(w, has))
    for group in (None, has):
        assert torch.equal(bg.op_w4_read(bg.op_w4_quantize(w, group, bg.W4.empty(48, 520, has))), want)
    assert bg.op_w4_quantize(w).group == 64
    with pytest.raises(bg.BloomError):
        bg.op_w4_quantize(w, {32: 64, 64: 128, 128: 32}[has], bg.W4.empty(48, 520, has))
    with pytest.raises(bg.BloomError):
        bg.op_w4_quantize(w, 0)
