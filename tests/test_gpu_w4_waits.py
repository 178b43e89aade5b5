"""The 4-bit linear layer's bounded waits at a few tokens: long runs of tiles from HBM behind a bound that runs out."""
import pytest
import torch

import bloom_decoder_token_gb300 as bg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("M,n,k", [(1, 250880, 4096), (8, 250880, 4096), (2, 250880, 4608), (1, 60000, 33000)])
def test_waits_run_out(M, n, k):
    """Tiles that come from HBM four at a time: some wait of 20 ns runs out.  The call ends, says so, writes NaN or what
    it always does, and the next call is whole.  One CTA, clusters, and several passes over the rows."""
    g = torch.Generator(device=DEV).manual_seed(n + k)
    w = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    for a in range(0, n, 16384):
        w[a: a + 16384] = torch.randn(min(16384, n - a), k, generator=g, device=DEV) * 0.02
    w4, x = bg.op_w4_quantize(w, 64), torch.randn(M, k, generator=g, device=DEV).to(torch.bfloat16)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    want, lost = bg.op_linear_w4(x, w4, flag=flag), 0
    assert flag.item() == 0
    try:
        assert bg.lib().bloom_op_linear_w4_wait_ns(20) == 0
        for _ in range(10):
            flush.zero_()
            flag.zero_()
            got = bg.op_linear_w4(x, w4, flag=flag)
            torch.cuda.synchronize()
            nan = torch.isnan(got)
            assert flag.item() == (8 if nan.any() else 0)
            assert torch.equal(torch.where(nan, want, got), want)
            lost += int(nan.any())
    finally:
        assert bg.lib().bloom_op_linear_w4_wait_ns(0) == 0
    assert lost > 0
    flag.zero_()
    assert torch.equal(bg.op_linear_w4(x, w4, flag=flag), want) and flag.item() == 0
