"""Read-back into views of every order: K and V side by side in one buffer, tokens, rows
or heads outermost, slices with room between."""
import pytest
import torch

import bloom_decoder_token_gb300 as bg

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, T, N, D, S = 3, 37, 4, 64, 96


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def views():
    mk = lambda *shape: torch.full(shape, 7.0, dtype=torch.bfloat16, device=DEV)
    x = mk(B, T, N, 3, D)
    yield "fused", x, x[:, :, :, 1], x[:, :, :, 2]
    x = mk(2, B, N, T + 5, D + 8)
    yield "heads", x, x[0, :, :, 2:T + 2, :D].transpose(1, 2), x[1, :, :, 5:, 8:].transpose(1, 2)
    x = mk(T, N, B, 2 * D)
    yield "tokens outermost", x, x[..., :D].permute(2, 0, 1, 3), x[..., D:].permute(2, 0, 1, 3)
    x = mk(N, 2, T, B, D)
    yield "heads outermost", x, x[:, 0].permute(2, 1, 0, 3), x[:, 1].permute(2, 1, 0, 3)


def test_read_back_into_views():
    g = torch.Generator().manual_seed(1)
    kv = bg.KV8.empty(B, N, S, D, torch.int8, DEV)
    z = torch.zeros(B, dtype=torch.int32, device=DEV)
    bg.op_kv8_write(kv, *(torch.randn(2, B, S, N, D, generator=g).to(torch.bfloat16).to(DEV)), z)
    start = torch.tensor([0, 31, 59], dtype=torch.int32, device=DEV)
    want = bg.op_kv8_read(kv, start, T)
    for name, buf, k, v in views():
        bg.op_kv8_read(kv, start, T, k=k, v=v)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1]), name
        k.fill_(7.0)
        v.fill_(7.0)
        assert (buf == 7).all(), name        # nothing beside the views
