"""GPU: what follows an eviction in its stream sees all of its results, also when the
call moves nothing."""
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from pkvq_ref64 import D, random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [pk.KV_INT8_BLOCK, pk.KV_FP8_E4M3])
@pytest.mark.parametrize("lens", [[0] * 64, [0] * 63 + [5]])
def test_results_of_empty_sequences_are_ordered(fmt, lens):
    """Long result rows to clear, few or no tokens to move; copies and a decode
    step (which starts early, behind the last kernel of its stream) follow at once."""
    B, H, budget = len(lens), 4, 4096
    cache = random_cache(fmt, 300, 16, H, 111)
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    dst = (100 + torch.arange(B, device="cuda").to(torch.int32))[:, None].expand(B, 256).contiguous()
    W = torch.ones((B, H, 16), device="cuda")
    q = torch.randn((B, 1, H, D), device="cuda").half()
    for _ in range(10):
        wout = torch.full((B, H, 20_000), 7.0, device="cuda")
        keep = torch.full((B, H, budget), 7, dtype=torch.int32, device="cuda")
        new = torch.full((B,), 9, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        pk.kv_evict(cache, W, table, ctx, dst, budget, weights_out=wout, keep=keep, new_context_lens=new)
        out = pk.paged_attn_decode(cache, q, dst, new, 16, 1.0)
        seen = new.clone(), keep.clone(), wout.clone()
        torch.cuda.synchronize()
        assert seen[0].tolist() == lens
        assert (out[ctx == 0] == 0).all()
        for b in {0, B - 1}:
            n = lens[b]
            assert (seen[1][b, :, :n] == torch.arange(n, device="cuda")).all() and (seen[1][b, :, n:] == -1).all()
            assert (seen[2][b, :, :n] == 1).all() and (seen[2][b, :, n:] == 0).all()
        assert (seen[1][:B - 1] == -1).all() and (seen[2][:B - 1] == 0).all()
    assert pk.device_status() == 0
