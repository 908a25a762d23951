"""Decode calls behind kernels that write their inputs: the library's kernels
start while the ones in front of them run, and have to wait for what these write."""
import pytest
import torch

from sparse_attention_top_idx_gb300 import dsaidx, latent
from sparse_attention_top_idx_gb300 import workloads as wl
from tests.parity import build_cache, decode_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("between", ["nothing", "store", "append", "rope"])
def test_lengths_staged_right_before_the_call(between):
    """The sequence lengths are the last bytes of a 64 MB copy from pinned host
    memory, which takes many times as long as a launch; the calls behind it
    are issued at once.  Every step's selection is that of its own lengths."""
    W = wl.make_workload("staged", [2000, 1500, 3000, 700], [1] * 4, topk=64, seed=5)
    cache = build_cache(W, dsaidx.FP8)
    ins = decode_inputs(W)
    ws = dsaidx.new_workspace(dsaidx.workspace_bytes_decode(cache, 4, 3000, W.H, 64))
    lens = [[2000, 10, 3000, 1], [5, 1500, 64, 700], [1999, 0, 1, 699], [200, 1400, 2900, 65]]
    n = 1 << 26
    hosts = [torch.zeros(n, dtype=torch.uint8).pin_memory() for _ in lens]
    for h, x in zip(hosts, lens):
        h[-16:] = torch.tensor(x, dtype=torch.int32).view(torch.uint8)
    stage = torch.zeros(n, dtype=torch.uint8, device="cuda")
    seq_lens = stage[-16:].view(torch.int32)

    def decode(sl, out):
        dsaidx.score_topk_decode(cache, ins["q"], ins["w"], ins["block_table"], sl, 3000, 64, out, ws)

    want = []
    for x in lens:
        out = torch.full((4, 64), -7, dtype=torch.int32, device="cuda")
        decode(torch.tensor(x, dtype=torch.int32, device="cuda"), out)
        torch.cuda.synchronize()
        want.append(out)
    keys = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")
    none = torch.full((1,), -1, dtype=torch.int64, device="cuda")       # no slot: nothing is stored
    records = latent.LatentCache.allocate(1, 64)
    c, pe = torch.zeros(1, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    plan, x, pos = latent.rope_plan(64), torch.zeros(1, 1, 64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    got = [torch.full((4, 64), -7, dtype=torch.int32, device="cuda") for _ in lens]
    torch.cuda.synchronize()
    for h, out in zip(hosts, got):
        dsaidx.copy(stage, h)
        if between == "store":
            dsaidx.store_keys(cache, keys, none)
        elif between == "append":
            latent.latent_append(records, c, pe, None, none, None)
        elif between == "rope":
            latent.rope(x, pos, plan)
        decode(seq_lens, out)
    torch.cuda.synchronize()
    assert dsaidx.read_device_status(ws) == 0
    for out, w in zip(got, want):
        assert torch.equal(out, w)
