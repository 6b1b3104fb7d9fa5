"""decode and decode8 captured over one workspace and replayed in turn."""

import pytest
import torch

import grouped_query_attention_attn_b200 as gqa
from test_gpu_cache8 import bf16, ints, make, to_gpu

pytestmark = pytest.mark.gpu


def test_graphs_of_both_decodes_share_a_workspace(gqa_lib):
    lens = [3000, 100, 0, 1500]
    rng, p, table = make(12, "e4m3", 2, 128, 64, 64, lens)
    c, t, n, q = to_gpu(p), ints(table), ints(lens), bf16(rng, (4, 8, 128)).cuda()
    k, v = gqa.cache8_read(c, t, n, 3008)
    size = max(gqa.decode8_workspace_size(4, 8, 2, 128, t.shape[1] * 64), gqa.decode_workspace_size(4, 8, 2, 128, 3008))
    ws = torch.randint(0, 255, (size,), dtype=torch.uint8, device="cuda")
    want = [gqa.decode8(q, c, t, n), gqa.decode(q, k, v, n)]
    outs, graphs = [torch.empty_like(q) for _ in range(2)], []
    for i, o in enumerate(outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gqa.decode(q, k, v, n, workspace=ws, out=o) if i else gqa.decode8(q, c, t, n, workspace=ws, out=o)
        graphs.append(g)
    for i in (0, 1, 0, 0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])
    gqa.device_status()
