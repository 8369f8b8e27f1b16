"""GPU parity of the bias's gradient where its partial sums would pass half a gigabyte, so that grad_q goes over the units in batches."""
import pytest

from test_gpu_attention import NAN, _case, _check, _form, _make, _run

pytestmark = pytest.mark.gpu

# in order up to 512 sequences, by a stride beyond; few heads and many
SHAPES = [dict(nq=[1, 4, 2] * 100, nk=[3, 4, 5] * 100, heads=16, kv=4, reach=4096, causal=True), dict(nq=[2, 3] * 350, heads=8, kv=4, reach=4096),
          dict(nq=[130, 0, 1] * 30, heads=64, kv=4, reach=3000, window=40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s['nq'])}x{s['heads']}x{s['reach']}")
def test_batches_of_units(gpu_lib, shape, dtype):
    import torch
    c = _case(**{**dict(width=16, dtype=dtype, buckets=40), **shape})
    t, val = _make(c)
    need = gpu_lib.muon_attention_backward_workspace_bytes(t["q"], t["k"], bias=t["bias"], bucket_map=t["map"], sequences=len(c["nq"]))
    # in one go: a slot for each of the 4 waves of a unit, at least one unit a sequence and 128 queries
    units = sum(c["nq"]) // 128 + len(c["nq"])
    assert units * 4 * c["heads"] * (2 * c["reach"] + 1) * 4 > 1 << 29 > need - (1 << 24)
    o = _run(gpu_lib, c, t)
    _check(c, o, val)
    # the same bits again, with a workspace that holds NaN, and in a graph that is replayed
    ws = torch.full((max(need, gpu_lib.muon_attention_workspace_bytes(t["q"], t["k"], sequences=len(c["nq"]))),), 255, dtype=torch.uint8, device="cuda")
    again = _run(gpu_lib, c, t, workspace=ws)
    names = ("q", "k", "v", "bias")
    assert all(torch.equal(o[k], again[k]) for k in names)
    form = dict(_form(c, t), out_low=o["low"], workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.muon_attention_backward(t["q"], t["k"], t["v"], o["out"], o["lse"], t["do"], *(again[k] for k in ("q", "k", "v")), grad_bias=again["bias"],
                                        **form)
    for _ in range(3):
        for k in names:
            again[k].fill_(NAN)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], again[k]) for k in names)
