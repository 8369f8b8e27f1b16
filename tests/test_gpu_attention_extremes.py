"""GPU parity of attention and its gradients where a bias is large, against the fp64 oracle; bounds as in test_gpu_attention.

A constant added to the whole table changes no probability, so a table around +100, whose exponential no fp32 holds, is an
ordinary one.
"""
import numpy as np
import pytest

from test_gpu_attention import _case, _check, _make, _np, _run

pytestmark = pytest.mark.gpu

# a wave has 32 queries: counts that fill none, one or the last of them in part; over 1024 keys the gradients come from separate launches
PARTLY = [dict(nq=[40], nk=[128]), dict(nq=[77]), dict(nq=[1], nk=[300]), dict(nq=[3, 70, 33], nk=[200, 70, 150], heads=4, kv=2),
          dict(nq=[140], causal=True, width=128), dict(nq=[1], nk=[1100], heads=1, kv=1), dict(nq=[1101], heads=1, kv=1, width=24),
          dict(nq=[70], nk=[1150], causal=True, heads=1, kv=1, width=72), dict(nq=[90], nk=[60], causal=True, window=20)]


def _with_bias(c, t, val, table):
    """The case with this table (buckets, same for every head) for the distances below, within and above the reach."""
    import torch
    reach = c["reach"]
    t["map"] = torch.ones(2 * reach + 1, dtype=torch.int32, device="cuda")
    t["map"][0], t["map"][-1] = 0, 2
    t["bias"] = torch.tensor(table, device="cuda")[:, None].expand(-1, c["heads"]).to(t["q"].dtype).contiguous()
    return t, {**val, "map": t["map"].cpu().numpy(), "bias": _np(t["bias"])}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", PARTLY, ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()).replace(" ", ""))
@pytest.mark.parametrize("reach", [3, 64, 1200])
def test_a_large_bias_in_partly_filled_waves(gpu_lib, shape, reach, dtype):
    c = _case(dtype=dtype, buckets=3, reach=reach, **shape)
    t, val = _make(c)
    for table in ([100.0, 0.5, -0.25], [0.5, 100.0, -0.25], [0.5, -0.25, 100.0], [100.5, 99.0, 101.0]):
        t, val = _with_bias(c, t, val, table)
        _check(c, _run(gpu_lib, c, t), val)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_buckets_of_distances_that_no_pair_has_reach_nothing(gpu_lib, value, dtype):
    # 40 queries at the end of 128 keys: distances -127 .. 39; the places of a wave behind its last query would have the next ones
    import torch
    c = _case(dtype=dtype, nq=[40], nk=[128], buckets=3, reach=135)
    t, val = _make(c)
    t["map"] = torch.zeros(271, dtype=torch.int32, device="cuda")
    t["map"][100:135] = 1
    clean, _ = _with_bias(c, dict(t), val, [0.25, -0.5, value])
    clean["map"] = t["map"]
    want = _run(gpu_lib, c, clean)
    _check(c, want, {**val, "map": t["map"].cpu().numpy(), "bias": np.where(np.isfinite(_np(clean["bias"])), _np(clean["bias"]), 0.0)})
    clean["map"] = t["map"].clone()
    clean["map"][:135 - 127] = clean["map"][135 + 40:] = 2
    got = _run(gpu_lib, c, clean)
    for k in ("out", "lse", "q", "k", "v", "bias"):
        assert torch.equal(want[k], got[k]), k
