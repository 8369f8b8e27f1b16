"""GPU parity of attention and its gradients where a bias is large, against the fp64 oracle; bounds as in test_gpu_attention.

A constant added to the whole table changes no probability, so a table around +100, whose exponential no fp32 holds, is an
ordinary one.
"""
import numpy as np
import pytest

from test_gpu_attention import U, _bounds, _case, _check, _make, _near, _np, _reference, _run

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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 100.0])
@pytest.mark.parametrize("reach", [135, 70])
def test_buckets_of_distances_that_only_masked_keys_have_reach_nothing(gpu_lib, reach, value, dtype):
    # the first 64 of 128 keys are padding: 40 queries see distances -63 .. 39, places behind the last one would have some to -87
    import torch
    c = _case(dtype=dtype, nq=[40], nk=[128], buckets=3, reach=reach)
    t, val = _make(c)
    t["mask"] = torch.arange(128, device="cuda") >= 64
    got = []
    for v in (0.125, value):
        p, v2 = _with_bias(c, dict(t), val, [0.25, -0.5, v])
        p["map"] = torch.zeros(2 * reach + 1, dtype=torch.int32, device="cuda")
        p["map"][reach - 63:reach] = 1
        p["map"][:reach - 63] = 2
        got.append(_run(gpu_lib, c, p))
        if v == 0.125:
            _check(c, got[0], {**v2, "map": p["map"].cpu().numpy(), "mask": t["mask"].cpu().numpy()})
    for k in ("out", "lse", "q", "k", "v", "bias"):
        assert torch.equal(got[0][k], got[1][k]), k


@pytest.mark.parametrize("causal", [False, True])
def test_a_window_over_as_many_keys_as_there_may_be(gpu_lib, causal):
    # one query behind 2^30 - 1 keys, all of them one broadcast row: key positions and windows that sum to more than 2^31
    import torch
    n, width = 1 << 30, 8
    if torch.cuda.mem_get_info()[0] < 3 * n * width * 2:
        pytest.skip("needs 52 GB")
    r = np.random.default_rng(3)
    put = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).bfloat16().cuda()
    q, k, v, do = put(1, 1, width), put(1, 1, width), put(1, 1, width), put(1, 1, width)
    keys, values = k.expand(n, 1, width), v.expand(n, 1, width)
    gk, gv = (torch.full((n, 1, width), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out, lse, gq = torch.full_like(q, float("nan")), torch.full((1, 1), float("nan"), device="cuda"), torch.full_like(q, float("nan"))
    form = dict(causal=causal, window=n - 1, scale=0.25)
    gpu_lib.muon_attention(q, keys, values, out, lse, **form)
    gpu_lib.muon_attention_backward(q, keys, values, out, lse, do, gq, gk, gv, **form)
    torch.cuda.synchronize()
    # It sees n - 1 keys alike.  A part of the walk (64 at most) takes 2^18 tiles: 2^18 x 4 steps x 2 parts = 2^21 additions to an element of
    # out, each within 2 u of a running sum that grows evenly, so half of 2^22 u = 2^-3 in all; a lane adds 2^23 probabilities, each
    # addition within u, half of 2^23 u = 2^-2.
    assert (np.abs(_np(out) - _np(v)) <= (2.0 ** -3 + 2.0 ** -2) * np.abs(_np(v))).all() and out.any()
    z, low, high = 0.25 * float((_np(q) * _np(k)).sum()), np.log(0.75), np.log(1.25)
    assert low - 1e-4 <= float(lse) - (z + np.log(n - 1)) <= high + 1e-4
    # grad_v = p grad_out with p from lse, the same for every key that is seen
    p = np.exp(z - float(lse))
    want = _np(do)[0, 0] * p
    assert not gv[0].any() and not gk[0].any()
    for part in gv[1:].split(1 << 27):
        lo, hi = part.amin((0, 1)), part.amax((0, 1))
        # p: the score and lse in fp32, an exponential, 2^-16 in all for |lse| up to 64; then bf16
        assert (lo == hi).all() and (np.abs(_np(lo) - want) <= (2.0 ** -8 + 2.0 ** -15) * np.abs(want)).all()
    # dz = p (do.v - do.out), the same for every key: what out is off by
    dz = float((_np(do) * (_np(v) - _np(out))).sum())
    size = float((np.abs(_np(do)) * np.abs(_np(v))).sum())
    bound = 0.25 * p * (2.0 ** -7 * abs(dz) + 2.0 ** -18 * size)
    for part in gk[1:].split(1 << 27):
        lo, hi = part.amin((0, 1)), part.amax((0, 1))
        assert (lo == hi).all() and (np.abs(_np(lo) - 0.25 * p * dz * _np(q)[0, 0]) <= bound * np.abs(_np(q)[0, 0])).all()
    assert (np.abs(_np(gq)) <= 0.25 * 1.5 * (abs(dz) + 2.0 ** -18 * size) * np.abs(_np(k))).all()
    del gk, gv, part
    torch.cuda.empty_cache()


def _two_part(mao, c, t):
    import torch
    low = torch.full(t["q"].shape[:2], float("nan"), device="cuda")
    return {**_run(mao, c, t, lse_low=low), "lse_low": low}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [dict(nq=[77]), dict(nq=[3, 0, 200], nk=[40, 9, 300], causal=True, width=128, heads=4, kv=2), dict(nq=[1], nk=[5000], heads=8, kv=2),
                                   dict(nq=[60], nk=[20], causal=True), dict(nq=[130], nk=[260], buckets=8, reach=20, window=33),
                                   dict(nq=[1, 2], nk=[1700, 900], buckets=7, reach=500, causal=True), dict(nq=[1150], heads=1, kv=1, causal=True, masked=0.1)],
                         ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()).replace(" ", ""))
def test_lse_in_two_parts(gpu_lib, shape, dtype):
    import torch
    c = _case(dtype=dtype, **shape)
    t, val = _make(c)
    o, alone, ref = _two_part(gpu_lib, c, t), _run(gpu_lib, c, t), _reference(c, val)
    _check(c, o, val, ref)
    assert torch.equal(o["lse"], alone["lse"]) and torch.equal(o["out"], alone["out"])
    hi, low = _np(o["lse"]), _np(o["lse_low"])
    blind = np.isinf(hi)
    assert (hi[blind] == -np.inf).all() and not low[blind].any() and (blind == np.isinf(ref["lse"])).all()
    # half a step of lse, and the sum of both within the bound of test_gpu_attention's lse without its own rounding
    assert (np.abs(low) <= 2.0 ** -24 * np.where(blind, 0.0, np.abs(hi))).all()
    bound = _bounds(c, ref, val["q"], val["k"], val["v"], None, val["bias"], None)["lse"] - U * np.where(blind, 0.0, np.abs(ref["lse"]))
    with np.errstate(invalid="ignore"):
        off = np.where(blind, 0.0, np.abs(hi + low - ref["lse"]))
    assert (off <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("level", [1000.0, -16000.0])
@pytest.mark.parametrize("with_bias", [False, True])
def test_a_rows_probabilities_add_up_to_one_in_the_backward_pass(gpu_lib, with_bias, level, dtype):
    # One query a head; grad_out is 1 in one column, so a key's grad_v there is its probability.  lse alone is off by up to 3.1e-5 at 1000
    # and 4.9e-4 at 16000.  In two parts what is left are the sum's chain (32 or 288 additions of u each: 1.7e-5), the exponents'
    # roundings (30 u) and exponentials (2^-22) of both passes, 4e-6, and in bf16 the outputs' own: within 2^-8 of each and of either
    # sign, so that their sum passes 6 x 2^-8 sqrt(sum p^2) with a probability below 2 exp(-18) (Hoeffding's bound).
    import torch
    n = 64 if level > 0 else 1150
    c = _case(nq=[1], nk=[n], heads=4, kv=4, dtype=dtype, scale=1.0, logits=0.25, **(dict(buckets=1, reach=3) if with_bias else {}))
    t, val = _make(c, seed=7)
    if with_bias:
        t["bias"].fill_(level)
    else:
        # the scores' common part by one column of q and k
        t["q"][:, :, 0], t["k"][:, :, 0] = 32.0, level / 32
    t["do"].zero_()
    t["do"][:, :, 0] = 1.0
    o = _two_part(gpu_lib, c, t)
    p = _np(o["v"])[:, :, 0]
    bound = (2.0 ** -14 if level < 0 else 2.0 ** -17) + (6 * 2.0 ** -8 * np.sqrt((p * p).sum(0)) if dtype == "bf16" else 0.0)
    assert (np.abs(p.sum(0) - 1) <= bound).all(), p.sum(0) - 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [None, -1e9, -1e6])
@pytest.mark.parametrize("shape", [dict(nq=[150], window=30), dict(nq=[70, 1, 40], nk=[90, 5, 60], causal=True, heads=4, kv=2, width=40), dict(nq=[1], nk=[900], width=128),
                                   dict(nq=[1101], heads=1, kv=1, width=24, causal=True), dict(nq=[200], nk=[1101], heads=1, kv=1, width=128, masked=0.3)],
                         ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()).replace(" ", ""))
def test_gradients_where_a_row_sees_nothing_but_a_very_low_bias(gpu_lib, shape, value, dtype):
    # Keys count alike, also in the gradients.  At the lowest value (None) a score is the bias, whatever the product; else q is 0.
    import torch
    c = _case(dtype=dtype, buckets=3, reach=17, **shape)
    t, val = _make(c)
    t["bias"].fill_(float(torch.finfo(t["q"].dtype).min) if value is None else value)
    if value is not None:
        t["q"].zero_()
    val = {**val, "q": _np(t["q"]), "bias": _np(t["bias"])}
    o, ref = _two_part(gpu_lib, c, t), _reference(c, val)
    count = np.full(ref["lse"].shape, 0.0)
    for s in ref["parts"]:
        assert np.ptp(s["z"][s["seen"]]) == 0
        s["z"] = np.zeros_like(s["z"])
        count[s["rows"], s["head"]] = s["seen"].sum(1)
    seen = count > 0
    want = np.log(np.maximum(count, 1))
    over = _np(o["lse"])[seen] - val["bias"][0, 0]                  # exact: equal, or within a factor of two
    off = np.zeros_like(want)
    off[seen] = np.abs(over + _np(o["lse_low"])[seen] - want[seen])
    off -= (2.0 ** -20 + 2.0 ** -22 * want + count * U)
    assert off.max() <= 0, off.max()
    # the bounds for scores of 0 (no rounding in them), against the probabilities 1 / n
    flat = {**ref, "lse": np.where(seen, want, -np.inf)}
    b = _bounds(c, flat, val["q"], val["k"], val["v"], val["do"], np.zeros((3, c["heads"])), o["low"])
    for name in ("out", "q", "k", "v", "bias"):
        _near(o[name], ref[name], b[name], name)
