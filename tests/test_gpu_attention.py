"""GPU parity of attention and its gradients against the fp64 oracle (through the public entry points).

Bounds, elementwise, with u = 2^-24, n the keys (or queries) that a sum goes over and D the width.  The matrix unit's
sums of exact products are within 2 u (terms + 4) of the sum of the magnitudes, whatever its order:
  score     dz_ij = 2 u (D + 4) |scale| sum |q||k| + 2 u (|z| + |bias|)
  exponent  4 u (|z_ij| + max_j |z_ij|) for the product with log2 e, its difference and the reference; 2^-21 for exp2 and the
            factors by which a row is rescaled
so a probability before its division is within e_ij = dz_ij + 4 u (..) + 2^-21 of itself; a row takes its largest, e_i.
  out       (2 e_i + 3 n u + PART) sum p|v|, PART = 2^-16 where the probabilities go in as two bf16 parts
  lse       e_i + n u + 4 u |lse| + 2^-21
  p again, from lse:  e'_i = 2 e_i + (n + 4 |lse|) u + 2^-20
  dp        2 u (D + 4) sum |do||v|
  delta     sum |do| (bound of out, and what out was rounded by: 2^-16 |out| with out_low in bf16) + 2 u (D + 4) sum |do||out|
  dz        p (e'_i (|dp| + |delta|) + bound of dp + bound of delta + 2 u (|dp| + |delta|))
  grad_q    |scale| (sum (bound of dz)|k| + (PART + n u) sum |dz||k|), grad_k and grad_v alike
  grad_bias sum (bound of dz) + (n + 128) u sum |dz|
An output's own rounding is u of it in fp32 and 2^-8 in bf16.
"""
import numpy as np
import pytest

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {"f32": U, "bf16": 2.0 ** -8}
PART = {"f32": 0.0, "bf16": 2.0 ** -16}
NAN = float("nan")


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _put(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(_dt(dtype)).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _bounds(case, ref, q, k, v, do, bias, low):
    """Bounds of every output (see the module's docstring)."""
    dtype, scale = case["dtype"], abs(case["scale"])
    D, R, P = q.shape[2], ROUND[dtype], PART[dtype]
    b = {n: np.zeros_like(ref[n]) for n in ("out", "lse", "q", "k", "v", "bias") if n in ref}
    for s in ref["parts"]:
        h, g, rows, cols = s["head"], s["kv"], s["rows"], s["cols"]
        Q, K, V = np.abs(q[rows, h]), np.abs(k[cols, g]), np.abs(v[cols, g])
        n = max(len(rows), len(cols)) * (q.shape[1] // k.shape[1])
        z = np.where(s["seen"] & np.isfinite(s["z"]), np.abs(s["z"]), 0.0)
        zb = 2 * U * (D + 4) * scale * (Q @ K.T) + 2 * U * z
        if bias is not None:
            inside = (s["bucket"] >= 0) & (s["bucket"] < len(bias))
            bv = np.where(inside, bias[np.where(inside, s["bucket"], 0), h], 0.0)
            zb = zb + 2 * U * np.where(np.isfinite(bv), np.abs(bv), 0.0)
        e = zb + 4 * U * (z + z.max(1, keepdims=True)) + 2.0 ** -21
        e = np.where(s["seen"], e, 0).max(1)
        l = np.where(np.isfinite(ref["lse"][rows, h]), np.abs(ref["lse"][rows, h]), 0.0)
        out = (2 * e + 3 * n * U + P)[:, None] * (s["p"] @ V)
        b["out"][rows, h] = out
        b["lse"][rows, h] = e + n * U + 4 * U * l + 2.0 ** -21
        if do is None:
            continue
        dO, o = np.abs(do[rows, h]), np.abs(ref["out"][rows, h])
        e2 = 2 * e + (n + 4 * l) * U + 2.0 ** -20
        dp = 2 * U * (D + 4) * (dO @ V.T)
        kept = R if low is None else (2.0 ** -16 if dtype == "bf16" else U)
        delta = (dO * (out + kept * o)).sum(1) + 2 * U * (D + 4) * (dO * o).sum(1)
        size = np.abs(s["dp"]) + (dO * o).sum(1)[:, None]
        dz = s["p"] * ((e2[:, None] + 2 * U) * size + dp + delta[:, None])
        z1 = np.abs(s["dz"])
        b["q"][rows, h] = scale * (dz @ K + (P + n * U) * (z1 @ K))
        b["k"][cols, g] += scale * (dz.T @ Q + (P + n * U) * (z1.T @ Q))
        b["v"][cols, g] += (s["p"] * (e2[:, None] + P + n * U)).T @ dO
        if bias is not None:
            inside = (s["bucket"] >= 0) & (s["bucket"] < len(bias))
            np.add.at(b["bias"], (s["bucket"][inside], h), (dz + (n + 128) * U * z1)[inside])
    for name in b:
        r = np.where(np.isfinite(ref[name]), np.abs(ref[name]), 0.0)
        b[name] = 1.05 * b[name] + (U if name == "lse" else R) * r + 1e-37
    return b


def _near(got, want, bound, what):
    got = _np(got)
    with np.errstate(invalid="ignore"):
        off = np.where(got == want, 0.0, np.abs(got - want))
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.size, float(np.nanmax(off / bound)), np.argwhere(bad)[:4].tolist())


def _case(**kw):
    c = dict(dtype="bf16", nq=[77], nk=None, heads=2, kv=2, width=64, causal=False, window=0, masked=0.0, buckets=0, reach=0, scale=None,
             low=True, grad=True, logits=2.0, before=0, after=0, mean=0.0)
    c.update(kw)
    c["nk"] = c["nq"] if c["nk"] is None else c["nk"]
    c["scale"] = c["width"] ** -0.5 if c["scale"] is None else c["scale"]
    return c


def _make(c, seed=0):
    """(tensors on the GPU, the fp64 values they hold)."""
    import torch
    r = np.random.default_rng(seed)
    n, m = (c["before"] + sum(c[k]) + c["after"] for k in ("nq", "nk"))
    t = dict(q=_put(r.standard_normal((n, c["heads"], c["width"])) * c["logits"], c["dtype"]),
             k=_put(r.standard_normal((m, c["kv"], c["width"])), c["dtype"]),
             v=_put(r.standard_normal((m, c["kv"], c["width"])) + c["mean"], c["dtype"]),
             do=_put(r.standard_normal((n, c["heads"], c["width"])) * 1e-2, c["dtype"]), mask=None, bias=None, map=None)
    t["off"], t["koff"] = (torch.from_numpy(np.cumsum([c["before"]] + c[k])).cuda() for k in ("nq", "nk"))
    if c["masked"]:
        t["mask"] = torch.from_numpy(r.random(m) >= c["masked"]).cuda()
    if c["buckets"]:
        t["bias"] = _put(r.standard_normal((c["buckets"], c["heads"])), c["dtype"])
        t["map"] = torch.from_numpy(r.integers(0, c["buckets"], 2 * c["reach"] + 1).astype(np.int32)).cuda()
    return t, {k: None if v is None else v.cpu().numpy() if k in ("mask", "off", "koff", "map") else _np(v) for k, v in t.items()}


def _form(c, t):
    return dict(offsets=t["off"], key_offsets=t["koff"], key_mask=t["mask"], bias=t["bias"], bucket_map=t["map"], scale=c["scale"],
                causal=c["causal"], window=c["window"])


def _reference(c, val, grad=None):
    return bo.attention(val["q"], val["k"], val["v"], offsets=val["off"], key_offsets=val["koff"], mask=val["mask"], bias=val["bias"],
                        bucket_map=val["map"], scale=float(np.float32(c["scale"])), causal=c["causal"], window=c["window"],
                        grad_out=val["do"] if (c["grad"] if grad is None else grad) else None)


def _run(mao, c, t, **kw):
    """Outputs of both calls; every buffer is full of NaN before."""
    import torch
    like = lambda x: torch.full_like(x, NAN)
    o = dict(out=like(t["q"]), lse=torch.full(t["q"].shape[:2], NAN, device="cuda"), low=like(t["q"]) if c["low"] else None)
    form = {**_form(c, t), "out_low": o["low"], **kw}
    mao.muon_attention(t["q"], t["k"], t["v"], o["out"], o["lse"], **form)
    if c["grad"]:
        o.update(q=like(t["q"]), k=like(t["k"]), v=like(t["v"]), bias=None if t["bias"] is None else like(t["bias"]))
        mao.muon_attention_backward(t["q"], t["k"], t["v"], o["out"], o["lse"], t["do"], o["q"], o["k"], o["v"], grad_bias=o["bias"], **form)
    torch.cuda.synchronize()
    return o


def _check(c, o, val, ref=None):
    ref = _reference(c, val) if ref is None else ref
    b = _bounds(c, ref, val["q"], val["k"], val["v"], val["do"] if c["grad"] else None, val["bias"], o["low"])
    for name, bound in b.items():
        _near(o[name], ref[name], bound, name)
    if o["low"] is not None:
        # what rounding took: together 16 bits (bf16), nothing (fp32)
        whole = _np(o["out"]) + _np(o["low"])
        bound = b["out"] - ROUND[c["dtype"]] * np.abs(ref["out"]) + max(PART[c["dtype"]], U) * np.abs(ref["out"])
        assert (np.abs(whole - ref["out"]) <= bound).all()


SHAPES = [
    dict(nq=[1]), dict(nq=[1], nk=[1], width=1, heads=1, kv=1), dict(nq=[31]), dict(nq=[32], causal=True), dict(nq=[33], causal=True),
    dict(nq=[63]), dict(nq=[64], causal=True), dict(nq=[65], causal=True, window=9), dict(nq=[127]), dict(nq=[128], causal=True),
    dict(nq=[129], causal=True), dict(nq=[257], width=128, causal=True), dict(nq=[200], nk=[300], causal=True, width=128),
    dict(nq=[3, 0, 70, 1, 130], causal=True, heads=4), dict(nq=[3, 5, 0, 40], nk=[9, 0, 7, 33], causal=True),
    dict(nq=[50, 2], nk=[20, 1], causal=True),                       # more queries than keys: the first see none
    dict(nq=[90], heads=6, width=128, kv=2, causal=True), dict(nq=[90], heads=5, kv=1, width=40), dict(nq=[40], width=7, causal=True),
    dict(nq=[70, 66], width=72, kv=1), dict(nq=[100], width=101), dict(nq=[140], width=128, masked=0.4, causal=True),
    dict(nq=[140, 20], masked=0.9, window=5), dict(nq=[140], window=1), dict(nq=[300], window=70, width=32),
    dict(nq=[300], window=64, causal=True, width=128), dict(nq=[1], nk=[5000], width=128, heads=4), dict(nq=[1, 1], nk=[700, 2100], causal=True, kv=1),
    dict(nq=[5], nk=[3000], width=36, masked=0.2), dict(nq=[2500], nk=[3], heads=1, kv=1, width=48), dict(nq=[1] * 70, nk=[3] * 70),
    dict(nq=[4] * 150, causal=True, width=16), dict(nq=[66], before=5, after=9, causal=True), dict(nq=[80], scale=-0.2, causal=True),
    dict(nq=[80], scale=0.0), dict(nq=[130], low=False, causal=True),
]
BIASES = [
    dict(nq=[77], buckets=5, reach=6), dict(nq=[200], buckets=32, reach=128, causal=True, width=128), dict(nq=[300], buckets=3, reach=0),
    dict(nq=[300], buckets=9, reach=1), dict(nq=[40, 0, 150], buckets=32, reach=600, masked=0.2), dict(nq=[3], nk=[1000], buckets=7, reach=500),
    dict(nq=[130], nk=[260], buckets=8, reach=20, causal=True, window=33, heads=6, kv=2, width=24), dict(nq=[260], buckets=8, reach=64, window=50),
    dict(nq=[1], buckets=1, reach=4096), dict(nq=[1] * 40, nk=[90] * 40, buckets=6, reach=40), dict(nq=[60], nk=[20], causal=True, buckets=4, reach=9),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES + BIASES, ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()).replace(" ", "")[:70])
def test_attention(gpu_lib, shape, dtype):
    c = _case(dtype=dtype, **shape)
    t, val = _make(c)
    _check(c, _run(gpu_lib, c, t), val)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [
    dict(nq=[1], nk=[900], heads=8, kv=2, causal=True), dict(nq=[3, 1, 0, 5], nk=[40, 1, 7, 300], heads=32, kv=1, width=40, causal=True),
    dict(nq=[7], nk=[200], heads=64, kv=1, width=16, window=30), dict(nq=[100, 20], heads=12, kv=3, masked=0.3), dict(nq=[9], nk=[4], heads=8, kv=4, causal=True),
    dict(nq=[70, 5], nk=[90, 66], heads=4, kv=1, width=101, causal=True, scale=-0.1),
], ids=lambda s: f"{s['heads']}of{s['kv']}")
def test_heads_that_share_a_workgroups_rows(gpu_lib, shape, dtype):
    c = _case(dtype=dtype, **shape)
    t, val = _make(c)
    _check(c, _run(gpu_lib, c, t), val)


@pytest.mark.parametrize("count", [61, 62, 300, 512, 513, 2000])
def test_many_sequences(gpu_lib, count):
    # by lane up to 61, in order up to 512, by a stride beyond; lengths from nothing to more than a workgroup's rows
    r = np.random.default_rng(count)
    nq = [int(v) for v in r.integers(0, 5, count)]
    nq[count // 3], nq[count // 2], nq[-1] = 150, 300, 129
    nk = [n + int(v) for n, v in zip(nq, r.integers(0, 4, count))]
    c = _case(nq=nq, nk=nk, heads=1, kv=1, width=16, dtype="f32", causal=bool(count % 2), before=2, after=140)
    t, val = _make(c)
    _check(c, _run(gpu_lib, c, t), val)


def test_more_units_than_a_launch_holds(gpu_lib):
    # 2.2 million sequences, nearly all empty: more workgroups than the 2^21 of one launch
    import torch
    c = _case(nq=[90, 40], heads=1, kv=1, width=16, dtype="f32", causal=True)
    t, val = _make(c)
    want = _run(gpu_lib, c, t)
    off = torch.full((2_200_001,), 130, dtype=torch.int64, device="cuda")
    off[:5] = 0
    off[5:2_199_000] = 90
    got = _run(gpu_lib, c, {**t, "off": off, "koff": off})
    # the walks are the same; the split of few units is not, so the sums may be taken in another order
    ref = _reference(c, val)
    _check(c, got, val, ref)
    _check(c, want, val, ref)


def test_a_workspace_for_other_layouts_is_refused(gpu_lib):
    import torch
    c = _case(nq=[200], causal=True)
    t, _ = _make(c)
    ws = torch.empty(gpu_lib.muon_attention_workspace_bytes(t["q"], t["k"]), dtype=torch.uint8, device="cuda")
    odd = torch.zeros(200 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(200, 2, 64)
    out, lse = torch.empty_like(t["q"]), torch.empty(200, 2, device="cuda")
    with pytest.raises(gpu_lib.MuonError, match="needed"):
        gpu_lib.muon_attention(t["q"], t["k"], odd, out, lse, workspace=ws)
    gpu_lib.muon_attention(t["q"], t["k"], odd, out, lse)
    assert gpu_lib.muon_attention_workspace_bytes(odd, odd) >= 3 * 200 * 128 * 2           # a copy of each of q, k and v
    torch.cuda.synchronize()


def test_one_sequence_without_offsets(gpu_lib):
    for c in (_case(nq=[90], causal=True), _case(nq=[20], nk=[90], causal=True, dtype="f32")):
        t, val = _make(c)
        want = _run(gpu_lib, c, t)
        got = _run(gpu_lib, c, {**t, "off": None, "koff": None})
        for k in ("out", "lse", "q", "k", "v"):
            assert (_np(want[k]) == _np(got[k])).all()
        if c["nq"] == c["nk"]:
            got = _run(gpu_lib, c, {**t, "koff": None})
            assert (_np(want["k"]) == _np(got["k"])).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "interleaved", "heads_first", "odd_pitch", "odd_start", "broadcast"])
def test_attention_layouts(gpu_lib, layout, dtype):
    import torch
    c = _case(nq=[70, 65], heads=3, kv=3, width=64, causal=True, dtype=dtype)
    t, val = _make(c)
    n = sum(c["nq"])
    names = ("q", "k", "v")

    def views(fill=None):
        if layout == "fused":
            buf = torch.full((n, 3, 3, 64), NAN, dtype=_dt(dtype), device="cuda")
            return buf, [buf[:, i] for i in range(3)]
        if layout == "interleaved":
            buf = torch.full((n, 3, 3, 64), NAN, dtype=_dt(dtype), device="cuda")
            return buf, [buf[:, :, i] for i in range(3)]
        if layout == "heads_first":
            buf = torch.full((3, 3, n, 64), NAN, dtype=_dt(dtype), device="cuda")
            return buf, [buf[i].transpose(0, 1) for i in range(3)]
        if layout == "odd_pitch":
            buf = torch.full((3, n, 3, 67), NAN, dtype=_dt(dtype), device="cuda")
            return buf, [buf[i][:, :, :64] for i in range(3)]
        buf = torch.full((3, n * 3 * 64 + 8), NAN, dtype=_dt(dtype), device="cuda")
        return buf, [buf[i][1 + i:1 + i + n * 192].view(n, 3, 64) for i in range(3)]
    _, ins = views()
    for v, k in zip(ins, names):
        v.copy_(t[k])
    if layout == "broadcast":
        # one key head behind three: as many gradients as there are views of it
        one = t["k"][:, :1].contiguous()
        t = {**t, "k": one.expand(-1, 3, -1), "v": t["v"][:1].expand(n, -1, -1)}
        val = {**val, "k": np.broadcast_to(val["k"][:, :1], val["k"].shape), "v": np.broadcast_to(val["v"][:1], val["v"].shape)}
        ins = [t[k] for k in names]
    gbuf, grads = views()
    out, low = (torch.full_like(t["q"], NAN) for _ in range(2))
    lse = torch.full(t["q"].shape[:2], NAN, device="cuda")
    form = dict(_form(c, t), out_low=low)
    gpu_lib.muon_attention(*ins, out, lse, **form)
    gpu_lib.muon_attention_backward(*ins, out, lse, t["do"], *grads, **form)
    torch.cuda.synchronize()
    _check(c, dict(out=out, lse=lse, low=low, q=grads[0], k=grads[1], v=grads[2]), val)
    if layout == "odd_pitch":
        assert torch.isnan(gbuf[..., 64:]).all()                    # the gaps stay as they were


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_is_hidden_reaches_nothing(gpu_lib, dtype):
    import torch
    # masked keys, rows of no sequence, and queries that see nothing hold NaN and infinities
    c = _case(nq=[40, 9, 70], nk=[50, 4, 70], before=3, after=6, masked=0.3, causal=True, dtype=dtype, buckets=4, reach=8)
    t, val = _make(c)
    t["mask"][3 + 50:3 + 54] = False                                # the second sequence: nobody sees anything
    val["mask"] = t["mask"].cpu().numpy()
    ref = _reference(c, val)
    clean = _run(gpu_lib, c, t)
    blind = torch.from_numpy(np.isinf(ref["lse"]).all(1)).cuda()
    assert blind.sum() >= 18
    for bad in (NAN, float("inf")):
        p = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in t.items()}
        hidden = ~t["mask"]
        hidden[:3] = True
        hidden[-6:] = True
        for k in ("k", "v"):
            p[k][hidden] = bad
        for k in ("q", "do"):
            p[k][blind] = bad
        got = _run(gpu_lib, c, p)
        for k in ("out", "lse", "q", "k", "v", "bias"):
            assert torch.equal(got[k], clean[k]), (k, bad)
    _check(c, clean, val, ref)
    for k in ("out", "q"):
        assert not clean[k][blind].any()
    assert not clean["k"][hidden].any() and not clean["v"][hidden].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bias_of_the_lowest_value_and_infinity(gpu_lib, dtype):
    import torch
    low = float(torch.finfo(_dt(dtype)).min)
    c = _case(nq=[150], dtype=dtype, buckets=3, reach=40, heads=2, window=30)
    t, val = _make(c)
    for value in (low, -float("inf")):
        t["map"].fill_(1)
        t["map"][:35] = 0                                           # distances up to -6
        t["map"][60:] = 2
        t["bias"].copy_(torch.tensor([[value, 0.5], [0.25, -0.5], [0.125, value]], device="cuda"))
        v2 = {**val, "bias": _np(t["bias"]), "map": t["map"].cpu().numpy()}
        _check(c, _run(gpu_lib, c, t), v2)
    # all that a query sees at the lowest value: they count alike; at -infinity: it sees nothing
    t["bias"].fill_(low)
    c2 = {**c, "grad": False}
    o = _run(gpu_lib, c2, t)
    ref = _reference(c2, {**val, "bias": np.zeros((3, 2)), "q": val["q"] * 0})
    assert (np.abs(_np(o["out"]) - ref["out"]) <= (2.0 ** -16 + ROUND[dtype]) * np.abs(val["v"]).max()).all()
    assert (_np(o["lse"]) == float(np.float32(low))).all()
    t["bias"].fill_(-float("inf"))
    o = _run(gpu_lib, c, t)
    assert (_np(o["lse"]) == -np.inf).all()
    for k in ("out", "q", "k", "v", "bias"):
        assert not o[k].any(), k


def test_buckets_beyond_the_table_add_nothing(gpu_lib):
    import torch
    c = _case(nq=[90], buckets=4, reach=10, dtype="f32")
    t, val = _make(c)
    t["map"][::3] = torch.tensor([-1, 4, 1 << 30, -(1 << 31), 4, 5, 6], dtype=torch.int32, device="cuda")
    _check(c, _run(gpu_lib, c, t), {**val, "map": t["map"].cpu().numpy()})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_certain_rows(gpu_lib, dtype):
    # logits of standard deviation 40: most rows see one key only, and its dz is a small difference, which out_low keeps
    c = _case(nq=[130], width=64, logits=40.0, causal=True, dtype=dtype)
    t, val = _make(c)
    _check(c, _run(gpu_lib, c, t), val)
    c = _case(nq=[130], width=64, logits=40.0, causal=True, dtype=dtype, low=False)
    _check(c, _run(gpu_lib, c, t), val)


@pytest.mark.parametrize("mean", [0.0, 30.0])
def test_bf16_error_is_the_outputs_rounding(gpu_lib, mean):
    # With probabilities and dz in 16 bits an output's error is its own rounding: at most 2^-8 of a value, on average over
    # the values' place between powers of two 2^-8 / sqrt(3) * 0.72 = 0.0016 of the norm.  One bf16 part would add 2^-8 / sqrt(3)
    # of each term, 0.0016 of the terms' root sum of squares, which is the norm's size here: 0.0023.
    for shape in (dict(nq=[700], width=128, causal=True, heads=2), dict(nq=[500], width=64, buckets=32, reach=128, heads=2)):
        c = _case(mean=mean, **shape)
        t, val = _make(c, seed=5)
        o, ref = _run(gpu_lib, c, t), _reference(c, val)
        for k in ("out", "q", "k", "v"):
            if mean == 0.0 or k in ("out", "v"):
                assert np.linalg.norm(_np(o[k]) - ref[k]) <= 0.0019 * np.linalg.norm(ref[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_outside_the_rows_are_clamped(gpu_lib, dtype):
    import torch
    c = _case(nq=[60, 70], dtype=dtype, causal=True)
    t, val = _make(c)
    want = _run(gpu_lib, c, t)
    off = torch.tensor([-7, 60, 1 << 40], device="cuda")
    got = _run(gpu_lib, c, {**t, "off": off, "koff": off})
    for k in ("out", "lse", "q", "k", "v"):
        assert torch.equal(want[k], got[k])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [dict(nq=[90], buckets=3, reach=95), dict(nq=[90], buckets=3, reach=96), dict(nq=[2] * 40, nk=[3] * 40, buckets=4, reach=9),
                                   dict(nq=[2] * 70, nk=[3] * 70, buckets=4, reach=9), dict(nq=[300], nk=[900], buckets=1, reach=300)],
                         ids=lambda s: f"{len(s['nq'])}x{s['nq'][0]}-{s['buckets']}-{s['reach']}")
def test_both_ways_to_add_up_the_biass_slots(gpu_lib, shape, dtype):
    c = _case(dtype=dtype, **shape)
    t, val = _make(c)
    _check(c, _run(gpu_lib, c, t), val)


@pytest.mark.parametrize("reach", [2, 400])
def test_a_bias_of_no_queries(gpu_lib, reach):
    c = _case(nq=[0], nk=[9], buckets=3, reach=reach)
    t, val = _make(c)
    o = _run(gpu_lib, c, t)
    assert not o["k"].any() and not o["v"].any() and not o["bias"].any()


def test_no_queries_and_no_keys(gpu_lib):
    import torch
    c = _case(nq=[0], nk=[9], buckets=3, reach=2)
    t, val = _make(c)
    o = _run(gpu_lib, c, t)
    assert not o["k"].any() and not o["v"].any() and not o["bias"].any()
    c = _case(nq=[9], nk=[0], buckets=3, reach=2)
    t, val = _make(c)
    o = _run(gpu_lib, c, t)
    assert not o["out"].any() and (_np(o["lse"]) == -np.inf).all() and not o["q"].any() and not o["bias"].any()
    c = _case(nq=[0], nk=[0])
    t, val = _make(c)
    _run(gpu_lib, c, t)


@pytest.mark.parametrize("shape", [dict(nq=[300, 20], causal=True, width=128), dict(nq=[200], buckets=32, reach=128, heads=4),
                                   dict(nq=[2], nk=[4000], heads=4, buckets=5, reach=1000), dict(nq=[130], dtype="f32", kv=1)])
def test_same_bits_every_time_on_another_stream_and_in_a_graph(gpu_lib, shape):
    import torch
    c = _case(**shape)
    t, val = _make(c)
    want = _run(gpu_lib, c, t)
    n = len(c["nq"])
    ws = torch.empty(max(gpu_lib.muon_attention_workspace_bytes(t["q"], t["k"], sequences=n),
                         gpu_lib.muon_attention_backward_workspace_bytes(t["q"], t["k"], sequences=n, bias=t["bias"], bucket_map=t["map"])),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(255)                                                    # NaN to whoever reads what it did not write
    names = [k for k in ("out", "lse", "q", "k", "v", "bias") if want.get(k) is not None]
    got = _run(gpu_lib, c, t, workspace=ws)
    assert all(torch.equal(want[k], got[k]) for k in names)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _run(gpu_lib, c, t, stream=side)
    assert all(torch.equal(want[k], got[k]) for k in names)

    o = {k: None if v is None else torch.full_like(v, NAN) for k, v in want.items()}

    def call():
        form = dict(_form(c, t), out_low=o["low"], workspace=ws)
        gpu_lib.muon_attention(t["q"], t["k"], t["v"], o["out"], o["lse"], **form)
        gpu_lib.muon_attention_backward(t["q"], t["k"], t["v"], o["out"], o["lse"], t["do"], o["q"], o["k"], o["v"], grad_bias=o["bias"], **form)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for k in names:
            o[k].fill_(NAN)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[k], o[k]) for k in names)


def test_long_rows_and_pitches_beyond_32_bits(gpu_lib):
    import torch
    # keys 2^23 elements apart: offsets pass 2^31 elements and 2^32 bytes within the sequence
    n, pitch = 300, 1 << 23
    if torch.cuda.mem_get_info()[0] < 3 * n * pitch:
        pytest.skip("needs 15 GB")
    c = _case(nq=[3], nk=[n], heads=1, kv=1, causal=True)
    t, val = _make(c)
    far = torch.zeros(n * pitch, dtype=torch.bfloat16, device="cuda").view(n, 1, pitch)
    kv = {}
    for i, k in enumerate(("k", "v")):
        far[:, :, 64 * i:64 * i + 64] = t[k]
        kv[k] = far[:, :, 64 * i:64 * i + 64]
    want = _run(gpu_lib, c, t)
    got = _run(gpu_lib, {**c, "grad": False}, {**t, **kv})
    assert torch.equal(want["out"], got["out"]) and torch.equal(want["lse"], got["lse"])
    grads = [torch.full_like(t["q"], NAN), far[:, :, 128:192], far[:, :, 192:256]]
    gpu_lib.muon_attention_backward(t["q"], kv["k"], kv["v"], got["out"], got["lse"], t["do"], *grads, out_low=got["low"], **_form(c, t))
    torch.cuda.synchronize()
    for g, k in zip(grads, ("q", "k", "v")):
        assert torch.equal(g, want[k])
