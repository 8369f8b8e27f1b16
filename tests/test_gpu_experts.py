"""GPU parity of the tokens' sort by expert, their weighted return and both gradients against the fp64 oracle.

Rows that are only moved, slots and offsets have to be equal.  A sum over `chosen` terms in order is within chosen u of the sum
of the magnitudes (u = 2^-24), a dot product of `cols` terms within (cols / 64 + 8) u (a lane's chain, then a tree over 64
lanes); an output's own rounding is u of it in fp32 and 2^-8 in bf16.
"""
import numpy as np
import pytest

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {"f32": U, "bf16": 2.0 ** -8}
NAN = float("nan")


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _np(t):
    return t.detach().double().cpu().numpy()


def _make(tokens, cols, experts, chosen, dtype, dropped=0.1, seed=0, pick=None):
    import torch
    r = np.random.default_rng(seed)
    ids = r.integers(0, experts, (tokens, chosen)) if pick is None else pick
    if dropped:
        ids = np.where(r.random(ids.shape) < dropped, r.choice([-1, experts, -(1 << 40), 1 << 40]), ids)
    put = lambda a: torch.from_numpy(a.astype(np.float32)).to(_dt(dtype)).cuda()
    n = tokens * chosen
    t = dict(x=put(r.standard_normal((tokens, cols))), y=put(r.standard_normal((n, cols))), g=put(r.standard_normal((tokens, cols))),
             gs=put(r.standard_normal((n, cols))), w=torch.from_numpy(r.random((tokens, chosen)).astype(np.float32)).cuda(),
             ids=torch.from_numpy(ids.astype(np.int64)).cuda())
    return t


def _buffers(t, experts):
    import torch
    like = lambda x: torch.full_like(x, NAN)
    return dict(s=like(t["gs"]), slots=torch.full(t["ids"].shape, 7, dtype=torch.int32, device="cuda"),
                off=torch.full((experts + 1,), 7, dtype=torch.int64, device="cuda"), out=like(t["x"]), gx=like(t["x"]), gy=like(t["y"]), gw=like(t["w"]))


def _calls(mao, t, o, **kw):
    only = {k: v for k, v in kw.items() if k == "stream"}
    mao.muon_expert_sort(t["x"], t["ids"], o["s"], o["slots"], o["off"], **kw)
    mao.muon_expert_combine(t["y"], o["slots"], t["w"], o["out"], **only)
    mao.muon_expert_combine_backward(t["g"], t["y"], o["slots"], t["w"], o["off"], o["gy"], o["gw"], **only)
    mao.muon_expert_sort_backward(t["gs"], o["slots"], o["gx"], **only)


def _check(t, o, experts, dtype):
    R, v = ROUND[dtype], {k: _np(x) for k, x in t.items()}
    ids = t["ids"].cpu().numpy()
    s, slots, off = bo.expert_sort(v["x"], ids, experts)
    assert (o["off"].cpu().numpy() == off).all()
    assert (o["slots"].cpu().numpy() == slots).all()
    assert (_np(o["s"]) == s).all()
    chosen, cols = ids.shape[1], v["x"].shape[1]

    def near(got, want, size, what, r=R):
        off = np.abs(_np(got) - want)
        bound = size + r * np.abs(want) + 1e-38
        assert (off <= bound).all(), (what, float((off / bound).max()))
    near(o["out"], bo.expert_combine(v["y"], slots, v["w"]), chosen * U * bo.expert_combine(np.abs(v["y"]), slots, v["w"]), "out")
    near(o["gx"], bo.expert_sort_backward(v["gs"], slots), chosen * U * bo.expert_sort_backward(np.abs(v["gs"]), slots), "grad_x")
    gy, gw = bo.expert_combine_backward(v["g"], v["y"], slots, v["w"])
    near(o["gy"], gy, U * np.abs(gy), "grad_y")
    _, size = bo.expert_combine_backward(np.abs(v["g"]), np.abs(v["y"]), slots, v["w"])
    near(o["gw"], gw, (cols / 64 + 8) * U * size, "grad_weights", U)


SHAPES = [(1, 2048, 64, 6), (1, 1, 1, 1), (5, 7, 3, 2), (33, 8, 8, 4), (64, 9, 5, 8), (512, 16, 64, 1), (513, 15, 64, 1), (300, 65, 7, 3), (100, 520, 256, 8),
          (40, 2056, 10, 2), (700, 33, 2048, 2), (33, 4100, 4, 5), (2000, 3, 1, 2), (9, 24, 130, 64), (40000, 2, 50, 2), (3000, 40, 16, 6)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_experts(gpu_lib, shape, dtype):
    import torch
    t = _make(*shape, dtype)
    o = _buffers(t, shape[2])
    _calls(gpu_lib, t, o)
    torch.cuda.synchronize()
    _check(t, o, shape[2], dtype)


@pytest.mark.parametrize("shape", [(1024, 4, 128, 1), (1024, 4, 129, 1), (131072, 1, 128, 1), (131073, 1, 128, 1), (131073, 1, 7, 1), (2000, 3, 2048, 2)], ids=str)
def test_both_ways_to_add_up_the_chunks_counts(gpu_lib, shape):
    import torch
    t = _make(*shape, "f32")
    o = _buffers(t, shape[2])
    _calls(gpu_lib, t, o)
    torch.cuda.synchronize()
    _check(t, o, shape[2], "f32")


@pytest.mark.parametrize("pick", ["one", "none", "same_twice", "reversed"])
def test_uneven_choices(gpu_lib, pick):
    import torch
    tokens, experts, chosen = 700, 9, 4
    ids = {"one": np.full((tokens, chosen), 4), "none": np.full((tokens, chosen), -1),
           "same_twice": np.repeat(np.arange(tokens)[:, None] % experts, chosen, 1),
           "reversed": (experts - 1) - (np.arange(tokens * chosen) * experts // (tokens * chosen)).reshape(tokens, chosen)}[pick]
    t = _make(tokens, 20, experts, chosen, "f32", dropped=0.0, pick=ids)
    o = _buffers(t, experts)
    _calls(gpu_lib, t, o)
    torch.cuda.synchronize()
    _check(t, o, experts, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pitches_and_odd_starts(gpu_lib, dtype):
    import torch
    tokens, cols, experts, chosen = 60, 37, 6, 3
    t = _make(tokens, cols, experts, chosen, dtype)
    o = _buffers(t, experts)
    whole = {}
    for d, keys in ((t, ("x", "y", "g", "gs")), (o, ("s", "out", "gx", "gy"))):
        for i, k in enumerate(keys):
            buf = torch.full((d[k].shape[0], cols + 5 + i), NAN, dtype=_dt(dtype), device="cuda")
            whole[k] = buf
            view = buf[:, 1 + i:1 + i + cols]
            view.copy_(d[k])
            d[k] = view
    _calls(gpu_lib, t, o)
    torch.cuda.synchronize()
    _check(t, o, experts, dtype)
    for k in ("s", "out", "gx", "gy"):
        buf = whole[k].clone()
        i = ("s", "out", "gx", "gy").index(k)
        buf[:, 1 + i:1 + i + cols] = NAN
        assert torch.isnan(buf).all()


def test_dropped_choices_reach_nothing(gpu_lib):
    import torch
    t = _make(90, 24, 5, 3, "f32", dropped=0.3)
    o, p = _buffers(t, 5), _buffers(t, 5)
    _calls(gpu_lib, t, o)
    torch.cuda.synchronize()
    count = int(o["off"][-1])
    assert 0 < count < 270
    q = {k: v.clone() for k, v in t.items()}
    q["w"][o["slots"] < 0] = NAN
    q["y"][count:] = NAN
    q["gs"][count:] = float("inf")
    _calls(gpu_lib, q, p)
    torch.cuda.synchronize()
    for k in o:
        assert torch.equal(o[k], p[k]), k


def test_no_tokens(gpu_lib):
    import torch
    t = _make(0, 8, 4, 2, "bf16", dropped=0.0, pick=np.zeros((0, 2), np.int64))
    o = _buffers(t, 4)
    _calls(gpu_lib, t, o)
    torch.cuda.synchronize()
    assert not o["off"].any()


@pytest.mark.parametrize("shape", [(40, 64, 8, 2), (3000, 64, 64, 6), (70000, 8, 16, 2)])
def test_another_stream_and_a_graph(gpu_lib, shape):
    import torch
    t = _make(*shape, "bf16")
    want, got = _buffers(t, shape[2]), _buffers(t, shape[2])
    ws = torch.full((gpu_lib.muon_expert_sort_workspace_bytes(t["x"], t["ids"], shape[2]),), 255, dtype=torch.uint8, device="cuda")
    _calls(gpu_lib, t, want, workspace=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    _calls(gpu_lib, t, got, stream=side)
    side.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _calls(gpu_lib, t, got, workspace=ws)
    for _ in range(3):
        for v in list(got.values()) + [ws]:
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[k], got[k]) for k in want)


def test_more_choices_than_a_launch_has_waves(gpu_lib):
    import torch
    tokens, chosen, experts = 8_500_000, 2, 300
    ids = torch.randint(-1, experts, (tokens, chosen), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    x = torch.arange(tokens, device="cuda").float()[:, None] % 1021
    n = tokens * chosen
    y = torch.arange(n, device="cuda").float()[:, None] % 509
    s, gy, slots = torch.full_like(y, NAN), torch.full_like(y, NAN), torch.zeros((tokens, chosen), dtype=torch.int32, device="cuda")
    off, w = torch.zeros(experts + 1, dtype=torch.int64, device="cuda"), torch.rand((tokens, chosen), device="cuda")
    gw, out, gx = torch.full_like(w, NAN), torch.full_like(x, NAN), torch.full_like(x, NAN)
    gpu_lib.muon_expert_sort(x, ids, s, slots, off)
    gpu_lib.muon_expert_combine(y, slots, w, out)
    gpu_lib.muon_expert_combine_backward(x, y, slots, w, off, gy, gw)
    gpu_lib.muon_expert_sort_backward(y, slots, gx)
    key = torch.where(ids < 0, experts, ids).reshape(-1)
    order = torch.sort(key, stable=True).indices
    count = int((key < experts).sum())
    assert off.tolist() == torch.searchsorted(key[order], torch.arange(experts + 1, device="cuda")).tolist()
    place = torch.empty_like(order)
    place[order] = torch.arange(n, device="cuda")
    assert torch.equal(slots.reshape(-1).long(), torch.where(key < experts, place, -1))
    assert torch.equal(s[:count], x[order[:count] // chosen]) and not s[count:].any()
    live = (slots >= 0)
    picked = torch.where(live, y[slots.clamp(min=0).long(), 0], 0.0)
    assert torch.equal(gw, torch.where(live, x * picked, 0.0))             # one product each
    assert torch.equal(gy[:count, 0], (w * x).reshape(-1)[order[:count]]) and not gy[count:].any()
    assert torch.equal(gx, picked.sum(1, keepdim=True))                    # whole numbers
    assert ((out[:, 0] - (picked.double() * w).sum(1)).abs() <= 3 * U * (picked.double() * w).sum(1) + 1e-30).all()
