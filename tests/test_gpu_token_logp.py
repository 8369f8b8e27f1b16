"""GPU parity of the token log-probabilities against the fp64 oracle (through the public entry points).

Bounds, with u = 2^-24 and S_ij = |scale| sum_k |h_ik w_jk|.  A logit is a sum of d products in
fp32: within E_ij = (d / 16 + 32) u S_ij (bf16 operands: exact products; fp32 operands may be
multiplied in parts that keep 2^-22 of each product).  lse and logp move by at most
max_j E_ij each, plus the rounding of the sums, (v / 64 + 64) u.
dz is rounded to the operands' precision before its products: e = 2^-8 relative for bf16, and twice
that on p, since a kept exp(z - m) may have been rounded as well; 2^-21 for fp32.  So dz_ij is off by
at most |c_i| (|[j = y] - p| e + p_ij (2 e + 2 max_j E_ij + (v / 64 + 64) u)), and a gradient by the
products of that with the operand's magnitudes, its own sum's rounding and its own rounding.
"""
import numpy as np
import pytest

from oracle import train_oracle as to

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {"f32": 2 * U, "bf16": 2.0 ** -8}
PARTS = {"f32": 2.0 ** -21, "bf16": 2.0 ** -8}


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(seed, t, d, v, dtype, ignored=0.25, lift=10.0):
    import torch
    rng = np.random.default_rng(seed)
    w = torch.from_numpy((rng.standard_normal((v, d)) / np.sqrt(d)).astype(np.float32)).to(_dt(dtype))
    y = rng.integers(0, v, t)
    h = rng.standard_normal((t, d)) + lift * rng.random((t, 1)) * w.double().numpy()[y]
    h = torch.from_numpy(h.astype(np.float32)).to(_dt(dtype))
    y[rng.random(t) < ignored] = -100
    c = (rng.standard_normal(t) / max(1, t)).astype(np.float32)
    return h.cuda(), w.cuda(), torch.from_numpy(y).cuda(), torch.from_numpy(c).cuda()


def _bounds(h, w, y, scale, dtype):
    h, w = _np(h), _np(w)
    h = np.where((np.asarray(y.cpu()) >= 0)[:, None], h, 0.0)
    d, v = h.shape[1], w.shape[0]
    S = abs(scale) * (np.abs(h) @ np.abs(w).T)
    E = ((d / 16 + 32) * U + (2.0 ** -22 if dtype == "f32" else 0.0)) * S.max(1)
    return h, w, E, (v / 64 + 64) * U


def _forward(mao, h, w, y, scale=1.0, saved=None, **kw):
    import torch
    logp = torch.full((h.shape[0],), float("nan"), device="cuda")
    lse = torch.full((h.shape[0],), float("nan"), device="cuda")
    mao.muon_token_logp(h, w, y, logp, lse, scale=scale, saved=saved, **kw)
    return logp, lse


def _check_forward(h, w, y, scale, dtype, logp, lse):
    hv, wv, E, sums = _bounds(h, w, y, scale, dtype)
    rl, rs, _ = to.token_logp(hv, wv, np.asarray(y.cpu()), scale=np.float32(scale))
    gl, gs = _np(logp), _np(lse)
    assert np.all(np.abs(gl - rl) <= 2 * E + sums + 8 * U * np.abs(rl)), float(np.max(np.abs(gl - rl) / (2 * E + sums)))
    assert np.all(np.abs(gs - rs) <= 2 * E + sums + 8 * U * np.abs(rs))
    dead = np.asarray(y.cpu()) < 0
    assert not gl[dead].any() and not gs[dead].any()


def _backward(mao, h, w, y, lse, c, scale=1.0, saved=None, want=("h", "w")):
    import torch
    gh = torch.full_like(h, float("nan")) if "h" in want else None
    gw = torch.full_like(w, float("nan")) if "w" in want else None
    mao.muon_token_logp_backward(h, w, y, lse, c, gh, gw, scale=scale, saved=saved)
    return gh, gw


def _check_backward(h, w, y, c, scale, dtype, gh, gw):
    hv, wv, E, sums = _bounds(h, w, y, scale, dtype)
    yv, cv = np.asarray(y.cpu()), _np(c)
    rh, rw, dz, p = to.token_logp_backward(hv, wv, yv, cv, scale=np.float32(scale))
    e = PARTS[dtype]
    off = np.abs(dz) * e + np.abs(scale * cv)[:, None] * p * (2 * e + 2 * E[:, None] + sums)
    t, v = dz.shape
    if gh is not None:
        b = off @ np.abs(wv) + (v / 16 + 32) * U * (np.abs(dz) @ np.abs(wv)) + ROUND[dtype] * np.abs(rh) + 1e-38
        err = np.abs(_np(gh) - rh)
        assert np.all(err <= b), ("grad_hidden", float(np.max(err / b)))
        assert not _np(gh)[yv < 0].any()
    if gw is not None:
        b = off.T @ np.abs(hv) + (t / 16 + 32) * U * (np.abs(dz).T @ np.abs(hv)) + ROUND[dtype] * np.abs(rw) + 1e-38
        err = np.abs(_np(gw) - rw)
        assert np.all(err <= b), ("grad_head", float(np.max(err / b)))


def _saved(mao, h, w):
    import torch
    return torch.full((mao.muon_token_logp_saved_bytes(h, w),), 255, dtype=torch.uint8, device="cuda")


SHAPES = [(1, 8, 1), (1, 64, 300), (2, 63, 257), (3, 256, 1000), (16, 100, 515), (17, 128, 4096), (33, 72, 2000), (64, 512, 777),
          (65, 200, 1025), (255, 64, 256), (257, 320, 513), (300, 96, 3001), (513, 65, 129), (1030, 192, 700)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,d,v", SHAPES)
def test_token_logp_shapes(gpu_lib, t, d, v, dtype):
    import torch
    print("[token_logp]", t, d, v, dtype, flush=True)
    h, w, y, c = _inputs(t * 1009 + v, t, d, v, dtype, ignored=0.25 if t > 1 else 0.0)
    scale = 0.8
    saved = _saved(gpu_lib, h, w)
    logp, lse = _forward(gpu_lib, h, w, y, scale)
    _check_forward(h, w, y, scale, dtype, logp, lse)
    gh, gw = _backward(gpu_lib, h, w, y, lse, c, scale)
    _check_backward(h, w, y, c, scale, dtype, gh, gw)
    logp2, lse2 = _forward(gpu_lib, h, w, y, scale, saved=saved)
    _check_forward(h, w, y, scale, dtype, logp2, lse2)
    gh2, gw2 = _backward(gpu_lib, h, w, y, lse2, c, scale, saved=saved)
    _check_backward(h, w, y, c, scale, dtype, gh2, gw2)
    # again, the same bits; one gradient alone, the same bits
    gh3, _ = _backward(gpu_lib, h, w, y, lse2, c, scale, saved=saved, want=("h",))
    _, gw3 = _backward(gpu_lib, h, w, y, lse2, c, scale, saved=saved, want=("w",))
    assert torch.equal(gh2, gh3) and torch.equal(gw2, gw3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [5, 40, 300])
def test_token_logp_ignored_and_invalid_targets(gpu_lib, dtype, t):
    import torch
    print("[token_logp targets]", t, dtype, flush=True)
    h, w, y, c = _inputs(5, t, 128, 600, dtype, ignored=0.5)
    y[0] = 3
    # what ignored tokens hold does not matter
    base = _forward(gpu_lib, h, w, y)
    grads = _backward(gpu_lib, h, w, y, base[1], c)
    dead = y < 0
    h2, c2 = h.clone(), c.clone()
    h2[dead] = float("nan")
    h2[dead.nonzero()[::2, 0]] = float("inf")
    c2[dead] = float("nan")
    got = _forward(gpu_lib, h2, w, y)
    assert torch.equal(got[0], base[0]) and torch.equal(got[1], base[1])
    again = _backward(gpu_lib, h2, w, y, got[1], c2)
    assert torch.equal(again[0], grads[0]) and torch.equal(again[1], grads[1])
    # nothing scored at all
    none = torch.full_like(y, -1)
    logp, lse = _forward(gpu_lib, h2, w, none)
    assert not logp.any() and not lse.any()
    gh, gw = _backward(gpu_lib, h2, w, none, lse, c2)
    assert not torch.count_nonzero(gh) and not torch.count_nonzero(gw)
    # a target beyond the vocabulary is not silently scored
    y2 = y.clone()
    y2[0] = 600
    logp, lse = _forward(gpu_lib, h, w, y2)
    assert torch.isnan(logp[0]) and torch.equal(logp[1:], base[0][1:]) and torch.isfinite(lse[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,d,pitch,shift", [(4, 128, 136, 0), (70, 128, 131, 1), (300, 192, 200, 8), (20, 70, 77, 3)])
def test_token_logp_strides_and_alignment(gpu_lib, dtype, t, d, pitch, shift):
    import torch
    print("[token_logp strides]", t, d, pitch, shift, dtype, flush=True)
    v = 530
    h, w, y, c = _inputs(6, t, d, v, dtype)

    def wide(x):
        buf = torch.full((x.shape[0] * pitch + shift,), float("nan"), dtype=x.dtype, device="cuda")
        view = buf[shift:].view(x.shape[0], pitch)[:, :d]
        view.copy_(x)
        return view
    hw, ww = wide(h), wide(w)
    logp, lse = _forward(gpu_lib, hw, ww, y)
    _check_forward(h, w, y, 1.0, dtype, logp, lse)
    gh, gw = wide(torch.zeros_like(h)), wide(torch.zeros_like(w))
    gpu_lib.muon_token_logp_backward(hw, ww, y, lse, c, gh, gw)
    _check_backward(h, w, y, c, 1.0, dtype, gh, gw)
    # the padding between the rows is untouched
    tail = gh.as_strided((t - 1, pitch - d), (pitch, 1), gh.storage_offset() + d)
    assert torch.isnan(tail).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [3, 100, 260])
def test_token_logp_extreme_logits(gpu_lib, dtype, t):
    # logits far apart: a certain token (logp tiny but not lost), one far from the best, a whole row of equal logits,
    # and logits beyond the range of exp
    import torch
    d, v = 64, 900
    h = torch.zeros((t, d), device="cuda")
    w = torch.zeros((v, d), device="cuda")
    w[:, 0] = 1.0
    w[7, 1] = 1.0
    h[0, 1] = 30.0                 # the target 30 above the rest: logp = -log1p((v - 1) e^-30)
    h[1, 1] = 200.0                # another token 200 above the target
    h[2, 0] = 500.0                # every logit 500 (and 0 at token 7's own column 1)
    y = torch.full((t,), -100, dtype=torch.int64, device="cuda")
    y[0], y[1], y[2] = 7, 8, 9
    h, w = h.to(_dt(dtype)), w.to(_dt(dtype))
    logp, lse = _forward(gpu_lib, h, w, y)
    ref = [-np.log1p((v - 1) * np.exp(-30.0)), -200.0, -np.log(v)]
    got = _np(logp)[:3]
    assert np.all(np.abs(got - ref) <= 1e-5 * np.abs(ref)), (got, ref)
    c = torch.ones(t, device="cuda")
    gh, gw = _backward(gpu_lib, h, w, y, lse, c)
    assert torch.isfinite(gh).all() and torch.isfinite(gw).all()
    assert abs(float(gh[1, 1]) + 1.0) <= 1e-2        # -p_7 = -1 along column 1


def test_token_logp_no_tokens(gpu_lib):
    import torch
    h, w, y, c = _inputs(1, 1, 64, 300, "bf16")
    logp, lse = _forward(gpu_lib, h[:0], w, y[:0])
    gw = torch.full_like(w, 7.0)
    gpu_lib.muon_token_logp_backward(h[:0], w, y[:0], lse, c[:0], h[:0].clone(), gw)
    assert logp.numel() == 0 and not torch.count_nonzero(gw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_token_logp_gradient_against_differences(gpu_lib, dtype):
    # d(sum c logp) along a random direction of hidden and of head, by differences of the fp64 oracle
    t, d, v = 40, 96, 500
    h, w, y, c = _inputs(9, t, d, v, dtype)
    _, lse = _forward(gpu_lib, h, w, y)
    gh, gw = _backward(gpu_lib, h, w, y, lse, c)
    rng = np.random.default_rng(1)
    hv, wv, yv, cv = _np(h), _np(w), np.asarray(y.cpu()), _np(c)
    for val, grad, which in ((hv, _np(gh), 0), (wv, _np(gw), 1)):
        e = rng.standard_normal(val.shape)
        step = 1e-5

        def f(s):
            args = (hv + s * e, wv) if which == 0 else (hv, wv + s * e)
            return float((cv * to.token_logp(*args, yv)[0]).sum())
        num = (f(step) - f(-step)) / (2 * step)
        size = np.sqrt((grad * grad).sum())     # a random direction sees rounding of about |grad| ROUND
        assert abs((grad * e).sum() - num) <= 8 * max(ROUND[dtype], 2.0 ** -20) * size + 1e-7


def test_token_logp_in_a_graph_and_on_another_stream(gpu_lib):
    import torch
    h, w, y, c = _inputs(10, 300, 256, 1111, "bf16")
    for t in (2, 300):
        h, y, c = h[:t], y[:t], c[:t]
        saved = _saved(gpu_lib, h, w)
        need = max(gpu_lib.muon_token_logp_workspace_bytes(h, w),
                   gpu_lib.muon_token_logp_backward_workspace_bytes(h, w, use_saved=True))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        def buffers():
            return [torch.empty(t, device="cuda"), torch.empty(t, device="cuda"), torch.empty_like(h), torch.empty_like(w)]
        def call(b, stream=None):
            gpu_lib.muon_token_logp(h, w, y, b[0], b[1], saved=saved, workspace=ws, stream=stream)
            gpu_lib.muon_token_logp_backward(h, w, y, b[1], c, b[2], b[3], saved=saved, workspace=ws, stream=stream)
        want, got = buffers(), buffers()
        call(want)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        call(got, side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(got)
        for _ in range(3):
            for b in got + [saved, ws]:
                b.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        h, w, y, c = _inputs(10, 300, 256, 1111, "bf16")


@pytest.mark.parametrize("hs,ws", [(1e-20, 1e18), (1e12, 1e-13), (2e-38, 1e36)])
@pytest.mark.parametrize("t", [20, 150])
def test_token_logp_fp32_magnitudes(gpu_lib, t, hs, ws):
    # the logits of ordinary size from operands far from it, and a gradient of 1e-15; then one huge entry of head that
    # meets zeros of hidden
    import torch
    h, w, y, c = _inputs(23, t, 96, 1500, "f32")
    h, w, c = h * hs, w * ws, c * 1e-15
    scale = 1.0 / (np.float64(hs) * ws)
    for big in (False, True):
        if big and 1e6 * ws > 3e38:
            break                                              # not an fp32 value
        if big:
            h[:, 5] = 0
            w[7, 5] = 1e6 * ws
        saved = _saved(gpu_lib, h, w)
        logp, lse = _forward(gpu_lib, h, w, y, scale, saved=saved)
        hv, wv = _np(h) / hs, _np(w) / ws                      # the same problem in ordinary size
        rl, _, _ = to.token_logp(hv, wv, np.asarray(y.cpu()), scale=np.float32(scale) * np.float64(hs) * ws)
        assert np.all(np.abs(_np(logp) - rl) <= 1e-4)
        gh, gw = _backward(gpu_lib, h, w, y, lse, c, scale, saved=saved)
        rh, rw, _, _ = to.token_logp_backward(hv, wv, np.asarray(y.cpu()), _np(c), scale=1.0)
        for got, ref in ((gh, rh / hs), (gw, rw / ws)):
            g, ref = _np(got), ref.astype(np.float32).astype(np.float64)   # 1e-56 is 0 in fp32
            assert np.linalg.norm(g - ref) <= 1e-4 * np.linalg.norm(ref)


# products with enough 256 x 256 tiles for the chip (the shapes above take the smaller tile), widths that end inside a k-step
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,d,v", [(600, 72, 20000), (520, 1100, 16500), (1500, 136, 8200)])
def test_token_logp_many_tiles(gpu_lib, t, d, v, dtype):
    import torch
    print("[token_logp many tiles]", t, d, v, dtype, flush=True)
    h, w, y, c = _inputs(21, t, d, v, dtype)
    saved = _saved(gpu_lib, h, w)
    logp, lse = _forward(gpu_lib, h, w, y, saved=saved)
    _check_forward(h, w, y, 1.0, dtype, logp, lse)
    _check_backward(h, w, y, c, 1.0, dtype, *_backward(gpu_lib, h, w, y, lse, c, saved=saved))
    plain = _forward(gpu_lib, h, w, y)
    assert torch.equal(plain[0], logp) and torch.equal(plain[1], lse)
    _check_backward(h, w, y, c, 1.0, dtype, *_backward(gpu_lib, h, w, y, lse, c))


@pytest.mark.parametrize("use_saved", [True, False])
def test_token_logp_tokens_in_chunks(gpu_lib, use_saved):
    # dz of 6000 tokens x 65536 entries in fp32 is beyond what the backward pass forms at once, so the tokens go in
    # two chunks whose grad_head adds up; against fp64 on the GPU, by norms: every gradient entry is a sum whose terms
    # are within a few 2^-21 of exact, and 1e-5 is forty times that
    import torch
    t, d, v = 6000, 32, 65536
    h, w, y, c = _inputs(22, t, d, v, "f32")
    saved = _saved(gpu_lib, h, w) if use_saved else None
    _, lse = _forward(gpu_lib, h, w, y, saved=saved)
    gh, gw = _backward(gpu_lib, h, w, y, lse, c, saved=saved)
    H, W = h.double(), w.double()
    rh, rw = torch.zeros_like(H), torch.zeros_like(W)
    for rows in torch.nonzero(y >= 0)[:, 0].split(1000):
        dz = -torch.softmax(H[rows] @ W.T, 1)
        dz[torch.arange(len(rows), device="cuda"), y[rows]] += 1
        dz *= c[rows].double()[:, None]
        rh[rows] = dz @ W
        rw += dz.T @ H[rows]
    for got, ref in ((gh, rh), (gw, rw)):
        assert float((got.double() - ref).norm() / ref.norm()) <= 1e-5
    assert not gh[y < 0].any()


# bf16 calls of up to 64 tokens: dz goes as two bf16 parts (2^-16 of it is lost) formed from exp(z - m) in fp16 (2^-11 of it,
# and 2^-25 of the largest p below fp16's normal range), so the bounds are tighter than in the general case
@pytest.mark.parametrize("t,d,v", [(1, 7, 33), (15, 131, 4100), (16, 1000, 95), (31, 130, 513), (33, 264, 1027), (64, 77, 2000)])
@pytest.mark.parametrize("scale", [0.8, -1.3])
@pytest.mark.parametrize("use_saved", [True, False])
def test_token_logp_few_tokens_gradients(gpu_lib, t, d, v, scale, use_saved):
    print("[token_logp few]", t, d, v, scale, use_saved, flush=True)
    h, w, y, c = _inputs(t * 31 + d, t, d, v, "bf16", ignored=0.25 if t > 1 else 0.0)
    saved = _saved(gpu_lib, h, w) if use_saved else None
    logp, lse = _forward(gpu_lib, h, w, y, scale, saved=saved)
    _check_forward(h, w, y, scale, "bf16", logp, lse)
    gh, gw = _backward(gpu_lib, h, w, y, lse, c, scale, saved=saved)
    hv, wv, E, sums = _bounds(h, w, y, scale, "bf16")
    yv, cv = np.asarray(y.cpu()), _np(c)
    rh, rw, dz, p = to.token_logp_backward(hv, wv, yv, cv, scale=np.float32(scale))
    off = np.abs(dz) * 2.0 ** -16 + np.abs(scale * cv)[:, None] * (p * (2.0 ** -11 + 2 * E[:, None] + sums) + 2.0 ** -25 * p.max(1)[:, None])
    b = off @ np.abs(wv) + (v / 16 + 32) * U * (np.abs(dz) @ np.abs(wv)) + ROUND["bf16"] * np.abs(rh) + 1e-38
    assert np.all(np.abs(_np(gh) - rh) <= b), float(np.max(np.abs(_np(gh) - rh) / b))
    b = off.T @ np.abs(hv) + (t / 16 + 32) * U * (np.abs(dz).T @ np.abs(hv)) + ROUND["bf16"] * np.abs(rw) + 1e-38
    assert np.all(np.abs(_np(gw) - rw) <= b), float(np.max(np.abs(_np(gw) - rw) / b))
    assert not _np(gh)[yv < 0].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [3, 70, 300])
@pytest.mark.parametrize("scale", [-2.0, 0.0])
@pytest.mark.parametrize("use_saved", [True, False])
def test_token_logp_scales_of_any_sign(gpu_lib, dtype, t, scale, use_saved):
    print("[token_logp scale]", t, dtype, scale, use_saved, flush=True)
    h, w, y, c = _inputs(41, t, 96, 700, dtype)
    saved = _saved(gpu_lib, h, w) if use_saved else None
    logp, lse = _forward(gpu_lib, h, w, y, scale, saved=saved)
    _check_forward(h, w, y, scale, dtype, logp, lse)
    _check_backward(h, w, y, c, scale, dtype, *_backward(gpu_lib, h, w, y, lse, c, scale, saved=saved))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [4, 90, 300])
@pytest.mark.parametrize("use_saved", [True, False])
def test_token_logp_target_far_below_the_best(gpu_lib, dtype, t, use_saved):
    # logits 300 apart in exact arithmetic: the target's probability is 0 in fp32, the best token's 1
    import torch
    h, w, y, c = _inputs(42, t, 64, 500, dtype, ignored=0.0, lift=0.0)
    h[:, :2], w[:, :2] = 0, 0
    w[7, 0], w[8, 0] = 16, -16
    h[0, 0], h[1, 0] = 16, -16                        # 7 wins by 256 (over 8, by 512), or 8 does
    y[0], y[1], y[2] = 8, 11, 499
    saved = _saved(gpu_lib, h, w) if use_saved else None
    logp, lse = _forward(gpu_lib, h, w, y, saved=saved)
    _check_forward(h, w, y, 1.0, dtype, logp, lse)
    assert float(logp[0]) < -500 and float(logp[1]) < -200
    gh, gw = _backward(gpu_lib, h, w, y, lse, c, saved=saved)
    _check_backward(h, w, y, c, 1.0, dtype, gh, gw)
    assert torch.isfinite(gh).all() and torch.isfinite(gw).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [20, 100, 300])
@pytest.mark.parametrize("use_saved", [True, False])
def test_token_logp_gradient_of_certain_tokens(gpu_lib, dtype, t, use_saved):
    # Token i's target stands x_i above v - 1 equal logits of 0, in exact arithmetic, and column 1 of head holds nothing but
    # the target: grad_hidden[i, 1] = c_i (1 - p) = -c_i expm1(logp), from 6e-3 down to 2e-6 of c_i.  Its relative error: the sum
    # of v terms (v / 64 + 64) u, 2^(k x) with k x rounded at 32 (2^-19 ln 2), dz's and the output's rounding.
    import torch
    print("[token_logp certain]", t, dtype, use_saved, flush=True)
    d, v = 64, 900
    x = torch.tensor([12.0, 16.0, 18.5, 20.0], device="cuda").repeat(t // 4)
    h, w = torch.zeros((t, d), device="cuda"), torch.zeros((v, d), device="cuda")
    w[7, 1] = 1.0
    h[:, 1] = x
    h, w = h.to(_dt(dtype)), w.to(_dt(dtype))
    y = torch.full((t,), 7, dtype=torch.int64, device="cuda")
    c = torch.linspace(0.5, 1.0, t, device="cuda")
    saved = _saved(gpu_lib, h, w) if use_saved else None
    logp, lse = _forward(gpu_lib, h, w, y, saved=saved)
    gh, gw = _backward(gpu_lib, h, w, y, lse, c, saved=saved)
    rest = (v - 1) * np.exp(-_np(x))
    ref = _np(c) * rest / (1 + rest)
    tol = (v / 64 + 64) * U + 2.0 ** -19 + PARTS[dtype] + ROUND[dtype]
    err = np.abs(_np(gh)[:, 1] - ref) / ref
    assert err.max() <= tol, (float(err.max()), tol)
    assert abs(_np(gw)[7, 1] - (ref * _np(x)).sum()) <= tol * (ref * _np(x)).sum()


@pytest.mark.parametrize("t,v,dtype", [(20, 100, "bf16"), (20, 900, "bf16"), (100, 100, "bf16"), (300, 900, "bf16"),
                                       (600, 17000, "bf16"), (20, 100, "f32"), (20, 900, "f32"), (100, 100, "f32"),
                                       (300, 900, "f32"), (600, 17000, "f32")])
@pytest.mark.parametrize("use_saved", [True, False])
def test_token_logp_gradients_beside_a_certain_target(gpu_lib, dtype, t, v, use_saved):
    # The target stands 12 to 24 above entries of logits 0 .. -3 (exact arithmetic): column 0 of grad_hidden sums over the other
    # entries of the target's tile alone, and the rows of grad_head hold one entry's share each.  Relative to fp64, term by
    # term of one sign: exp(z - m) in fp16 2^-11, then as in test_token_logp_gradient_of_certain_tokens.
    import torch
    print("[token_logp beside]", t, v, dtype, use_saved, flush=True)
    d = 64
    x = torch.tensor([12.0, 16.0, 20.0, 24.0], device="cuda").repeat(t // 4)
    h, w = torch.zeros((t, d), device="cuda"), torch.zeros((v, d), device="cuda")
    w[:100, 0] = 1.0
    w[7, 0], w[7, 1] = 0.0, 1.0
    w[:, 2] = -(torch.arange(v, device="cuda") % 4).float()
    w[7, 2] = 0.0
    h[:, 1], h[:, 2] = x, 1.0
    h, w = h.to(_dt(dtype)), w.to(_dt(dtype))
    y = torch.full((t,), 7, dtype=torch.int64, device="cuda")
    c = torch.linspace(0.5, 1.0, t, device="cuda")
    saved = _saved(gpu_lib, h, w) if use_saved else None
    logp, lse = _forward(gpu_lib, h, w, y, saved=saved)
    z = _np(h) @ _np(w).T
    others = np.exp(z)
    others[:, 7] = 0.0
    rest = others.sum(1) * np.exp(-_np(x))
    assert np.all(np.abs(_np(logp) + np.log1p(rest)) <= ((v / 64 + 64) * U + 2.0 ** -19) * rest)
    gh, gw = _backward(gpu_lib, h, w, y, lse, c, saved=saved)
    dz = -_np(c)[:, None] * others * np.exp(-_np(x))[:, None] / (1 + rest)[:, None]
    tol = (v / 64 + 64) * U + 2.0 ** -19 + PARTS[dtype] + ROUND[dtype] + (2.0 ** -11 if dtype == "bf16" else 0.0)
    ref = dz @ _np(w)[:, 0]
    assert np.all(np.abs(_np(gh)[:, 0] - ref) <= tol * np.abs(ref)), float(np.max(np.abs(_np(gh)[:, 0] / ref - 1)))
    ref = dz.sum(0)
    keep = np.arange(v) != 7
    assert np.all(np.abs(_np(gw)[:, 2] - ref)[keep] <= (tol + (t / 16) * U) * np.abs(ref)[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,v", [(40, 500), (100, 500), (300, 2000)])
@pytest.mark.parametrize("use_saved", [True, False])
def test_token_logp_gradients_of_uneven_tokens(gpu_lib, dtype, t, v, use_saved):
    # incoming gradients from 1 down to 1e-14, tokens from unsure to certain: the bounds are relative to each token's own c, so
    # a token's row of grad_hidden may not lose bits beside the others
    import torch
    print("[token_logp uneven]", t, v, dtype, use_saved, flush=True)
    h, w, y, _ = _inputs(51, t, 96, v, dtype, ignored=0.2, lift=15.0)
    c = (torch.logspace(0, -14, t, dtype=torch.float64) * (1 - 2 * (torch.arange(t) % 2))).float().cuda()
    saved = _saved(gpu_lib, h, w) if use_saved else None
    logp, lse = _forward(gpu_lib, h, w, y, saved=saved)
    _check_forward(h, w, y, 1.0, dtype, logp, lse)
    _check_backward(h, w, y, c, 1.0, dtype, *_backward(gpu_lib, h, w, y, lse, c, saved=saved))


@pytest.mark.parametrize("t,d,v", [(65, 200, 1025), (300, 256, 3000), (1030, 192, 700), (600, 72, 20000)])
@pytest.mark.parametrize("use_saved", [True, False])
def test_token_logp_bf16_gradients_cost_little_more_than_their_rounding(gpu_lib, t, d, v, use_saved):
    # dz and exp(z - m) carry 11 bits: each entry of dz is off by at most 2^-12 + 2^-12 of itself, so the gradients, as sums of
    # independent errors, by less than 2^-11 of the root of the sum of their terms' squares (twice that square here, for
    # chance), beside the rounding of the output (its square within 10 %).  With 8 bits in dz the squares come to twice that.
    import torch
    print("[token_logp bits]", t, d, v, use_saved, flush=True)
    h, w, y, c = _inputs(61, t, d, v, "bf16")
    saved = _saved(gpu_lib, h, w) if use_saved else None
    _, lse = _forward(gpu_lib, h, w, y, saved=saved)
    gh, gw = _backward(gpu_lib, h, w, y, lse, c, saved=saved)
    hv, wv, yv = _np(h), _np(w), np.asarray(y.cpu())
    rh, rw, dz, _ = to.token_logp_backward(hv, wv, yv, _np(c))
    hv = np.where((yv >= 0)[:, None], hv, 0.0)
    for got, ref, terms in ((gh, rh, (dz ** 2) @ (wv ** 2)), (gw, rw, (dz ** 2).T @ (hv ** 2))):
        rounded = _np(torch.from_numpy(ref).to(torch.bfloat16))
        most = 1.1 * ((rounded - ref) ** 2).sum() + 2 * 2.0 ** -22 * terms.sum()
        assert ((_np(got) - ref) ** 2).sum() <= most, float(((_np(got) - ref) ** 2).sum() / most)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [5, 40, 300])
@pytest.mark.parametrize("use_saved", [True, False])
def test_token_logp_huge_values_in_unscored_rows(gpu_lib, dtype, t, use_saved):
    # finite values near the type's end in rows that are not scored: the same bits as without them
    import torch
    print("[token_logp huge]", t, dtype, use_saved, flush=True)
    h, w, y, c = _inputs(71, t, 128, 600, dtype, ignored=0.4)
    y[0], y[1] = 3, -100
    huge = h.clone()
    dead = (y < 0).nonzero()[:, 0]
    huge[dead] = torch.finfo(_dt(dtype)).min
    huge[dead[::2], 1::3] = torch.finfo(_dt(dtype)).max
    out = []
    for x in (h, huge):
        saved = _saved(gpu_lib, x, w) if use_saved else None
        logp, lse = _forward(gpu_lib, x, w, y, saved=saved)
        out.append((logp, lse, *_backward(gpu_lib, x, w, y, lse, c, saved=saved)))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_token_logp_more_tiles_than_a_launch_has_threads(gpu_lib):
    # 2^23 tiles of 512 threads; tokens from the first, middle and last tiles against the oracle
    import torch
    t, d, v = 1 << 20, 8, (1 << 19) + 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("40 GB needed")
    g = torch.Generator(device="cuda").manual_seed(3)
    h, w = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((t, d), (v, d)))
    y = torch.randint(0, v, (t,), generator=g, device="cuda")
    logp, lse = _forward(gpu_lib, h, w, y)
    pick = torch.cat([torch.arange(a, a + 8, device="cuda") for a in (0, 255, t // 2 - 4, t - 8)])
    _check_forward(h[pick], w, y[pick], 1.0, "bf16", logp[pick], lse[pick])
    assert torch.isfinite(logp).all() and torch.isfinite(lse).all()


def test_token_logp_more_tokens_than_a_launch_has_threads(gpu_lib):
    # 2^29 tokens: eight threads a token where the tiles' statistics are joined
    import torch
    t, d, v = (1 << 29) + 7, 8, 3
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GB needed")
    period = 1 << 16
    hp, w, yp, _ = _inputs(81, period, d, v, "bf16")
    base = _forward(gpu_lib, hp, w, yp)
    _check_forward(hp, w, yp, 1.0, "bf16", *base)
    h, y = torch.empty((t, d), dtype=torch.bfloat16, device="cuda"), torch.empty((t,), dtype=torch.int64, device="cuda")
    full = t // period
    h[:full * period].view(full, period, d).copy_(hp.expand(full, period, d))
    y[:full * period].view(full, period).copy_(yp.expand(full, period))
    h[full * period:], y[full * period:] = hp[:t - full * period], yp[:t - full * period]
    for got, ref in zip(_forward(gpu_lib, h, w, y), base):
        assert bool((got[:full * period].view(full, period) == ref).all()) and torch.equal(got[full * period:], ref[:t - full * period])
