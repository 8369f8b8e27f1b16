"""GPU parity of the norms around a block against the fp64 oracle (through the public entry points).

Bounds, elementwise, with u = 2^-24.  A sum over d products of fp32 values is within
(d / 64 + 16) u of the sum of their magnitudes for any order the kernels use (at most d / 64
terms in a thread's chain, then a tree); 1 / sqrt adds a few u.  A factor K = d / 32 + 64 covers the
sums, the inverse roots and the products of one element.  Sums over the rows are chains of at
most `rows` additions.  An output's own rounding is u of it in fp32 and 2^-8 of it in bf16.
"""
import numpy as np
import pytest

from oracle import train_oracle as to

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {"f32": 2 * U, "bf16": 2.0 ** -8}


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _draw(rng, shape, dtype, std=1.0, mean=0.0):
    """A tensor on the GPU and the fp64 values it holds."""
    import torch
    t = torch.from_numpy((mean + std * rng.standard_normal(shape)).astype(np.float32)).to(_dt(dtype))
    return t.cuda(), t.double().numpy()


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(got, ref, bound, what):
    got = _np(got)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - ref) / (bound + 1e-300))))


def _case(rng, rows, cols, dtype, wdtype, gate, post=True, pre=True):
    ten, val = {}, {}
    for k, std in (("x", 1.0), ("residual", 2.0), ("grad_norm", 1e-2), ("grad_out_residual", 1e-2)):
        ten[k], val[k] = _draw(rng, (rows, cols), dtype, std)
    ten["post_weight"], val["post_weight"] = _draw(rng, (cols,), wdtype, 0.2, 1.0) if post else (None, None)
    ten["pre_weight"], val["pre_weight"] = _draw(rng, (cols,), wdtype, 0.2, 1.0) if pre else (None, None)
    ten["gate"], val["gate"] = None, None
    if gate == "channel":
        ten["gate"], val["gate"] = _draw(rng, (cols,), wdtype, 0.3, 0.5)
    elif gate == "full":
        ten["gate"], val["gate"] = _draw(rng, (rows, cols), dtype, 0.3, 0.5)
    return ten, val


ALPHA, EPS = 0.75, 1e-5


def _forward(mao, ten, with_rstd=True, **kw):
    import torch
    x = ten["x"]
    out_r = torch.full_like(x, float("nan"))
    out_n = torch.full_like(x, float("nan")) if ten["pre_weight"] is not None else None
    rstd = torch.full((2, x.shape[0]), float("nan"), device="cuda") if with_rstd else None
    mao.muon_block_norm(x, ten["residual"], out_r, out_n, post_weight=ten["post_weight"], gate=ten["gate"],
                        pre_weight=ten["pre_weight"], rstd=rstd, residual_scale=ALPHA, eps=EPS, **kw)
    return out_r, out_n, rstd


def _check_forward(ten, val, out_r, out_n, rstd, dtype):
    kw = {k: val[k] for k in ("post_weight", "gate", "pre_weight")}
    f = to.block_norm(val["x"], val["residual"], residual_scale=np.float32(ALPHA), eps=np.float32(EPS), **kw)
    d = val["x"].shape[1]
    K = d / 32 + 64
    size = np.abs(ALPHA * val["residual"]) + np.abs(f["r"] - np.float32(ALPHA) * val["residual"])
    _near(out_r, f["r"], K * U * size + ROUND[dtype] * np.abs(f["r"]) + 1e-38, "r")
    if out_n is not None:
        s1 = f["rstd1"][:, None]
        rel = K * U * (1 + (size * size).mean(1, keepdims=True) * s1 * s1)
        _near(out_n, f["n"], np.abs(s1 * val["pre_weight"]) * K * U * size + (rel + ROUND[dtype]) * np.abs(f["n"]) + 1e-38, "n")
    if rstd is not None:
        _near(rstd[0], f["rstd0"], K * U * f["rstd0"], "rstd0")
        if out_n is not None:
            _near(rstd[1], f["rstd1"], K * U * f["rstd1"] * (1 + (size * size).mean(1) * f["rstd1"] ** 2), "rstd1")
        else:
            assert (_np(rstd[1]) == 1).all()


def _backward(mao, ten, out_r, rstd, use_norm=True, use_res=True):
    import torch
    g = {"grad_x": torch.full_like(ten["x"], float("nan")), "grad_residual": torch.full_like(ten["x"], float("nan"))}
    for k in ("post_weight", "gate", "pre_weight"):
        g["grad_" + k] = None if ten[k] is None else torch.full_like(ten[k], float("nan"))
    mao.muon_block_norm_backward(
        ten["x"], out_r, rstd, ten["grad_norm"] if use_norm else None, g["grad_x"], g["grad_residual"],
        grad_out_residual=ten["grad_out_residual"] if use_res else None, post_weight=ten["post_weight"],
        gate=ten["gate"], pre_weight=ten["pre_weight"], grad_post_weight=g["grad_post_weight"],
        grad_gate=g["grad_gate"], grad_pre_weight=g["grad_pre_weight"], residual_scale=ALPHA)
    return g


def _check_backward(ten, val, out_r, rstd, g, dtype, wdtype, use_norm=True, use_res=True):
    r, s0, s1 = _np(out_r), _np(rstd[0]), _np(rstd[1])
    dn = val["grad_norm"] if use_norm else None
    dr = val["grad_out_residual"] if use_res else None
    wp, gate, wq = val["post_weight"], val["gate"], val["pre_weight"]
    b = to.block_norm_backward(val["x"], r, s0, s1, dn, dr, post_weight=wp, gate=gate, pre_weight=wq,
                               residual_scale=np.float32(ALPHA))
    rows, d = val["x"].shape
    K = d / 32 + 64
    # sums of magnitudes in place of sums
    tot = np.zeros((rows, d)) if dr is None else np.abs(dr)
    hs = np.abs(r * s1[:, None])
    if dn is not None:
        dh = np.abs(dn * wq)
        tot = tot + s1[:, None] * (dh + hs * (dh * hs).mean(1, keepdims=True))
    ga = 1.0 if gate is None else np.abs(gate)
    w = 1.0 if wp is None else np.abs(wp)
    xs = np.abs(val["x"]) * (1.0 if wp is None else s0[:, None])
    dxh = tot * ga * w
    dx = dxh if wp is None else s0[:, None] * (dxh + xs * (dxh * xs).mean(1, keepdims=True))
    R, RW = ROUND[dtype], ROUND[wdtype]
    _near(g["grad_x"], b["x"], K * U * dx + R * np.abs(b["x"]) + 1e-38, "grad_x")
    _near(g["grad_residual"], b["residual"], K * U * ALPHA * tot + R * np.abs(b["residual"]) + 1e-38, "grad_residual")
    KR = K + rows
    if wp is not None:
        _near(g["grad_post_weight"], b["post_weight"], KR * U * (tot * ga * xs).sum(0) + RW * np.abs(b["post_weight"]) + 1e-38,
              "grad_post_weight")
    if wq is not None:
        size = (np.abs(dn) * hs).sum(0) if dn is not None else 0.0
        _near(g["grad_pre_weight"], b["pre_weight"], KR * U * size + RW * np.abs(b["pre_weight"]) + 1e-38, "grad_pre_weight")
    if gate is not None:
        if gate.ndim == 1:
            _near(g["grad_gate"], b["gate"], KR * U * (tot * xs * w).sum(0) + RW * np.abs(b["gate"]) + 1e-38, "grad_gate")
        else:
            _near(g["grad_gate"], b["gate"], K * U * tot * xs * w + R * np.abs(b["gate"]) + 1e-38, "grad_gate")


SHAPES = [(1, 1), (1, 2048), (3, 7), (2, 255), (5, 256), (33, 1000), (7, 2049), (300, 513), (2, 8192), (3, 16384), (2, 20001),
          (2, 32768), (1031, 64)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_block_norm_shapes(gpu_lib, rows, cols, dtype, wdtype):
    gate = ("channel", "full", "none")[(rows + cols) % 3]
    print("[block_norm]", rows, cols, dtype, wdtype, gate, flush=True)
    ten, val = _case(np.random.default_rng(rows * 100003 + cols), rows, cols, dtype, wdtype, gate)
    out_r, out_n, rstd = _forward(gpu_lib, ten)
    _check_forward(ten, val, out_r, out_n, rstd, dtype)
    g = _backward(gpu_lib, ten, out_r, rstd)
    _check_backward(ten, val, out_r, rstd, g, dtype, wdtype)
    # the same call again gives the same bits
    again = _backward(gpu_lib, ten, out_r, rstd)
    import torch
    for k, v in g.items():
        assert v is None or torch.equal(v, again[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "channel", "full"])
@pytest.mark.parametrize("post,pre,use_norm,use_res", [(True, True, True, False), (True, True, False, True),
                                                       (False, True, True, True), (True, False, False, True),
                                                       (False, False, False, True)])
def test_block_norm_parts(gpu_lib, dtype, gate, post, pre, use_norm, use_res):
    for rows, cols in ((9, 640), (4, 333)):
        print("[block_norm parts]", rows, cols, dtype, gate, post, pre, use_norm, use_res, flush=True)
        ten, val = _case(np.random.default_rng(11), rows, cols, dtype, dtype, gate, post, pre)
        out_r, out_n, rstd = _forward(gpu_lib, ten)
        _check_forward(ten, val, out_r, out_n, rstd, dtype)
        g = _backward(gpu_lib, ten, out_r, rstd, use_norm, use_res)
        _check_backward(ten, val, out_r, rstd, g, dtype, dtype, use_norm, use_res)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_norm_strides_offsets_and_in_place(gpu_lib, dtype):
    import torch
    rng = np.random.default_rng(12)
    for rows, cols, pitch, shift in ((6, 512, 520, 0), (6, 512, 515, 1), (5, 301, 400, 3)):
        print("[block_norm strides]", rows, cols, pitch, shift, dtype, flush=True)
        ten, val = _case(rng, rows, cols, dtype, dtype, "full")
        wide = {}
        for k in ("x", "residual", "gate", "grad_norm", "grad_out_residual"):
            buf = torch.full((rows * pitch + shift,), float("nan"), dtype=_dt(dtype), device="cuda")
            view = buf[shift:].view(rows, pitch)[:, :cols]
            view.copy_(ten[k])
            wide[k] = view
        ten.update(wide)
        out_r, out_n, rstd = _forward(gpu_lib, ten)
        _check_forward(ten, val, out_r, out_n, rstd, dtype)
        g = _backward(gpu_lib, ten, out_r, rstd)
        _check_backward(ten, val, out_r, rstd, g, dtype, dtype)
        # in place: r' over the residual, its gradient over the incoming one
        pad = wide["residual"].storage_offset() + cols
        gpu_lib.muon_block_norm(ten["x"], wide["residual"], wide["residual"], None, post_weight=ten["post_weight"],
                                gate=ten["gate"], residual_scale=ALPHA, eps=EPS)
        assert torch.equal(wide["residual"], out_r)
        assert torch.isnan(wide["residual"].as_strided((1,), (1,), pad)).all()      # the padding is untouched
        g2 = torch.empty_like(g["grad_x"])
        args = [torch.empty_like(t) for t in (ten["post_weight"], ten["gate"], ten["pre_weight"])]
        gpu_lib.muon_block_norm_backward(ten["x"], out_r, rstd, ten["grad_norm"], g2, wide["grad_out_residual"],
                                         grad_out_residual=wide["grad_out_residual"], post_weight=ten["post_weight"],
                                         gate=ten["gate"], pre_weight=ten["pre_weight"], grad_post_weight=args[0],
                                         grad_gate=args[1], grad_pre_weight=args[2], residual_scale=ALPHA)
        assert torch.equal(wide["grad_out_residual"], g["grad_residual"]) and torch.equal(g2, g["grad_x"])


def test_block_norm_no_rows_writes_zero_weight_gradients(gpu_lib):
    import torch
    ten, _ = _case(np.random.default_rng(1), 1, 96, "bf16", "bf16", "channel")
    for k in ("x", "residual", "grad_norm", "grad_out_residual"):
        ten[k] = ten[k][:0]
    out_r, _, rstd = _forward(gpu_lib, ten)
    g = _backward(gpu_lib, ten, out_r, rstd)
    assert all(not torch.count_nonzero(g["grad_" + k]) for k in ("post_weight", "gate", "pre_weight"))


def test_block_norm_zero_rows_of_zeros_and_nan_rows_stay_apart(gpu_lib):
    # a row of zeros gives rstd = 1 / sqrt(eps) and finite results; a NaN row stays in its row
    import torch
    ten, val = _case(np.random.default_rng(2), 4, 384, "f32", "f32", "none")
    for k in ("x", "residual"):
        ten[k][1] = 0
        val[k][1] = 0
    out_r, out_n, rstd = _forward(gpu_lib, ten)
    _check_forward(ten, val, out_r, out_n, rstd, "f32")
    ten["x"][2] = float("nan")
    again = _forward(gpu_lib, ten)
    keep = [0, 1, 3]
    assert torch.equal(again[0][keep], out_r[keep]) and torch.equal(again[1][keep], out_n[keep])
    assert torch.isnan(again[0][2]).all()


def test_block_norm_on_another_stream_and_in_a_graph(gpu_lib):
    import torch
    ten, val = _case(np.random.default_rng(3), 64, 2048, "bf16", "bf16", "channel")
    ref = _forward(gpu_lib, ten)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(t) for t in ref]
    def call(stream=None):
        gpu_lib.muon_block_norm(ten["x"], ten["residual"], out[0], out[1], post_weight=ten["post_weight"],
                                gate=ten["gate"], pre_weight=ten["pre_weight"], rstd=out[2], residual_scale=ALPHA,
                                eps=EPS, stream=stream)
    call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("rows,cols", [((1 << 26) + 5, 8), ((1 << 24) + 3, 1032), ((1 << 22) + 3, 4100)])
def test_block_norm_more_rows_than_a_launch_has_threads(gpu_lib, rows, cols):
    # 64, 256 and 1024 threads a row: 2^32 threads are more than one launch takes.  The same 64 rows over and over: each has the bits
    # that it has in a small call.
    import torch
    print("[block_norm rows]", rows, cols, flush=True)
    need = rows * cols * 2 * 3
    if torch.cuda.mem_get_info()[0] < need + (16 << 30):
        pytest.skip(f"{need >> 30} GB needed")
    period, full = 64, rows // 64
    ten, _ = _case(np.random.default_rng(8), period, cols, "bf16", "bf16", "channel")
    want = _forward(gpu_lib, ten)
    wide = {}
    for k in ("x", "residual"):
        wide[k] = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        wide[k][:full * period].view(full, period, cols).copy_(ten[k].expand(full, period, cols))
        wide[k][full * period:] = ten[k][:rows - full * period]
    rstd = torch.zeros((2, rows), device="cuda")
    norm = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    gpu_lib.muon_block_norm(wide["x"], wide["residual"], wide["residual"], norm, post_weight=ten["post_weight"], gate=ten["gate"],
                            pre_weight=ten["pre_weight"], rstd=rstd, residual_scale=ALPHA, eps=EPS)
    for got, ref in ((wide["residual"], want[0]), (norm, want[1]), (rstd[0][:, None], want[2][0][:, None]), (rstd[1][:, None], want[2][1][:, None])):
        for a in range(0, full, 1 << 14):
            part = got[a * period:min(full, a + (1 << 14)) * period]
            assert bool((part.reshape(-1, period, part.shape[1]) == ref).all())
        assert torch.equal(got[full * period:], ref[:rows - full * period])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_norm_on_column_ranges_of_one_buffer(gpu_lib, dtype):
    # every matrix of a call a range of columns of one wide buffer
    import torch
    rows, cols = 37, 301
    ten, _ = _case(np.random.default_rng(21), rows, cols, dtype, dtype, "full")
    want = _forward(gpu_lib, ten)
    back = _backward(gpu_lib, ten, want[0], want[2])
    wide = torch.full((rows, 8 * cols), float("nan"), dtype=_dt(dtype), device="cuda")
    part = [wide[:, k * cols:(k + 1) * cols] for k in range(8)]
    for k, name in enumerate(("x", "residual", "gate")):
        part[k].copy_(ten[name])
    rstd = torch.empty_like(want[2])
    gpu_lib.muon_block_norm(part[0], part[1], part[3], part[4], post_weight=ten["post_weight"], gate=part[2], pre_weight=ten["pre_weight"],
                            rstd=rstd, residual_scale=ALPHA, eps=EPS)
    assert torch.equal(part[3], want[0]) and torch.equal(part[4], want[1]) and torch.equal(rstd, want[2])
    part[1].copy_(ten["grad_norm"])
    part[4].copy_(ten["grad_out_residual"])
    weights = {k: torch.empty_like(ten[k]) for k in ("post_weight", "pre_weight")}
    gpu_lib.muon_block_norm_backward(part[0], part[3], rstd, part[1], part[5], part[6], grad_out_residual=part[4], post_weight=ten["post_weight"],
                                     gate=part[2], pre_weight=ten["pre_weight"], grad_post_weight=weights["post_weight"], grad_gate=part[7],
                                     grad_pre_weight=weights["pre_weight"], residual_scale=ALPHA)
    for got, name in ((part[5], "grad_x"), (part[6], "grad_residual"), (part[7], "grad_gate"), (weights["post_weight"], "grad_post_weight"),
                      (weights["pre_weight"], "grad_pre_weight")):
        assert torch.equal(got, back[name]), name
