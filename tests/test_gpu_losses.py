"""GPU parity of the preference and policy losses against the fp64 oracle (through the public entry points).

Bounds, with u = 2^-24.  A sum of n fp32 terms in the kernels' orders is within (n / 64 + 64) u
of the sum of the magnitudes (chains of at most n / 64 terms a thread, then trees; short inputs are
covered by the 64).  A log ratio lp - old of fp32 values is rounded once, so exp of it is
within (|lp - old| + 4) u, relative; expf and expm1f are within 2 ulp.
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


def _put(x, dtype):
    """(GPU tensor in dtype, the fp64 values it holds); None passes through."""
    import torch
    if x is None:
        return None, None
    t = torch.from_numpy(np.asarray(x, np.float32)).to(_dt(dtype))
    return t.cuda(), t.double().numpy()


def _np(t):
    return t.detach().double().cpu().numpy()


def _offsets(lengths, before=0):
    return np.concatenate([[before], before + np.cumsum(lengths)]).astype(np.int64)


def _lengths(rng, name, count):
    if name == "ones":
        return np.ones(count, np.int64)
    if name == "empty":
        return np.zeros(count, np.int64)
    if name == "ragged":
        return rng.integers(0, 700, count)
    if name == "skewed":       # one very long sequence among short ones
        n = rng.integers(0, 5, count)
        n[count // 2] = 70001
        return n
    return np.full(count, 4096)


LAYOUTS = [("ragged", 2), ("ragged", 64), ("ones", 5000), ("empty", 6), ("skewed", 40), ("tile", 8), ("ragged", 1000)]


def _inputs(seed, name, count, dtype, masked):
    rng = np.random.default_rng(seed)
    off = _offsets(_lengths(rng, name, count), before=3)
    n = int(off[-1]) + 5                                    # tokens of no sequence at both ends
    old = -2.0 * rng.random(n)
    lp = old + 0.3 * rng.standard_normal(n)
    ref = old + 0.3 * rng.standard_normal(n)
    mask = None
    if masked:
        mask = (rng.random(n) < 0.7).astype(np.uint8) * rng.integers(1, 255, n).astype(np.uint8)
        if count > 2:
            mask[off[1]:off[2]] = 0                         # a sequence in which nothing counts
    return rng, off, n, lp, old, ref, mask


def _poison(t, mask):
    """NaN and infinities where the mask (and no sequence) keeps them out."""
    import torch
    if mask is not None:
        dead = torch.from_numpy(np.nonzero(mask == 0)[0]).cuda()
        t[dead] = float("nan")
        t[dead[::3]] = float("-inf")
        t[dead[1::3]] = float("inf")


def _seq_bound(size, n):
    return (n / 64 + 64) * U * size


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("layout,count", LAYOUTS)
@pytest.mark.parametrize("kind,average", [("sigmoid", False), ("hinge", True), ("squared", False), ("sigmoid", True)])
def test_preference_loss(gpu_lib, layout, count, masked, dtype, kind, average):
    import torch
    print("[preference]", layout, count, masked, dtype, kind, average, flush=True)
    rng, off, n, lp, _, ref, mask = _inputs(7, layout, count, dtype, masked)
    lp, lpv = _put(lp, dtype)
    ref, refv = _put(ref, dtype) if kind != "squared" else (None, None)
    maskv = None if mask is None else mask.copy()
    if mask is not None:
        # everything outside the sequences is dead as well
        dead = mask.copy()
        dead[:off[0]] = 0
        dead[off[-1]:] = 0
        _poison(lp, dead)
        lpv = np.where(dead == 0, 0.0, lpv)
        mask = torch.from_numpy(mask).cuda()
    kw = dict(beta=0.3, kind=kind, label_smoothing=0.1 if kind == "sigmoid" else 0.0, margin=0.05, average=average,
              grad_scale=2.0)
    o = to.preference_loss(lpv, off, ref_logp=refv, mask=maskv, **kw)
    loss = torch.full((1,), float("nan"), device="cuda")
    grad = torch.full_like(lp, float("nan"))
    rewards = torch.full((count,), float("nan"), device="cuda")
    offsets = torch.from_numpy(off).cuda()
    gpu_lib.muon_preference_loss(lp, offsets, loss, grad, ref_logp=ref, mask=mask, rewards=rewards, **kw)
    longest = int(np.diff(off).max())
    rb = _seq_bound(o["size"], longest) + 8 * U * np.abs(o["rewards"] / kw["beta"])
    assert np.all(np.abs(_np(rewards) - o["rewards"]) <= kw["beta"] * rb + 8 * U * np.abs(o["rewards"])), "rewards"
    # the loss and its slope move with u by at most their own derivative in u
    du = rb[0::2] + rb[1::2] + 4 * U * np.abs(o["u"])
    if kind == "squared":
        slope, second = np.abs(2 * (o["u"] - 0.5 / kw["beta"])), 2.0
    else:
        slope, second = kw["beta"], kw["beta"] ** 2 / 4
    lb = (slope * du + second * du ** 2 + 32 * U * (np.abs(o["losses"]) + 1)).mean()
    lb += (count / 64 + 64) * U * np.abs(o["losses"]).mean()
    assert abs(float(loss) - o["loss"]) <= lb, ("loss", float(loss), o["loss"], lb)
    # a gradient jumps where a hinge is met: the draws keep away from it
    if kind == "hinge":
        assert np.abs(o["h"] - 1).min() > 1e-4
    gb = np.zeros(n)
    pairs = count // 2
    for s in range(count):
        w = 1.0 / max(1, int((maskv[off[s]:off[s + 1]] != 0).sum()) if maskv is not None else off[s + 1] - off[s]) if average else 1.0
        gb[off[s]:off[s + 1]] = (second * du[s // 2] + 32 * U * kw["beta"]) * w / pairs * kw["grad_scale"]
    err = np.abs(_np(grad) - o["grad"])
    assert np.all(err <= gb + (ROUND[dtype] + 32 * U) * np.abs(o["grad"])), ("grad", float(err.max()))
    outside = np.ones(n, bool)
    outside[off[0]:off[-1]] = False
    if maskv is not None:
        outside |= maskv == 0
    assert not _np(grad)[outside].any()
    # without the gradient and the rewards, the loss is the same; and again, the same bits
    loss2, grad2 = torch.empty_like(loss), torch.empty_like(grad)
    gpu_lib.muon_preference_loss(lp, offsets, loss2, None, ref_logp=ref, mask=mask, **kw)
    assert torch.equal(loss, loss2)
    gpu_lib.muon_preference_loss(lp, offsets, loss2, grad2, ref_logp=ref, mask=mask, rewards=rewards, **kw)
    assert torch.equal(loss, loss2) and torch.equal(grad, grad2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("layout,count", LAYOUTS)
@pytest.mark.parametrize("kl,reduction,per_sequence,dual", [("k3", "token", True, 0.0), ("k2", "sequence", False, 1.25),
                                                            ("k1", "token", False, 1.25), ("none", "sequence", True, 0.0)])
def test_policy_loss(gpu_lib, layout, count, masked, dtype, kl, reduction, per_sequence, dual):
    import torch
    print("[policy]", layout, count, masked, dtype, kl, reduction, per_sequence, dual, flush=True)
    rng, off, n, lp, old, ref, mask = _inputs(9, layout, count, dtype, masked)
    adv = rng.standard_normal(count if per_sequence else n).astype(np.float32)
    # log ratios away from the bounds, where the gradient jumps: steps of 1/64 hit none of them
    old = np.round(old * 64) / 64
    lp = old + np.round((lp - old) * 64) / 64
    lp, lpv = _put(lp, dtype)
    old, oldv = _put(old, dtype)
    ref, refv = _put(ref, dtype) if kl != "none" else (None, None)
    maskv = None if mask is None else mask.copy()
    if mask is not None:
        dead = mask.copy()
        dead[:off[0]] = 0
        dead[off[-1]:] = 0
        for t in (lp, old):
            _poison(t, dead)
        lpv, oldv = np.where(dead == 0, 0.0, lpv), np.where(dead == 0, 0.0, oldv)
        mask = torch.from_numpy(mask).cuda()
    kw = dict(clip_low=0.2, clip_high=0.28, dual_clip=dual, kl_coef=0.1 if kl != "none" else 0.0, kl=kl,
              reduction=reduction, per_sequence=per_sequence, grad_scale=0.5)
    o = to.policy_loss(lpv, oldv, adv, off, ref_logp=refv, mask=maskv, **{k: np.float32(v) if isinstance(v, float) else v
                                                                         for k, v in kw.items()})
    for bound in (1 - 0.2, 1 + 0.28, dual or 9.0):
        assert np.abs(o["rho"] - bound).min(initial=1.0) > 1e-4
    loss = torch.full((1,), float("nan"), device="cuda")
    stats = torch.full((4,), float("nan"), device="cuda")
    grad = torch.full_like(lp, float("nan"))
    args = (lp, old, torch.from_numpy(adv).cuda(), torch.from_numpy(off).cuda())
    gpu_lib.muon_policy_loss(*args, loss, grad, ref_logp=ref, mask=mask, stats=stats, **kw)
    K = n / 64 + 128
    assert abs(float(loss) - o["loss"]) <= K * U * o["size"] + 1e-38, ("loss", float(loss), o["loss"])
    st = _np(stats)
    assert abs(st[0] - o["stats"][0]) <= K * U * o["ksize"] and st[3] == o["stats"][3]
    assert abs(st[1] - o["stats"][1]) <= 4 * U and abs(st[2] - o["stats"][2]) <= K * U * o["stats"][2]
    err = np.abs(_np(grad) - o["grad"])
    # the KL slope 1 - exp(q) is computed through expm1, a k2 slope from a difference rounded once
    assert np.all(err <= 48 * U * o["grad_size"] + ROUND[dtype] * np.abs(o["grad"])), ("grad", float(err.max()))
    assert not _np(grad)[~o["live"]].any()
    loss2, grad2 = torch.empty_like(loss), torch.empty_like(grad)
    gpu_lib.muon_policy_loss(*args, loss2, None, ref_logp=ref, mask=mask, **kw)
    assert torch.equal(loss, loss2)
    gpu_lib.muon_policy_loss(*args, loss2, grad2, ref_logp=ref, mask=mask, stats=stats, **kw)
    assert torch.equal(loss, loss2) and torch.equal(grad, grad2)


def test_losses_without_tokens_or_sequences(gpu_lib):
    import torch
    e = torch.empty(0, device="cuda")
    for off in ([0], [0, 0, 0], [5, 9, 2]):                # none, empty ones, ones beyond the tokens
        offsets = torch.tensor(off, dtype=torch.int64, device="cuda")
        q = len(off) - 1
        loss, rewards, stats = torch.full((1,), 7.0, device="cuda"), torch.full((q,), 7.0, device="cuda"), torch.full((4,), 7.0, device="cuda")
        gpu_lib.muon_preference_loss(e, offsets, loss, e.clone(), rewards=rewards)
        assert abs(float(loss) - (np.log(2.0) if q else 0.0)) < 1e-6 and not rewards.any()
        gpu_lib.muon_policy_loss(e, e, e, offsets, loss, e.clone(), stats=stats)
        assert float(loss) == 0.0 and not stats.any()
    # tokens, but no sequence: everything counts for nothing
    lp = torch.full((300,), float("nan"), device="cuda")
    grad = torch.full((300,), 7.0, device="cuda")
    offsets = torch.tensor([0], dtype=torch.int64, device="cuda")
    gpu_lib.muon_preference_loss(lp, offsets, loss, grad)
    assert float(loss) == 0.0 and not grad.any()
    grad.fill_(7.0)
    gpu_lib.muon_policy_loss(lp, lp, lp, offsets, loss, grad)
    assert float(loss) == 0.0 and not grad.any()


def test_losses_in_a_graph_and_on_another_stream(gpu_lib):
    import torch
    rng, off, n, lp, old, ref, mask = _inputs(3, "ragged", 64, "f32", True)
    lp, old, ref = (torch.from_numpy(v.astype(np.float32)).cuda() for v in (lp, old, ref))
    adv = torch.from_numpy(rng.standard_normal(64).astype(np.float32)).cuda()
    offsets, mask = torch.from_numpy(off).cuda(), torch.from_numpy(mask).cuda()
    def buffers():
        return [torch.empty(1, device="cuda"), torch.empty_like(lp), torch.empty(1, device="cuda"), torch.empty_like(lp)]
    ws = [torch.empty(gpu_lib.muon_preference_loss_workspace_bytes(lp, offsets), dtype=torch.uint8, device="cuda"),
          torch.empty(gpu_lib.muon_policy_loss_workspace_bytes(lp, offsets), dtype=torch.uint8, device="cuda")]
    def call(b, stream=None):
        gpu_lib.muon_preference_loss(lp, offsets, b[0], b[1], ref_logp=ref, mask=mask, workspace=ws[0], stream=stream)
        gpu_lib.muon_policy_loss(lp, old, adv, offsets, b[2], b[3], ref_logp=ref, mask=mask, kl="k3", kl_coef=0.1,
                                 per_sequence=True, workspace=ws[1], stream=stream)
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
        for t in got + ws:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("count", [16308, 3000])
def test_policy_loss_near_zero(gpu_lib, count):
    # two sequences whose advantages sum to nearly nothing: the loss is far smaller than its terms, whose rounding must not
    # show.  A term is 1 + expm1(d) times A in fp64: d is exact (both log-probabilities are multiples of 2^-20 below 8), expm1 is
    # within 2 ulp, so the mean is off by at most 2^-22 of the mean of |expm1(d) A|, and the loss itself is rounded once.
    import torch
    rng = np.random.default_rng(5)
    n = 2 * count
    old = -np.round(rng.random(n) * 2.0 ** 22) / 2.0 ** 20
    d = np.round(rng.standard_normal(n) * 0.01 * 2.0 ** 20) / 2.0 ** 20
    adv = np.array([1.0, -1.0], dtype=np.float32)
    offsets = torch.tensor([0, count, n], dtype=torch.int64, device="cuda")
    put = lambda x: torch.from_numpy(x.astype(np.float32)).cuda()
    loss = torch.empty(1, device="cuda")
    grad = torch.empty(n, device="cuda")
    gpu_lib.muon_policy_loss(put(old + d), put(old), put(adv), offsets, loss, grad_logp=grad, reduction="sequence", per_sequence=True,
                             clip_low=0.2, clip_high=0.28)
    a = np.repeat(adv.astype(np.float64), count)
    ref = -(np.exp(d) * a).sum() / n
    assert abs(float(loss) - ref) <= 2.0 ** -22 * np.abs(np.expm1(d) * a).mean() + 2.0 ** -23 * abs(ref), (float(loss), ref)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("count", [4000, 61003])
def test_preference_loss_of_nearly_equal_sequences(gpu_lib, kind, count):
    # No reference, two sequences of `count` tokens whose sums (some -1.3 count) differ by 0.25005: log-probabilities are multiples of
    # 2^-16 below 8, so fp64 sums are exact, u is, and beta u - margin, the loss and its slope are rounded a few times at
    # their own size (h up to 1: 32 u of loss + 1).
    import torch
    rng = np.random.default_rng(12)
    a = -np.round(rng.random(count) * 2.6 * 65536) / 65536
    b = rng.permutation(a)
    b[0] -= 16387 / 65536
    off = torch.tensor([0, count, 2 * count], dtype=torch.int64, device="cuda")
    logp = torch.from_numpy(np.concatenate([a, b]).astype(np.float32)).cuda()
    kw = dict(beta=2.0, kind=kind, label_smoothing=0.1 if kind == "sigmoid" else 0.0, margin=0.05)
    o = to.preference_loss(_np(logp), [0, count, 2 * count], **{k: float(np.float32(v)) if isinstance(v, float) else v for k, v in kw.items()})
    assert abs(o["u"][0] - 16387 / 65536) < 1e-9
    loss, grad = torch.empty(1, device="cuda"), torch.empty_like(logp)
    gpu_lib.muon_preference_loss(logp, off, loss, grad, **kw)
    assert abs(float(loss) - o["loss"]) <= 32 * U * (o["loss"] + 1), (float(loss), o["loss"])
    assert np.all(np.abs(_np(grad) - o["grad"]) <= 32 * U * (np.abs(o["grad"]) + 1))


def test_policy_loss_sequence_mean_takes_time_by_its_tokens(gpu_lib):
    # one masked sequence of 2^25 tokens among short ones: a mean within each sequence may cost more than one over all tokens (a
    # count of its own), not a multiple that grows with the sequence; and both means against sums in fp64
    import torch
    n = 1 << 25
    off = torch.tensor([0, 700, n - 5000, n - 4096, n], dtype=torch.int64, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    old = -torch.rand(n, generator=g, device="cuda")
    lp = old + 0.05 * torch.randn(n, generator=g, device="cuda")
    mask = (torch.rand(n, generator=g, device="cuda") < 0.8).to(torch.uint8)
    adv = torch.tensor([1.0, -0.5, 0.25, 2.0], device="cuda")
    loss, grad = torch.empty(1, device="cuda"), torch.empty_like(lp)
    ws = torch.empty(gpu_lib.muon_policy_loss_workspace_bytes(lp, off), dtype=torch.uint8, device="cuda")
    ms = {}
    a = torch.repeat_interleave(adv, off.diff()).double()
    rho = torch.exp(lp.double() - old.double())
    term = -torch.minimum(rho * a, rho.clamp(1 - 0.2, 1 + 0.2) * a) * mask
    edges = [int(v) for v in off]
    counts = torch.stack([mask[i:j].sum() for i, j in zip(edges, edges[1:])]).double()
    want = {"token": term.sum() / counts.sum(),
            "sequence": sum(term[i:j].sum() / k for i, j, k in zip(edges, edges[1:], counts)) / 4}
    for reduction in ("token", "sequence"):
        call = lambda: gpu_lib.muon_policy_loss(lp, old, adv, off, loss, grad, mask=mask, reduction=reduction, per_sequence=True, workspace=ws)
        call()
        assert abs(float(loss) - float(want[reduction])) <= 1e-6
        first, last = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        best = []
        for _ in range(5):
            first.record()
            call()
            last.record()
            torch.cuda.synchronize()
            best.append(first.elapsed_time(last))
        ms[reduction] = min(best)
        w = 1 / counts.sum() if reduction == "token" else torch.repeat_interleave(1 / (4 * counts), off.diff())
        ref = torch.where((a > 0) & (rho > 1.2) | (a < 0) & (rho < 0.8), 0.0, -rho * a) * mask * w
        off_by = (grad.double() - ref).abs() > 1e-5 * ref.abs()
        assert int(off_by.sum()) <= 64        # ratios within rounding of a clipping bound
    assert ms["sequence"] <= 3 * ms["token"] + 0.1, ms


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
def test_preference_loss_of_impossible_answers(gpu_lib, smoothing):
    # an answer with a token of probability 0: rejected, nothing is left to learn (loss and slope 0 but for the smoothing's share, which
    # is infinite); chosen, the loss is infinite and the slope its limit
    import torch
    inf = float("inf")
    off = torch.tensor([0, 3, 5, 8, 10], dtype=torch.int64, device="cuda")
    for pair, h in ((0, inf), (1, -inf)):
        logp = torch.full((10,), -1.0, device="cuda")
        logp[4 if pair == 0 else 6] = -inf
        loss, grad, rewards = torch.empty(1, device="cuda"), torch.empty_like(logp), torch.empty(4, device="cuda")
        gpu_lib.muon_preference_loss(logp, off, loss, grad, beta=0.5, label_smoothing=smoothing, rewards=rewards)
        share = smoothing if h > 0 else 1 - smoothing       # of the term that is infinite
        other = to.preference_loss(np.full(10, -1.0), [0, 3, 5, 8, 10], beta=0.5, label_smoothing=smoothing)["losses"][1 - pair]
        want = inf if share > 0 else other / 2
        assert float(loss) == want or abs(float(loss) - want) <= 32 * U, (float(loss), want)
        slope = 0.5 * (smoothing if h > 0 else smoothing - 1)
        a = 0 if pair == 0 else 5
        assert np.all(np.abs(_np(grad)[a:a + 3] - slope / 2) <= 8 * U) and np.all(np.abs(_np(grad)[a + 3:a + 5] + slope / 2) <= 8 * U)
        assert torch.isfinite(grad).all() and float(rewards[1 if pair == 0 else 2]) == -inf
