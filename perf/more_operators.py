"""The operators inside a block, between the matrices that ``muon_step`` updates, as measurable cases.

Attention over packed sequences ("attention"), the same with a learned relative
position bias by buckets ("bias"), and the tokens' way to the experts and back
("experts"), each with its gradients.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) when ``own`` is false, and calls the
framework's entry points when it is true; ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def _attention(name, dtype, sequences, queries, keys, heads, kv_heads, width, direction, causal=True, window=0,
               masked=0.0, op="attention", buckets=0, reach=0):
    """queries, keys: over all sequences (keys == queries: self-attention)."""
    case = dict(name=name) if name else {}
    case.update(op=op, dtype=dtype, sequences=sequences, queries=queries, keys=keys, heads=heads, kv_heads=kv_heads,
                width=width, direction=direction, causal=causal, window=window, masked=masked)
    if op == "bias":
        case.update(buckets=buckets, reach=reach)
    return case


def _experts(name, dtype, tokens, cols, experts, chosen, dropped, direction):
    case = dict(name=name) if name else {}
    case.update(op="experts", dtype=dtype, tokens=tokens, cols=cols, experts=experts, chosen=chosen, dropped=dropped,
                direction=direction)
    return case


def listed():
    return [
        # the next token of one sequence after 4096, four query heads to a key head
        _attention("attention_one_token", "bf16", 1, 1, 4096, 16, 4, 128, "fwd"),
        # a training batch of the d = 2048 transformer: 16 heads of 128, ragged sequences packed one after the other
        _attention("attention_train", "bf16", 6, 8192, 8192, 16, 16, 128, "both"),
        # one long document, shared key heads
        _attention("attention_long", "bf16", 1, 16384, 16384, 16, 4, 128, "both"),
        # single precision, odd widths and lengths, a window, padded keys
        _attention("attention_odd_f32", "f32", 3, 1003, 1003, 6, 3, 72, "both", window=200, masked=0.1),
        # a short sequence with a bias, both directions
        _attention("bias_short", "bf16", 1, 77, 77, 8, 8, 64, "both", causal=False, op="bias", buckets=32, reach=128),
        # an encoder's batch: every token sees its whole sequence, 32 buckets up to distance 128
        _attention("bias_train", "bf16", 12, 8192, 8192, 16, 16, 64, "both", causal=False, op="bias", buckets=32,
                   reach=128),
        # queries behind a longer past, single precision, padded keys, odd sizes
        _attention("bias_odd_f32", "f32", 2, 301, 901, 5, 5, 40, "both", masked=0.2, op="bias", buckets=20, reach=300),
        # one token to 6 of 64 experts, as a serving loop calls it
        _experts("experts_one_token", "bf16", 1, 2048, 64, 6, 0.0, "fwd"),
        # a training batch of the 64-expert model (d = 2048), 6 experts a token
        _experts("experts_train", "bf16", 8192, 2048, 64, 6, 0.0, "both"),
        # odd width, single precision, some choices dropped for capacity
        _experts("experts_odd_f32", "f32", 1003, 1407, 7, 2, 0.1, "both"),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["attention", "attention", "bias", "experts"])
    if op == "experts":
        cols = rng.choice([rng.randint(64, 1000), 64 * rng.randint(2, 64), rng.choice([1024, 2048, 4096])])
        chosen = rng.choice([1, 2, 4, 6, 8, rng.randint(1, 8)])
        tokens = _log_int(rng, 1, max(1, 8192 * 2048 * 6 // (cols * chosen)))
        return _experts(None, rng.choice(["bf16", "bf16", "f32"]), tokens, cols,
                        rng.choice([8, 64, rng.randint(1, 256)]), chosen, rng.choice([0.0, 0.1]),
                        rng.choice(["fwd", "both", "both"]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    width = rng.choice([64, 128, 8 * rng.randint(2, 16), rng.randint(9, 128)])
    kv_heads = rng.choice([1, 2, 4, 8, rng.randint(1, 8)])
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    longest = 16384 if dtype == "bf16" else 2048
    queries = _log_int(rng, 1, longest)
    direction = rng.choice(["fwd", "both", "both"])
    # a step's sequences have some tokens each; one token alone has no gradient but grad_v
    sequences = min(max(1, queries // 8 if direction == "both" else queries), _log_int(rng, 1, 24))
    queries = max(queries, 8) if direction == "both" else queries
    kind = rng.choice(["self", "self", "self", "past"])
    keys = queries if kind == "self" else queries + _log_int(rng, 1, 32768)
    case = _attention(None, dtype, sequences, queries, keys, heads, kv_heads, width, direction,
                      causal=rng.random() < 0.7, window=rng.choice([0, 0, _log_int(rng, 4, 4096)]),
                      masked=rng.choice([0.0, 0.0, 0.1]), op=op, buckets=rng.choice([8, 32, rng.randint(3, 64)]),
                      reach=rng.choice([128, _log_int(rng, 16, 1024)]))
    most = _pairs(_attention(None, "bf16", 1, 16384, 16384, 16, 4, 128, "both")) * 16 * 128
    while _pairs(case) * case["heads"] * max(64, width) > most:
        shrink = case["queries"] // 2
        case["keys"] = max(shrink, case["keys"] - (case["queries"] - shrink))
        case["queries"], case["sequences"] = shrink, min(case["sequences"], max(1, shrink // 8))
    return case


def _split(total, count):
    """Lengths of `count` sequences, spread over a factor of four, that add up to `total`."""
    part = [0.25 + 0.75 * ((0.381966 + 0.618034 * i) % 1.0) for i in range(count)]
    ends, run = [0], 0.0
    for p in part:
        run += p
        ends.append(round(total * run / sum(part)))
    return [b - a for a, b in zip(ends, ends[1:])]


def _lengths(case):
    """Queries and keys of every sequence."""
    nq = _split(case["queries"], case["sequences"])
    nk = nq if case["keys"] == case["queries"] else [
        q + e for q, e in zip(nq, _split(case["keys"] - case["queries"], case["sequences"]))]
    return nq, nk


def _pairs(case):
    """Query and key pairs that see each other, over all sequences (a mask aside)."""
    total = 0
    for nq, nk in zip(*_lengths(case)):
        at = torch.arange(nq, dtype=torch.int64) + (nk - nq)
        hi = at + 1 if case["causal"] else torch.full_like(at, nk)
        lo = torch.zeros_like(at)
        if case["window"]:
            lo, hi = (at - case["window"] + 1).clamp(min=0), torch.minimum(hi, at + case["window"])
        total += int((hi.clamp(max=nk) - lo).clamp(min=0).sum())
    return total


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(shape, g, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)


def _offsets(lengths):
    return torch.tensor([0] + lengths, device=DEV, dtype=torch.int64).cumsum(0)


def _bucket_map(buckets, reach, causal):
    """Bucket of every distance -reach .. reach: the near half of a side's buckets hold one distance each, the far
    half a factor more each, up to `reach`; with both sides visible, each has its half of the buckets."""
    side = buckets if causal else max(1, buckets // 2)
    near = max(1, side // 2)
    out = []
    for d in range(-reach, reach + 1):
        n = -d if causal else abs(d)
        base = 0 if causal or d <= 0 or buckets < 2 else buckets - side
        if n <= 0:
            b = 0
        elif n < near:
            b = n
        else:
            b = min(side - 1, near + int(math.log(n / near) / math.log(max(2.0, reach / near)) * (side - near)))
        out.append(base + b)
    return torch.tensor(out, device=DEV, dtype=torch.int32)


def _attention_inputs(case, seed):
    g = _generator(seed)
    dt, d = DTYPES[case["dtype"]], case["width"]
    nq, nk = _lengths(case)
    # logits of standard deviation two: rows from a few keys to all of them
    s = dict(q=_normal((case["queries"], case["heads"], d), g, 2.0, dtype=dt),
             k=_normal((case["keys"], case["kv_heads"], d), g, dtype=dt),
             v=_normal((case["keys"], case["kv_heads"], d), g, dtype=dt),
             lengths=(nq, nk), offsets=_offsets(nq), key_offsets=_offsets(nk), key_mask=None, scale=d ** -0.5,
             bias=None, bucket_map=None)
    if case["masked"]:
        s["key_mask"] = torch.rand(case["keys"], generator=g, device=DEV) >= case["masked"]
    if case["op"] == "bias":
        s["bias"] = _normal((case["buckets"], case["heads"]), g, dtype=dt)
        s["bucket_map"] = _bucket_map(case["buckets"], case["reach"], case["causal"])
    if case["direction"] == "both":
        s["grad_out"] = _normal((case["queries"], case["heads"], d), g, 1e-3, dtype=dt)
    return s


def _experts_inputs(case, seed):
    g = _generator(seed)
    dt, t, d, e, k = DTYPES[case["dtype"]], case["tokens"], case["cols"], case["experts"], case["chosen"]
    # experts differ in popularity; a token's choices are the largest of its scores
    scores = _normal((t, e), g) + _normal((e,), g, 0.5)
    order = scores.argsort(1, descending=True)
    chosen = order[:, torch.arange(k, device=DEV) % e].contiguous()
    weights = torch.softmax(scores.gather(1, chosen), 1)
    if case["dropped"]:
        chosen = torch.where(torch.rand((t, k), generator=g, device=DEV) < case["dropped"], -1, chosen)
    s = dict(x=_normal((t, d), g, dtype=dt), experts=chosen, weights=weights, y=_normal((t * k, d), g, dtype=dt))
    if case["direction"] == "both":
        s["grad_out"] = _normal((t, d), g, 1e-3, dtype=dt)
        s["grad_sorted"] = _normal((t * k, d), g, 1e-3, dtype=dt)
    return s


_INPUTS = {"attention": _attention_inputs, "bias": _attention_inputs, "experts": _experts_inputs}


def _own_buffers(case, s):
    """Outputs and workspaces that a program allocates once and passes to every call."""
    import matrix_aware_optimizer_amd as mao
    f32 = dict(dtype=torch.float32, device=DEV)
    both = case["direction"] == "both"
    if case["op"] == "experts":
        b = dict(sorted_x=torch.empty_like(s["y"]), out=torch.empty_like(s["x"]),
                 slots=torch.empty(s["experts"].shape, dtype=torch.int32, device=DEV),
                 offsets=torch.empty(case["experts"] + 1, dtype=torch.int64, device=DEV))
        if both:
            b.update(grad_y=torch.empty_like(s["y"]), grad_weights=torch.empty_like(s["weights"]),
                     grad_x=torch.empty_like(s["x"]))
        b["workspace"] = mao.allocate_workspace(
            mao.muon_expert_sort_workspace_bytes(s["x"], s["experts"], case["experts"]), DEV)
        return b
    b = dict(out=torch.empty_like(s["q"]), lse=torch.empty(s["q"].shape[:2], **f32), out_low=None)
    need = mao.muon_attention_workspace_bytes(s["q"], s["k"], sequences=case["sequences"])
    if both:
        b.update(grad_q=torch.empty_like(s["q"]), grad_k=torch.empty_like(s["k"]), grad_v=torch.empty_like(s["v"]),
                 grad_bias=None if s["bias"] is None else torch.empty_like(s["bias"]))
        if case["dtype"] == "bf16":
            b["out_low"] = torch.empty_like(s["q"])
        need = max(need, mao.muon_attention_backward_workspace_bytes(s["q"], s["k"], sequences=case["sequences"],
                                                                     bias=s["bias"], bucket_map=s["bucket_map"]))
    b["workspace"] = mao.allocate_workspace(need, DEV)
    return b


def prepare(case, seed):
    state = _INPUTS[case["op"]](case, seed)
    state["case"] = dict(case)
    if own:
        state["buffers"] = _own_buffers(case, state)
    return state


# ----------------------------------------------------------------------------
# The framework's calls
# ----------------------------------------------------------------------------

def _own_attention(c, s, b):
    import matrix_aware_optimizer_amd as mao
    form = dict(offsets=s["offsets"], key_offsets=s["key_offsets"], key_mask=s["key_mask"], bias=s["bias"],
                bucket_map=s["bucket_map"], scale=s["scale"], causal=c["causal"], window=c["window"],
                out_low=b["out_low"], workspace=b["workspace"])
    mao.muon_attention(s["q"], s["k"], s["v"], b["out"], b["lse"], **form)
    out = dict(out=b["out"], lse=b["lse"])
    if c["direction"] == "both":
        mao.muon_attention_backward(s["q"], s["k"], s["v"], b["out"], b["lse"], s["grad_out"], b["grad_q"], b["grad_k"],
                                    b["grad_v"], grad_bias=b["grad_bias"], **form)
        out.update(grad_q=b["grad_q"], grad_k=b["grad_k"], grad_v=b["grad_v"])
        if s["bias"] is not None:
            out["grad_bias"] = b["grad_bias"]
    return out


def _own_experts(c, s, b):
    import matrix_aware_optimizer_amd as mao
    mao.muon_expert_sort(s["x"], s["experts"], b["sorted_x"], b["slots"], b["offsets"], workspace=b["workspace"])
    mao.muon_expert_combine(s["y"], b["slots"], s["weights"], b["out"])
    out = dict(sorted_x=b["sorted_x"], slots=b["slots"], offsets=b["offsets"], out=b["out"])
    if c["direction"] == "both":
        mao.muon_expert_combine_backward(s["grad_out"], s["y"], b["slots"], s["weights"], b["offsets"], b["grad_y"],
                                         b["grad_weights"])
        mao.muon_expert_sort_backward(s["grad_sorted"], b["slots"], b["grad_x"])
        out.update(grad_y=b["grad_y"], grad_weights=b["grad_weights"], grad_x=b["grad_x"])
    return out


# ----------------------------------------------------------------------------
# The plain forms
# ----------------------------------------------------------------------------

def _plain_attention(c, s):
    dt, heads, group = s["q"].dtype, c["heads"], c["heads"] // c["kv_heads"]
    q, k, v = (s[n].float().transpose(0, 1) for n in ("q", "k", "v"))          # heads first
    both = c["direction"] == "both"
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device=q.device)
    if both:
        do = s["grad_out"].float().transpose(0, 1)
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dbias = None if s["bias"] is None else torch.zeros(s["bias"].shape, device=q.device)
    q0 = k0 = 0
    for nq, nk in zip(*s["lengths"]):
        qs, ks = slice(q0, q0 + nq), slice(k0, k0 + nk)
        q0, k0 = q0 + nq, k0 + nk
        at = torch.arange(nq, device=q.device)[:, None] + (nk - nq)
        dist = torch.arange(nk, device=q.device)[None, :] - at
        seen = torch.ones_like(dist, dtype=torch.bool)
        if c["causal"]:
            seen &= dist <= 0
        if c["window"]:
            seen &= dist.abs() < c["window"]
        if s["key_mask"] is not None:
            seen &= s["key_mask"][ks]
        if s["bias"] is not None:
            reach = s["bucket_map"].numel() // 2
            bucket = s["bucket_map"].long()[dist.clamp(-reach, reach) + reach]
        # heads in groups whose scores stay within a gigabyte
        step = max(group, (1 << 28) // max(1, nq * nk) // group * group)
        for h0 in range(0, heads, step):
            h = slice(h0, min(heads, h0 + step))
            hk = torch.arange(h.start, h.stop, device=q.device) // group
            qh, kh, vh = q[h, qs], k[:, ks][hk], v[:, ks][hk]
            z = torch.matmul(qh, kh.transpose(1, 2)) * s["scale"]
            if s["bias"] is not None:
                z += s["bias"].float().t()[h][:, bucket]
            z = z.masked_fill(~seen, -math.inf)
            top = z.max(2, keepdim=True).values if nk else z.new_full((z.shape[0], nq, 1), -math.inf)
            p = (z - top.masked_fill(top == -math.inf, 0.0)).exp()
            total = p.sum(2, keepdim=True)
            p = p / total.masked_fill(total == 0, 1.0)
            o = torch.matmul(p, vh)
            out[h, qs] = o
            lse[h, qs] = (top + total.log()).squeeze(2)
            if both:
                doh = do[h, qs]
                dz = p * (torch.matmul(doh, vh.transpose(1, 2)) - (doh * o).sum(2, keepdim=True))
                dq[h, qs] = torch.matmul(dz, kh) * s["scale"]
                fold = (-1, group, nk, c["width"])
                kv = slice(h.start // group, h.stop // group)
                dv[kv, ks] = torch.matmul(p.transpose(1, 2), doh).reshape(fold).sum(1)
                dk[kv, ks] = torch.matmul(dz.transpose(1, 2), qh).reshape(fold).sum(1) * s["scale"]
                if dbias is not None:
                    # rows shifted so that equal distances stand above each other; long sums in 64 bits
                    skew = torch.nn.functional.pad(dz.flip(1), (0, nq)).reshape(dz.shape[0], -1)
                    skew = skew[:, :nq * (nk + nq - 1)].reshape(-1, nq, nk + nq - 1).sum(1, dtype=torch.float64)
                    far = (torch.arange(nk + nq - 1, device=q.device) - (nk - 1)).clamp(-reach, reach) + reach
                    one = s["bucket_map"].long()[far][:, None] == torch.arange(dbias.shape[0], device=q.device)
                    dbias[:, h] += torch.matmul(skew, one.double()).t().float()
    back = lambda t: t.transpose(0, 1).contiguous().to(dt)
    res = dict(out=back(out), lse=lse.t().contiguous())
    if both:
        res.update(grad_q=back(dq), grad_k=back(dk), grad_v=back(dv))
        if dbias is not None:
            res["grad_bias"] = dbias.to(dt)
    return res


def _plain_experts(c, s):
    dt, (t, k), e = s["x"].dtype, s["experts"].shape, c["experts"]
    flat = s["experts"].reshape(-1)
    routed = (flat >= 0) & (flat < e)
    key = torch.where(routed, flat, e)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(t * k, device=order.device)
    slots = torch.where(routed, place, -1).reshape(t, k)
    offsets = torch.searchsorted(key[order], torch.arange(e + 1, device=order.device))
    count = offsets[-1]
    live = (torch.arange(t * k, device=order.device) < count)[:, None]
    sorted_x = torch.where(live, s["x"][order // k], 0)
    w = torch.where(routed.reshape(t, k), s["weights"], 0.0)
    at = slots.clamp(min=0)
    rows = s["y"].float()[at]
    out = (rows * w[:, :, None]).sum(1)
    res = dict(sorted_x=sorted_x, slots=slots.to(torch.int32), offsets=offsets, out=out.to(dt))
    if c["direction"] == "both":
        do = s["grad_out"].float()
        gy = do[order // k] * w.reshape(-1)[order][:, None]
        res["grad_y"] = torch.where(live, gy, 0.0).to(dt)
        res["grad_weights"] = torch.where(routed.reshape(t, k), (rows * do[:, None, :]).sum(2), 0.0)
        back = s["grad_sorted"].float()[at]
        res["grad_x"] = torch.where(routed.reshape(t, k, 1), back, 0.0).sum(1).to(dt)
    return res


_PLAIN = {"attention": _plain_attention, "bias": _plain_attention, "experts": _plain_experts}
_OWN = {"attention": _own_attention, "bias": _own_attention, "experts": _own_experts}


def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](case, state, state["buffers"])
    return _PLAIN[case["op"]](case, state)


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    both = case["direction"] == "both"
    if case["op"] == "experts":
        x = case["tokens"] * case["cols"]
        rows = round(x * case["chosen"] * (1 - case["dropped"]))
        small = case["tokens"] * case["chosen"] * 16 + 8 * case["experts"]
        # sort: x in, its rows out; combine: rows in, out out
        byt, fl = es * (2 * x + 2 * rows) + small, 2 * rows
        if both:
            # combine: grad_out and y in, grad_y out; sort: rows in, grad_x out
            byt, fl = byt + es * (2 * x + 3 * rows) + small, fl + 4 * rows
        return dict(bytes=byt, flops=fl)
    qo, kv = case["queries"] * case["heads"] * case["width"], case["keys"] * case["kv_heads"] * case["width"]
    pairs = _pairs(case) * case["heads"]
    stat = 4 * case["queries"] * case["heads"]
    byt, fl = es * (2 * qo + 2 * kv) + stat, pairs * (4 * case["width"] + 6)
    if both:
        # q, k, v, out and its gradient in, three gradients out; five products a pair
        byt, fl = byt + es * (4 * qo + 4 * kv) + stat, fl + pairs * (10 * case["width"] + 8)
    return dict(bytes=byt, flops=fl)


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------

def _exact_attention(c, s):
    f, dev = torch.float64, s["q"].device
    nh, group, width = c["heads"], c["heads"] // c["kv_heads"], c["width"]
    both = c["direction"] == "both"
    res = dict(out=torch.zeros(s["q"].shape, dtype=f, device=dev),
               lse=torch.zeros(s["q"].shape[:2], dtype=f, device=dev))
    if both:
        for n in ("q", "k", "v"):
            res["grad_" + n] = torch.zeros(s[n].shape, dtype=f, device=dev)
        if s["bias"] is not None:
            res["grad_bias"] = torch.zeros(s["bias"].shape, dtype=f, device=dev)
    qb, kb = s["offsets"].tolist(), s["key_offsets"].tolist()
    for i in range(len(qb) - 1):
        rows, cols = torch.arange(qb[i], qb[i + 1], device=dev), torch.arange(kb[i], kb[i + 1], device=dev)
        nq, nk = rows.numel(), cols.numel()
        position = rows - qb[i] + nk - nq
        dist = (cols - kb[i])[None] - position[:, None]
        hidden = torch.zeros((nq, nk), dtype=torch.bool, device=dev)
        if c["causal"]:
            hidden |= dist > 0
        if c["window"]:
            hidden |= (dist >= c["window"]) | (dist <= -c["window"])
        if s["key_mask"] is not None:
            hidden |= ~s["key_mask"][cols][None]
        empty = hidden.all(1)
        if s["bias"] is not None:
            reach = (s["bucket_map"].numel() - 1) // 2
            which = s["bucket_map"][(dist.clamp(min=-reach, max=reach) + reach)].long()
        for h in range(nh):
            q, k, v = s["q"][rows, h].to(f), s["k"][cols, h // group].to(f), s["v"][cols, h // group].to(f)
            logits = torch.matmul(q, k.T.contiguous()).mul_(s["scale"])
            if s["bias"] is not None:
                logits += s["bias"][:, h].to(f)[which]
            logits[hidden] = -math.inf
            norm = torch.logsumexp(logits, 1) if nk else torch.full((nq,), -math.inf, dtype=f, device=dev)
            res["lse"][rows, h] = norm
            prob = logits.sub_(torch.where(empty, torch.zeros_like(norm), norm)[:, None]).exp_()
            o = torch.matmul(prob, v)
            res["out"][rows, h] = o
            if both:
                g = s["grad_out"][rows, h].to(f)
                res["grad_v"][cols, h // group] += torch.matmul(prob.T.contiguous(), g)
                d = torch.matmul(g, v.T.contiguous())
                d -= (g * o).sum(1)[:, None]
                d *= prob
                res["grad_q"][rows, h] = torch.matmul(d, k) * s["scale"]
                res["grad_k"][cols, h // group] += torch.matmul(d.T.contiguous(), q) * s["scale"]
                if s["bias"] is not None:
                    for b in range(s["bias"].shape[0]):
                        res["grad_bias"][b, h] += d[which == b].sum()
    return res


def _exact_experts(c, s):
    f, dev = torch.float64, s["x"].device
    t, k = s["experts"].shape
    d, e = c["cols"], c["experts"]
    ids = s["experts"]
    slots = torch.full((t * k,), -1, dtype=torch.int64, device=dev)
    starts = [0]
    for expert in range(e):
        mine = torch.nonzero(ids.reshape(-1) == expert).squeeze(1)        # in the order of tokens and choices
        slots[mine] = starts[-1] + torch.arange(mine.numel(), device=dev)
        starts.append(starts[-1] + mine.numel())
    taken = torch.nonzero(slots >= 0).squeeze(1)
    token, row = taken // k, slots[taken]
    w = s["weights"].to(f).reshape(-1)[taken]
    sorted_x = torch.zeros((t * k, d), dtype=f, device=dev)
    sorted_x[row] = s["x"].to(f)[token]
    picked = s["y"].to(f)[row]
    out = torch.zeros((t, d), dtype=f, device=dev).index_add_(0, token, picked * w[:, None])
    res = dict(sorted_x=sorted_x, slots=slots.reshape(t, k).to(torch.int32),
               offsets=torch.tensor(starts, device=dev), out=out)
    if c["direction"] == "both":
        g = s["grad_out"].to(f)[token]
        gw = torch.zeros(t * k, dtype=f, device=dev)
        gw[taken] = (g * picked).sum(1)
        gy = torch.zeros((t * k, d), dtype=f, device=dev)
        gy[row] = g * w[:, None]
        res.update(grad_y=gy, grad_weights=gw.reshape(t, k))
        res["grad_x"] = torch.zeros((t, d), dtype=f, device=dev).index_add_(0, token, s["grad_sorted"].to(f)[row])
    return res


_EXACT = {"attention": _exact_attention, "bias": _exact_attention, "experts": _exact_experts}


def exact(case, seed):
    return _EXACT[case["op"]](case, _INPUTS[case["op"]](case, seed))
