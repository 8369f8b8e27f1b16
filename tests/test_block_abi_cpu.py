"""Argument checks of the operators inside a block: every refusal comes before any GPU work, so it shows on a CPU host."""
import ctypes

import pytest
import torch

import matrix_aware_optimizer_amd as mao

AT = [k << 44 for k in range(1, 24)]   # stand-in addresses; validation never dereferences them
WS, WS_BYTES = 1 << 60, 1 << 50
NAN, INF = float("nan"), float("inf")


def _set(a, kw):
    for k, v in kw.items():
        assert hasattr(a, k), k
        setattr(a, k, v)
    return a


def _attention(**kw):
    a = mao.MuonAttentionArgs(*AT[:11], 100, 120, 2, *[256, 64, 128, 64, 128, 64, 256, 64, 256, 64], 0, 0.125, 4, 2, 64, 8, 16, 1,
                              mao.MUON_BF16)
    return _set(a, kw)


def _backward(**kw):
    a = mao.MuonAttentionBackwardArgs(*AT[:16], 100, 120, 2, *[256, 64, 128, 64, 128, 64, 256, 64, 256, 64], *[256, 64, 256, 64, 128, 64, 128, 64],
                                      0, 0.125, 4, 2, 64, 8, 16, 1, mao.MUON_BF16)
    return _set(a, kw)


def _sort(**kw):
    return _set(mao.MuonExpertSortArgs(*AT[:5], 30, 64, 64, 64, 2, 8, mao.MUON_BF16), kw)


def _sort_backward(**kw):
    return _set(mao.MuonExpertSortBackwardArgs(*AT[:3], 30, 64, 64, 64, 2, mao.MUON_BF16), kw)


def _combine(**kw):
    return _set(mao.MuonExpertCombineArgs(*AT[:4], 30, 64, 64, 64, 2, mao.MUON_BF16), kw)


def _combine_backward(**kw):
    return _set(mao.MuonExpertCombineBackwardArgs(*AT[:7], 30, 64, 64, 64, 64, 2, 8, mao.MUON_BF16), kw)


SIZED = {_attention: "attention", _backward: "attention_backward", _sort: "expert_sort"}
PLAIN = {_sort_backward: "expert_sort_backward", _combine: "expert_combine", _combine_backward: "expert_combine_backward"}


def _status(make, a, ws=WS, ws_bytes=WS_BYTES):
    lib = mao.load()
    p = ctypes.byref(a) if a is not None else None
    if make in PLAIN:
        return getattr(lib, "muon_" + PLAIN[make])(p, None)
    return getattr(lib, "muon_" + SIZED[make])(p, ctypes.c_void_p(ws), ws_bytes, None)


INVALID = [
    (m, c) for m in (_attention, _backward) for c in (
        dict(dtype=3), dict(scale=NAN), dict(scale=INF), dict(queries=-1), dict(keys=-1), dict(sequences=0), dict(width=0), dict(heads=0),
        dict(kv_heads=0), dict(kv_heads=3), dict(window=-1), dict(offsets=None), dict(offsets=None, sequences=1), dict(q=None), dict(k=None),
        dict(v=None), dict(out=None), dict(lse=None), dict(q=AT[0] + 1), dict(lse=AT[9] + 2), dict(offsets=AT[3] + 4), dict(bias=None),
        dict(bucket_map=None), dict(buckets=0), dict(reach=-1), dict(bucket_map=AT[7] + 2), dict(ld_q=-1), dict(hs_k=(1 << 40) + 1))
] + [
    (_attention, dict(out=AT[0])), (_attention, dict(out=AT[1] + 64)), (_attention, dict(lse=AT[8] + 256)), (_attention, dict(hs_out=63)),
    (_attention, dict(ld_out=255)), (_attention, dict(ld_out=0)), (_attention, dict(out_low=AT[8])), (_attention, dict(out_low=AT[10] + 1)),
    (_attention, dict(hs_out_low=0)),
    (_backward, dict(grad_out=None)), (_backward, dict(grad_q=None)), (_backward, dict(grad_k=None)), (_backward, dict(grad_v=None)),
    (_backward, dict(grad_bias=None)), (_backward, dict(bias=None, bucket_map=None)), (_backward, dict(grad_q=AT[0])), (_backward, dict(grad_k=AT[14])),
    (_backward, dict(hs_grad_k=0)), (_backward, dict(ld_grad_v=127)), (_backward, dict(grad_q=AT[11])), (_backward, dict(grad_bias=AT[6])),
    (_sort, dict(dtype=5)), (_sort, dict(tokens=-1)), (_sort, dict(cols=0)), (_sort, dict(chosen=0)), (_sort, dict(num_experts=0)), (_sort, dict(x=None)),
    (_sort, dict(experts=None)), (_sort, dict(sorted=None)), (_sort, dict(slots=None)), (_sort, dict(offsets=None)), (_sort, dict(ld_x=63)),
    (_sort, dict(ld_sorted=63)), (_sort, dict(sorted=AT[0])), (_sort, dict(experts=AT[1] + 4)), (_sort, dict(slots=AT[1])), (_sort, dict(offsets=AT[3])),
    (_sort_backward, dict(grad_sorted=None)), (_sort_backward, dict(slots=None)), (_sort_backward, dict(grad_x=None)), (_sort_backward, dict(grad_x=AT[0])),
    (_sort_backward, dict(ld_grad_x=1)), (_sort_backward, dict(dtype=-1)), (_sort_backward, dict(chosen=0)),
    (_combine, dict(y=None)), (_combine, dict(slots=None)), (_combine, dict(weights=None)), (_combine, dict(out=None)), (_combine, dict(out=AT[0])),
    (_combine, dict(weights=AT[2] + 2)), (_combine, dict(ld_y=3)), (_combine, dict(cols=0)),
    (_combine_backward, dict(grad_out=None)), (_combine_backward, dict(y=None)), (_combine_backward, dict(offsets=None)), (_combine_backward, dict(grad_y=None)),
    (_combine_backward, dict(grad_weights=None)), (_combine_backward, dict(grad_y=AT[1])), (_combine_backward, dict(grad_weights=AT[3])),
    (_combine_backward, dict(num_experts=0)), (_combine_backward, dict(ld_grad_y=63)),
]


@pytest.mark.parametrize("make,change", INVALID, ids=lambda v: v.__name__ if callable(v) else ",".join(v))
def test_invalid_arguments_are_refused(make, change):
    assert _status(make, make(**change)) == mao.MUON_ERR_INVALID_ARG, mao.muon_last_error_message()
    assert mao.muon_last_error_message() != ""
    if make in SIZED:
        assert getattr(mao.load(), f"muon_{SIZED[make]}_workspace_bytes")(ctypes.byref(make(**change))) == 0


@pytest.mark.parametrize("make,change", [
    (_attention, dict(width=129, hs_q=129)), (_attention, dict(queries=(1 << 30) + 1)), (_backward, dict(keys=(1 << 30) + 1)),
    (_attention, dict(heads=8192)), (_attention, dict(reach=4097)), (_backward, dict(buckets=8194)), (_backward, dict(sequences=(1 << 30) + 1)),
    (_sort, dict(num_experts=2049)), (_sort, dict(chosen=65)), (_sort, dict(tokens=1 << 30)), (_sort, dict(cols=(1 << 20) + 1)),
    (_combine, dict(chosen=65)), (_combine_backward, dict(num_experts=2049)), (_sort_backward, dict(tokens=(1 << 29) + 1))])
def test_sizes_beyond_the_limits_are_unsupported(make, change):
    assert _status(make, make(**change)) == mao.MUON_ERR_UNSUPPORTED


@pytest.mark.parametrize("make", [_backward, _sort])
def test_workspace_is_checked(make):
    a = make() if make is _backward else make(tokens=3000)
    need = getattr(mao.load(), f"muon_{SIZED[make]}_workspace_bytes")(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    assert _status(make, a, ws=None) == mao.MUON_ERR_WORKSPACE
    assert _status(make, a, ws=WS + 8) == mao.MUON_ERR_WORKSPACE
    assert _status(make, a, ws_bytes=0) == mao.MUON_ERR_WORKSPACE
    assert _status(make, a, ws=AT[0] & ~255) == mao.MUON_ERR_INVALID_ARG       # over the first input


def test_null_args():
    lib = mao.load()
    for name in SIZED.values():
        assert getattr(lib, "muon_" + name)(None, ctypes.c_void_p(WS), WS_BYTES, None) == mao.MUON_ERR_INVALID_ARG
        assert getattr(lib, f"muon_{name}_workspace_bytes")(None) == 0
    for name in PLAIN.values():
        assert getattr(lib, "muon_" + name)(None, None) == mao.MUON_ERR_INVALID_ARG


def test_parts_of_one_buffer_do_not_overlap():
    ok = lambda a: _status(_backward, a) != mao.MUON_ERR_INVALID_ARG
    base, es, n = AT[12], 2, 4 * 64
    g = lambda lds, hs, k, v: _backward(kv_heads=4, hs_q=64, ld_k=256, ld_v=256, grad_q=base, grad_k=base + k * es, grad_v=base + v * es,
                                        **{f"ld_grad_{t}": lds for t in "qkv"}, **{f"hs_grad_{t}": hs for t in "qkv"})
    assert ok(g(3 * n, 64, n, 2 * n))                   # side by side: rows of q, k and v
    assert not ok(g(3 * n, 64, n - 1, 2 * n))
    assert ok(g(3 * n, 192, 64, 128))                   # by turns within a head
    assert not ok(g(3 * n, 192, 63, 128))
    assert not ok(g(3 * n, 192, 64, 127))
    forward = lambda **kw: _status(_attention, _attention(**kw)) != mao.MUON_ERR_INVALID_ARG
    assert forward(hs_q=0, ld_q=0, hs_k=0, ld_k=64, ld_v=0)              # broadcast inputs
    assert forward(ld_out=64, hs_out=6400)                               # heads first
    assert _status(_attention, _attention(ld_out=64, hs_out=6399)) == mao.MUON_ERR_INVALID_ARG


def test_structs_are_packed_whole():
    for cls in (mao.MuonAttentionArgs, mao.MuonAttentionBackwardArgs, mao.MuonExpertSortArgs, mao.MuonExpertSortBackwardArgs,
                mao.MuonExpertCombineArgs, mao.MuonExpertCombineBackwardArgs):
        pack = mao._packer(cls)
        zero = {ctypes.c_float: 0.0}
        assert len(pack(*[zero.get(t, 0) for _, t in cls._fields_])) == ctypes.sizeof(cls)


def test_binding_refuses_wrong_tensors():
    q, k = torch.zeros(5, 4, 8), torch.zeros(7, 2, 8)
    o, lse, off, koff = q.clone(), torch.zeros(5, 4), torch.tensor([0, 5]), torch.tensor([0, 7])
    call = lambda *a, **kw: mao.muon_attention(*a, **kw)
    form = dict(offsets=off, key_offsets=koff)
    for args, kw, match in (
            ((q, k, k, o, lse), form, "current GPU"), ((q[0], k, k, o, lse), form, "heads"), ((q, k, k[:6], o, lse), form, "k and v"),
            ((q, k[:, :, :7], k[:, :, :7], o, lse), form, "heads"), ((q, k, k, o[:4], lse), form, "out"), ((q, k, k, o, lse.double()), form, "lse"),
            ((q, k.bfloat16(), k, o, lse), form, "k must"), ((q, k, k, o, lse), dict(offsets=off), "key_offsets is needed"),
            ((q, k, k, o, lse), dict(key_offsets=koff), "key_offsets"), ((q, k, k, o, lse), dict(offsets=off.int()), "offsets"),
            ((q, k, k, o, lse), dict(form, key_mask=torch.ones(7)), "key_mask"), ((q, k, k, o, lse), dict(form, bias=torch.zeros(3, 4)), "go together"),
            ((q, k, k, o, lse), dict(form, bias=torch.zeros(3, 3), bucket_map=torch.zeros(5, dtype=torch.int32)), "bias"),
            ((q, k, k, o, lse), dict(form, bias=torch.zeros(3, 4), bucket_map=torch.zeros(4, dtype=torch.int32)), "bucket_map"),
            ((q, k, k, o, lse), dict(form, bias=torch.zeros(3, 4), bucket_map=torch.zeros(5)), "bucket_map"),
            ((q, k, k, o, lse), dict(form, out_low=o[:3]), "out_low"), ((q.half(), k.half(), k.half(), o.half(), lse), form, "unsupported dtype"),
            ((q.transpose(1, 2).contiguous().transpose(1, 2), k, k, o, lse), form, "unit stride")):
        with pytest.raises(ValueError, match=match):
            call(*args, **kw)
    with pytest.raises(ValueError, match="gradient go together"):
        mao.muon_attention_backward(q, k, k, o, lse, q, q, k, k, bias=torch.zeros(3, 4), bucket_map=torch.zeros(5, dtype=torch.int32), **form)
    with pytest.raises(ValueError, match="grad_k"):
        mao.muon_attention_backward(q, k, k, o, lse, q, q, q, k, **form)
    x, e = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)
    s, slots, eo, w = torch.zeros(8, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(5, dtype=torch.int64), torch.zeros(4, 2)
    for fn, args, match in (
            (mao.muon_expert_sort, (x, e, s, slots, eo), "current GPU"), (mao.muon_expert_sort, (x, e.int(), s, slots, eo), "experts"),
            (mao.muon_expert_sort, (x, e, s[:7], slots, eo), "sorted_x"), (mao.muon_expert_sort, (x, e, s, slots[:, :1].contiguous(), eo), "slots"),
            (mao.muon_expert_sort, (x, e, s, slots, eo[:1]), "offsets"), (mao.muon_expert_sort, (x, e, s.bfloat16(), slots, eo), "sorted_x"),
            (mao.muon_expert_sort_backward, (s[:7], slots, x), "grad_sorted"), (mao.muon_expert_combine, (s, slots, w.double(), x), "weights"),
            (mao.muon_expert_combine, (s, slots.long(), w, x), "slots"), (mao.muon_expert_combine_backward, (x, s, slots, w, eo, s, w[:3]), "grad_weights"),
            (mao.muon_expert_combine_backward, (x, s, slots, w, eo.int(), s, w), "offsets")):
        with pytest.raises(ValueError, match=match):
            fn(*args)


def test_lse_low_is_checked():
    lib = mao.load()
    for make, fn, other in ((_attention, lib.muon_attention_two_part, AT[8]), (_backward, lib.muon_attention_backward_two_part, AT[13])):
        call = lambda low, ws=WS: fn(ctypes.byref(make()), ctypes.c_void_p(low), ctypes.c_void_p(ws), WS_BYTES, None)
        assert call(AT[17] + 2) == mao.MUON_ERR_INVALID_ARG and "lse_low" in mao.muon_last_error_message()
        assert call(other) == mao.MUON_ERR_INVALID_ARG and "overlap" in mao.muon_last_error_message()
        if make is _backward:                                                   # this forward call takes no workspace
            assert call(AT[17], AT[17] & ~255) == mao.MUON_ERR_INVALID_ARG
        assert call(None) != mao.MUON_ERR_INVALID_ARG and call(AT[17]) != mao.MUON_ERR_INVALID_ARG
        assert fn(None, None, ctypes.c_void_p(WS), WS_BYTES, None) == mao.MUON_ERR_INVALID_ARG
    q, k = torch.zeros(5, 4, 8), torch.zeros(5, 2, 8)
    lse = torch.zeros(5, 4)
    for low in (lse.double(), lse[:4], torch.zeros(4, 5).t()):
        with pytest.raises(ValueError, match="lse_low"):
            mao.muon_attention(q, k, k, q.clone(), lse, lse_low=low)
        with pytest.raises(ValueError, match="lse_low"):
            mao.muon_attention_backward(q, k, k, q, lse, q, q.clone(), k.clone(), k.clone(), lse_low=low)
