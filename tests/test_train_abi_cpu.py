"""The training operators' argument checks: every refusal comes before any GPU work, so it shows on a CPU host."""
import ctypes

import pytest
import torch

import matrix_aware_optimizer_amd as mao

AT = [k << 44 for k in range(1, 24)]   # stand-in addresses; validation never dereferences them
WS, WS_BYTES = 1 << 60, 1 << 50


def _norm(**kw):
    a = mao.MuonBlockNormArgs(AT[0], AT[1], AT[2], AT[3], AT[4], AT[5], AT[6], AT[7], 4, 64, 64, 64, 64, 64, 64, 1.0,
                              1e-6, mao.MUON_BF16, mao.MUON_BF16, mao.GATE_CHANNEL)
    return _set(a, kw)


def _norm_backward(**kw):
    a = mao.MuonBlockNormBackwardArgs(*AT[:13], 4, 64, 64, 64, 64, 64, 64, 64, 64, 64, 1.0, mao.MUON_BF16, mao.MUON_BF16,
                                      mao.GATE_CHANNEL)
    return _set(a, kw)


def _logp(**kw):
    return _set(mao.MuonTokenLogpArgs(*AT[:6], 8, 64, 100, 64, 64, 1.0, mao.MUON_BF16), kw)


def _logp_backward(**kw):
    return _set(mao.MuonTokenLogpBackwardArgs(*AT[:8], 8, 64, 100, 64, 64, 64, 64, 1.0, mao.MUON_BF16), kw)


def _preference(**kw):
    return _set(mao.MuonPreferenceArgs(*AT[:7], 30, 4, 0.1, 0.0, 0.0, 1.0, 0, 0, mao.MUON_F32), kw)


def _policy(**kw):
    return _set(mao.MuonPolicyArgs(*AT[:9], 30, 4, 0.2, 0.2, 0.0, 0.1, 1.0, 3, 0, 0, mao.MUON_F32), kw)


def _set(a, kw):
    for k, v in kw.items():
        assert hasattr(a, k), k
        setattr(a, k, v)
    return a


def _status(a, ws=WS, ws_bytes=WS_BYTES):
    lib = mao.load()
    p = ctypes.byref(a) if a is not None else None
    if isinstance(a, mao.MuonBlockNormArgs):
        return lib.muon_block_norm(p, None)
    fn = {mao.MuonBlockNormBackwardArgs: lib.muon_block_norm_backward, mao.MuonTokenLogpArgs: lib.muon_token_logp,
          mao.MuonTokenLogpBackwardArgs: lib.muon_token_logp_backward, mao.MuonPreferenceArgs: lib.muon_preference_loss,
          mao.MuonPolicyArgs: lib.muon_policy_loss}[type(a)]
    return fn(p, ctypes.c_void_p(ws), ws_bytes, None)


NAN, INF = float("nan"), float("inf")
INVALID = [
    (_norm, dict(dtype=7)), (_norm, dict(weight_dtype=-1)), (_norm, dict(gate_kind=3)), (_norm, dict(rows=-1)),
    (_norm, dict(cols=0)), (_norm, dict(x=None)), (_norm, dict(residual=None)), (_norm, dict(out_residual=None)),
    (_norm, dict(gate=None)), (_norm, dict(gate_kind=0)), (_norm, dict(pre_weight=None)), (_norm, dict(out_norm=None)),
    (_norm, dict(ld_x=63)), (_norm, dict(ld_out_norm=10)), (_norm, dict(x=AT[0] + 1)), (_norm, dict(rstd=AT[7] + 2)),
    (_norm, dict(residual_scale=NAN)), (_norm, dict(eps=-1.0)), (_norm, dict(eps=INF)), (_norm, dict(out_norm=AT[5])),
    (_norm, dict(out_residual=AT[0])), (_norm, dict(out_residual=AT[1] + 2)), (_norm, dict(out_residual=AT[1], ld_residual=70)),
    (_norm_backward, dict(grad_norm=None, grad_out_residual=None)), (_norm_backward, dict(pre_weight=None)),
    (_norm_backward, dict(grad_post_weight=None)), (_norm_backward, dict(grad_gate=None)),
    (_norm_backward, dict(grad_pre_weight=None)), (_norm_backward, dict(rstd=None)), (_norm_backward, dict(grad_x=AT[0])),
    (_norm_backward, dict(grad_x=AT[9])), (_norm_backward, dict(ld_grad_x=3)), (_norm_backward, dict(residual_scale=INF)),
    (_norm_backward, dict(gate_kind=2, ld_gate=5)), (_norm_backward, dict(cols=-4)),
    (_logp, dict(dtype=2)), (_logp, dict(scale=NAN)), (_logp, dict(tokens=-1)), (_logp, dict(cols=0)), (_logp, dict(vocab=0)),
    (_logp, dict(hidden=None)), (_logp, dict(head=None)), (_logp, dict(targets=None)), (_logp, dict(logp=None)),
    (_logp, dict(lse=None)), (_logp, dict(ld_hidden=63)), (_logp, dict(ld_head=1)), (_logp, dict(saved=AT[5] + 4)),
    (_logp, dict(targets=AT[2] + 4)), (_logp, dict(lse=AT[3] + 4)), (_logp, dict(logp=AT[0] + 64)),
    (_logp_backward, dict(grad_hidden=None, grad_head=None)), (_logp_backward, dict(lse=None)),
    (_logp_backward, dict(grad_logp=None)), (_logp_backward, dict(grad_hidden=AT[0])), (_logp_backward, dict(ld_grad_head=63)),
    (_logp_backward, dict(saved=AT[5] + 8)), (_logp_backward, dict(grad_head=AT[5])), (_logp_backward, dict(scale=INF)),
    (_preference, dict(dtype=9)), (_preference, dict(tokens=-1)), (_preference, dict(sequences=3)),
    (_preference, dict(sequences=-2)), (_preference, dict(beta=NAN)), (_preference, dict(margin=INF)),
    (_preference, dict(label_smoothing=1.5)), (_preference, dict(label_smoothing=-0.1)), (_preference, dict(kind=3)),
    (_preference, dict(kind=2, beta=0.0)), (_preference, dict(logp=None)), (_preference, dict(offsets=None)),
    (_preference, dict(loss=None)), (_preference, dict(grad_logp=AT[0])), (_preference, dict(rewards=AT[4])),
    (_preference, dict(grad_scale=NAN)), (_preference, dict(offsets=AT[3] + 4)),
    (_policy, dict(kl=4)), (_policy, dict(kl=0)), (_policy, dict(ref_logp=None)), (_policy, dict(reduction=2)),
    (_policy, dict(clip_low=-0.1)), (_policy, dict(clip_high=INF)), (_policy, dict(dual_clip=0.5)), (_policy, dict(kl_coef=NAN)),
    (_policy, dict(old_logp=None)), (_policy, dict(advantages=None)), (_policy, dict(offsets=None)), (_policy, dict(loss=None)),
    (_policy, dict(stats=AT[6])), (_policy, dict(grad_logp=AT[1])), (_policy, dict(dtype=-3)),
]


@pytest.mark.parametrize("make,change", INVALID, ids=lambda v: v.__name__ if callable(v) else ",".join(v))
def test_invalid_arguments_are_refused(make, change):
    a = make(**change)
    assert _status(a) == mao.MUON_ERR_INVALID_ARG, mao.muon_last_error_message()
    assert mao.muon_last_error_message() != ""


@pytest.mark.parametrize("make", [_norm_backward, _logp, _logp_backward, _preference, _policy], ids=lambda f: f.__name__)
def test_workspace_is_checked(make):
    lib = mao.load()
    a = make()
    size = {_norm_backward: lib.muon_block_norm_backward_workspace_bytes, _logp: lib.muon_token_logp_workspace_bytes,
            _logp_backward: lib.muon_token_logp_backward_workspace_bytes,
            _preference: lib.muon_preference_loss_workspace_bytes, _policy: lib.muon_policy_loss_workspace_bytes}[make]
    need = size(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    assert _status(a, ws=None) == mao.MUON_ERR_WORKSPACE
    assert _status(a, ws=WS + 8) == mao.MUON_ERR_WORKSPACE
    assert _status(a, ws_bytes=0) == mao.MUON_ERR_WORKSPACE
    assert _status(a, ws=AT[0] & ~255) == mao.MUON_ERR_INVALID_ARG       # over the first input


@pytest.mark.parametrize("make,change", [(_norm, dict(cols=32769, ld_x=32769, ld_residual=32769, ld_out_residual=32769, ld_out_norm=32769)),
                                         (_norm, dict(rows=(1 << 30) + 1)), (_logp, dict(vocab=(1 << 24) + 1)),
                                         (_logp, dict(cols=(1 << 20) + 1)), (_logp_backward, dict(tokens=(1 << 30) + 1)),
                                         (_preference, dict(tokens=(1 << 30) + 1)), (_policy, dict(sequences=(1 << 30) + 2))])
def test_sizes_beyond_the_limits_are_unsupported(make, change):
    assert _status(make(**change)) == mao.MUON_ERR_UNSUPPORTED


def test_null_args():
    lib = mao.load()
    assert lib.muon_block_norm(None, None) == mao.MUON_ERR_INVALID_ARG
    for fn in (lib.muon_block_norm_backward, lib.muon_token_logp, lib.muon_token_logp_backward, lib.muon_preference_loss,
               lib.muon_policy_loss):
        assert fn(None, ctypes.c_void_p(WS), WS_BYTES, None) == mao.MUON_ERR_INVALID_ARG
    for fn in (lib.muon_block_norm_backward_workspace_bytes, lib.muon_token_logp_workspace_bytes,
               lib.muon_token_logp_saved_bytes, lib.muon_token_logp_backward_workspace_bytes,
               lib.muon_preference_loss_workspace_bytes, lib.muon_policy_loss_workspace_bytes):
        assert fn(None) == 0


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 8)
    v, f = torch.zeros(8), torch.zeros(4)
    with pytest.raises(ValueError, match="current GPU"):
        mao.muon_block_norm(x, x.clone(), x.clone())
    with pytest.raises(ValueError, match="residual"):
        mao.muon_block_norm(x, x[:3], x.clone())
    with pytest.raises(ValueError, match="unit column stride"):
        mao.muon_block_norm(x.t(), torch.zeros(8, 4), torch.zeros(8, 4))
    with pytest.raises(ValueError, match="overlapping rows"):
        mao.muon_block_norm(torch.zeros(1, 8).expand(4, 8), x, x.clone())
    with pytest.raises(ValueError, match="post_weight"):
        mao.muon_block_norm(x, x.clone(), x.clone(), post_weight=torch.zeros(7))
    with pytest.raises(ValueError, match="pre_weight"):
        mao.muon_block_norm(x, x.clone(), x.clone(), x.clone(), post_weight=v, pre_weight=v.bfloat16())
    with pytest.raises(ValueError, match="rstd"):
        mao.muon_block_norm(x, x.clone(), x.clone(), rstd=torch.zeros(4))
    with pytest.raises(ValueError, match="unsupported dtype"):
        mao.muon_block_norm(x.half(), x.half(), x.half())
    with pytest.raises(ValueError, match="go together"):
        mao.muon_block_norm_backward(x, x, torch.zeros(2, 4), x, x.clone(), x.clone(), post_weight=v)
    y = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="one dtype and width"):
        mao.muon_token_logp(x, torch.zeros(5, 9), y, f, f.clone())
    with pytest.raises(ValueError, match="targets"):
        mao.muon_token_logp(x, torch.zeros(5, 8), y.int(), f, f.clone())
    with pytest.raises(ValueError, match="lse"):
        mao.muon_token_logp(x, torch.zeros(5, 8), y, f, f.clone().double())
    o = torch.tensor([0, 2, 4])
    with pytest.raises(ValueError, match="offsets"):
        mao.muon_preference_loss(f, o.int(), torch.zeros(1))
    with pytest.raises(ValueError, match="mask"):
        mao.muon_preference_loss(f, o, torch.zeros(1), mask=torch.ones(4))
    with pytest.raises(ValueError, match="kind"):
        mao.muon_preference_loss(f, o, torch.zeros(1), kind="softmax")
    with pytest.raises(ValueError, match="ref_logp"):
        mao.muon_preference_loss(f, o, torch.zeros(1), ref_logp=f.double())
    with pytest.raises(ValueError, match="advantages"):
        mao.muon_policy_loss(f, f, torch.zeros(2), o, torch.zeros(1))
    with pytest.raises(ValueError, match="kl"):
        mao.muon_policy_loss(f, f, f, o, torch.zeros(1), kl="k4")
    with pytest.raises(ValueError, match="loss"):
        mao.muon_policy_loss(f, f, f, o, torch.zeros(2))



def test_profile_read_fills_what_its_first_callers_allocate():
    # muon_profile is two arrays of the nine classes that the optimizer steps have (144 bytes): a program built with it has no
    # more behind the pointer.  The other classes come through muon_profile_read_classes.
    lib = mao.load()
    room = (ctypes.c_uint8 * 512)(*([0xA5] * 512))
    assert lib.muon_profile_read(ctypes.cast(room, ctypes.POINTER(mao.MuonProfile))) == mao.MUON_OK
    assert bytes(room[:144]) == bytes(144) and set(room[144:]) == {0xA5}
    assert ctypes.sizeof(mao.MuonProfile) == 144
    n = len(mao.KERNEL_CLASSES)
    ms, launches = (ctypes.c_double * (n + 1))(*([7.0] * (n + 1))), (ctypes.c_int64 * (n + 1))(*([7] * (n + 1)))
    assert lib.muon_profile_read_classes(n, ms, launches) == mao.MUON_OK
    assert not any(ms[:n]) and not any(launches[:n]) and ms[n] == 7.0 and launches[n] == 7
    assert lib.muon_profile_read_classes(n, None, None) == mao.MUON_OK
    for bad in (-1, n + 1):
        assert lib.muon_profile_read_classes(bad, ms, launches) == mao.MUON_ERR_INVALID_ARG
    assert mao.muon_version() > 100          # how a program tells that the other classes and the operators are there


def test_column_ranges_of_one_buffer_do_not_overlap():
    # matrices of 64 bf16 columns in rows of 192: side by side they share no element, one column further in they do
    pitch = dict(ld_out_residual=192, ld_out_norm=192, ld_x=192)
    for base in (AT[5], AT[5] + 128, AT[5] + 256):          # also where the second starts before the first, in its previous row
        for other in (AT[5], AT[5] + 128, AT[5] + 256):
            status = _status(_norm(out_residual=base, out_norm=other, x=AT[0], **pitch))
            assert (status == mao.MUON_ERR_INVALID_ARG) == (base == other), mao.muon_last_error_message()
    assert _status(_norm(out_residual=AT[5], out_norm=AT[5] + 126, **pitch)) == mao.MUON_ERR_INVALID_ARG
    assert _status(_norm(out_residual=AT[5] + 384 * 2, out_norm=AT[5] + 256 + 2, **pitch)) == mao.MUON_ERR_INVALID_ARG   # into the next row
    assert _status(_norm(out_residual=AT[5], out_norm=AT[5] + 128, **{**pitch, "ld_out_norm": 191})) == mao.MUON_ERR_INVALID_ARG
    assert _status(_norm(x=AT[5] + 128, out_residual=AT[5], **pitch)) != mao.MUON_ERR_INVALID_ARG
    assert _status(_norm_backward(grad_x=AT[9], grad_residual=AT[9] + 128, ld_grad_x=128, ld_grad_residual=128)) != mao.MUON_ERR_INVALID_ARG
    assert _status(_logp_backward(grad_hidden=AT[6], hidden=AT[6] + 128, ld_hidden=128, ld_grad_hidden=128)) != mao.MUON_ERR_INVALID_ARG
