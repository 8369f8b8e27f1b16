"""GPU parity of attention at sizes of a training step against the fp64 oracle, where the gradients come from separate launches; bounds as in
test_gpu_attention.

One launch makes all gradients up to 256 units of 128 rows and 1024 keys a sequence; the shapes here lie beyond the one or the other.
"""
import numpy as np
import pytest

from test_gpu_attention import _case, _check, _make, _np, _run

pytestmark = pytest.mark.gpu

RAGGED = [1 + 97 * i % 211 for i in range(40)]                                # 40 sequences of 1 to 210 tokens
SHAPES = [
    dict(nq=[1500], heads=4, kv=2, causal=True),                              # walks in many parts, shared key heads
    dict(nq=[1100, 0, 30, 1300], heads=8, kv=8, window=300, masked=0.1),      # several sequences, a window
    dict(nq=RAGGED, heads=8, kv=8, causal=True),                              # walks in one part
    dict(nq=RAGGED, nk=[n + 40 * i for i, n in enumerate(RAGGED)], heads=8, kv=4, masked=0.2),      # queries behind a longer past
    dict(nq=[70], nk=[1900], heads=6, kv=2, causal=True),
    dict(nq=[1900], nk=[1030], heads=2, kv=1, causal=True),                   # the first 870 queries see nothing
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
# (buckets, reach) and width: with whole tiles of 64 and 128, and for the first two odd ones of each
@pytest.mark.parametrize("bias,width", [(None, 48), (None, 64), (None, 101), (None, 128), ((32, 128), 48), ((32, 128), 64), ((32, 128), 101),
                                        ((32, 128), 128), ((7, 1500), 64), ((7, 1500), 128)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s['nq'])}x{s['heads']}of{s['kv']}")
def test_separate_launches(gpu_lib, shape, bias, width, dtype):
    c = _case(dtype=dtype, width=width, **shape, **({} if bias is None else dict(buckets=bias[0], reach=bias[1])))
    t, val = _make(c)
    _check(c, _run(gpu_lib, c, t), val)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [dict(nq=[1]), dict(nq=[3]), dict(nq=[300], causal=True), dict(nq=[1], nk=[5000], heads=8, kv=2), dict(nq=[2], nk=[9000], buckets=3, reach=4),
                                   dict(nq=[130], nk=[700], masked=0.5, buckets=2, reach=900)], ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()).replace(" ", ""))
def test_lse_of_scores_of_zero(gpu_lib, shape, dtype):
    # every term is the same power of two, so their sum is exact and lse is the logarithm of the keys' number: its own rounding, the logarithm's
    # (2^-24 of a power of two) and, over parts of a walk, nothing else
    c = _case(dtype=dtype, grad=False, **shape)
    t, val = _make(c)
    t["q"].zero_()
    if t["bias"] is not None:
        t["bias"].zero_()
    o = _run(gpu_lib, c, t)
    off = len(val["k"]) - len(val["q"])
    mask = np.ones(len(val["k"]), bool) if val["mask"] is None else val["mask"]
    count = np.array([mask[:i + off + 1].sum() if c["causal"] else mask.sum() for i in range(len(val["q"]))])
    want = np.log(count)[:, None]
    assert (np.abs(_np(o["lse"]) - want) <= 2.0 ** -22 + 2.0 ** -23 * want).all()
