"""Flags of appending, exactly: an Inf or NaN in the input is that alone, whichever half of a rotated pair
it is in; a rotated value that passes fp16 is an overflow alone."""

import numpy as np
import pytest

import weight_only_bit_02_amd as awq
from weight_only_bit_02_amd import _abi

from . import kv_ref
from .gpu_util import flags_tensor, host, to_dev
from .kv_util import batch_of, on_device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,R", [(64, 64), (64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_flags_exactly(D, R, interleaved):
    rng = np.random.default_rng(D + R)
    b, pages, _, _ = batch_of(awq, [3], [3], 16, rng)
    tab = np.concatenate([np.full((3, R // 2), 0.8), np.full((3, R // 2), 0.6)], 1).astype(np.float32)
    q, k, v = (rng.standard_normal((3, 1, D)).astype(np.float16) for _ in "qkv")
    dev = on_device(awq, kv_ref.Cache(pages, 1, 16, D, 64, rng))

    def run(**changed):
        x = dict(dict(q=q, k=k, v=v), **changed)
        flags = flags_tensor()
        awq.kv_append(dev, b, to_dev(x["k"]), to_dev(x["v"]), to_dev(x["q"]), awq.Rotary(to_dev(tab), interleaved), flags=flags)
        return int(host(flags)[0])

    assert run() == 0
    for bad in (np.inf, -np.inf, np.nan):
        for name, x in (("q", q), ("k", k), ("v", v)):
            for at in {0, R // 2 - 1, R // 2, R - 1, D - 1}:
                y = x.copy()
                y[1, 0, at] = bad
                got = run(**{name: y})
                # an infinite key or value makes its group's scale infinite, which is clamped too
                clamped = _abi.FLAG_SCALE_CLAMPED if name != "q" else 0
                assert got & ~clamped == _abi.FLAG_NONFINITE_INPUT, (name, bad, at, got)
    pair = (2, 3) if interleaved else (3, 3 + R // 2)
    y = q.copy()
    y[0, 0, pair[0]], y[0, 0, pair[1]] = 60000, -60000  # 0.8 x 60000 + 0.6 x 60000
    assert run(q=y) == _abi.FLAG_OVERFLOW
    # both at once, in different rows
    y[2, 0, 5] = np.nan
    assert run(q=y) == _abi.FLAG_OVERFLOW | _abi.FLAG_NONFINITE_INPUT
