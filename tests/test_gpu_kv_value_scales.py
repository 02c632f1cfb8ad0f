"""Value scales of very different sizes where a row must not notice: in tokens that it does not see
(other rows of its tile do), in tokens without probability, in the other group of its head."""

import pytest
import torch

import weight_only_bit_02_amd as awq

from . import kv_exact
from .gpu_util import DEV

pytestmark = pytest.mark.gpu

SMALL, LARGE = 2.0 ** -11, 30000.0  # scales of some 2^-13 and 2^12


def attend(D, group, share, n, length, window, gains, k_gain=None, seed=0):
    """gains [length][D]: the values' sizes; k_gain [length]: keys are the first query's times it."""
    gen = torch.Generator(DEV).manual_seed(seed + D + group)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(-(-length // 32), **i32)[None]
    cache = awq.alloc_kv_cache(table.shape[1], 1, D, DEV, page_size=32, group=group)
    whole = awq.KVBatch(torch.tensor([0, length], **i32), torch.tensor([length], **i32), table)
    q = torch.randn(n, share, D, generator=gen, device=DEV).half()
    k = torch.randn(length, 1, D, generator=gen, device=DEV)
    if k_gain is not None:
        k = 0.2 * k + q[0, :1].float() * k_gain.to(DEV)[:, None, None]
    # within twice their size: 30000 times a normal value would pass fp16
    v = torch.rand(length, 1, D, generator=gen, device=DEV) * 4 - 2
    awq.kv_append(cache, whole, k.half(), (v * gains.to(DEV)[:, None]).half())
    lse = torch.empty(n, share, device=DEV)
    y = awq.attention_kv4(q, cache, awq.KVBatch(torch.tensor([0, n], **i32), whole.lengths, table), window=window, lse=lse)
    want = kv_exact.attention(q.cpu().double(), kv_exact.tokens(awq, cache, whole, 0, length), D ** -0.5, True, window,
                              D // group <= 2, n * share > 64)
    kv_exact.check(y, lse, want)


FORMS = [(128, 128, 1), (128, 64, 5), (64, 64, 2), (64, 32, 4), (256, 128, 3), (128, 32, 2), (256, 64, 1)]


@pytest.mark.parametrize("D,group,share", FORMS)
@pytest.mark.parametrize("length", [9, 40, 300])
def test_large_values_behind_a_row(D, group, share, length):
    """Five drafted tokens, the last one's values large: the rows before it do not see it."""
    gains = torch.full((length, D), SMALL)
    gains[-1] = LARGE
    attend(D, group, share, 5, length, 0, gains)


@pytest.mark.parametrize("D,group,share", FORMS)
@pytest.mark.parametrize("window", [20, 100])
def test_large_values_before_a_row_s_window(D, group, share, window):
    """The first row sees a token with large values, the others' windows begin behind it."""
    n, length = 4, 333
    gains = torch.full((length, D), SMALL)
    gains[:length - n - window + 2] = LARGE
    attend(D, group, share, n, length, window, gains)


@pytest.mark.parametrize("D,group,share", FORMS)
@pytest.mark.parametrize("large", [0, -1])
def test_groups_of_different_size(D, group, share, large):
    gains = torch.full((500, D), SMALL)
    gains.view(500, -1, group)[:, large] = LARGE
    attend(D, group, share, 2, 500, 0, gains)


@pytest.mark.parametrize("D,group,share", FORMS)
@pytest.mark.parametrize("rising", [True, False])
def test_large_values_without_probability(D, group, share, rising):
    """Tokens of large values score some 60 below the others, before them or behind them: first they are all
    that a row has, or come when it needs none of them."""
    length = 600
    first = torch.arange(length) < length // 2
    gains, k_gain = torch.full((length, D), SMALL), torch.ones(length)
    gains[first if rising else ~first] = LARGE
    k_gain[first if rising else ~first] = -60 / D ** 0.5
    attend(D, group, share, 1, length, 0, gains, k_gain)
