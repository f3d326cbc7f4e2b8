"""Windowed attention over caches with values that are not finite: a row that
sees such a token is not finite in that column, every other row of the same tile
and every other column is as if the value were finite."""
import math

import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_kv_attention_36_b200 import binding
    binding.pa_device_errors(clear=True)
    return binding


def _check(got, want, mean_abs, weight_error):
    """Where the definition is not finite (NaN, infinite) the output is not either; the
    others are within their bound (assert_attention over them, the rest replaced on both sides)."""
    got, ok = got.double().cpu(), torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), ok), \
        f"{(torch.isfinite(got) < ok).sum()} outputs spoiled, {(torch.isfinite(got) > ok).sum()} not"
    zero = torch.zeros_like(want)
    ref.assert_attention(torch.where(ok, got, zero), torch.where(ok, want, zero), torch.where(ok, mean_abs, zero),
                         weight_error)
    return ok


def _spoil(vp, bt, n, rng, tokens):
    """NaN, inf and -inf in a column each of the named tokens of sequence 0."""
    keys = []
    for i, t in enumerate(tokens):
        h, d = int(torch.randint(0, vp.shape[1], (1,), generator=rng)), int(torch.randint(0, vp.shape[3], (1,), generator=rng))
        bad = (math.nan, math.inf, -math.inf)[i % 3]
        vp[int(bt[0, t // 16]), h, t % 16, d] = bad
        keys.append((h, t, d, bad))
    return keys


# rows a CTA's tile each, then rows of which the CTAs of a cluster share the keys
SHAPES = [(300, 130, 40, 3), (300, 300, ref.ALL, 0), (300, 200, 1, 0), (1000, 70, 333, 21), (517, 64, 64, 100),
          (4001, 9, 2400, 4), (3000, 40, 100, 700), (2500, 3, ref.ALL, 0)]


@pytest.mark.parametrize("n,rows,window,sinks", SHAPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (4, 4, 128), (8, 1, 128)])
def test_prefill_window_values_not_finite(pa, n, rows, window, sinks, Hq, Hkv, D):
    g = torch.Generator().manual_seed(n + rows + D)
    ks, vs, kp, vp, bt = ref.bf16_batch(g, [n], Hkv, D)
    first = max(0, n - rows - min(window, n))
    # in the first row's window, at the diagonal, in the last page, among the sinks
    tokens = {first + 1, first + 5, n - rows + 1, n - rows // 2, n - 2, n - 1, min(2, n - 1)}
    for h, t, d, bad in _spoil(vp, bt, n, g, sorted(t for t in tokens if 0 <= t < n)):
        vs[0][h, t, d] = bad
    q = torch.randn((rows, Hq, D), generator=g).bfloat16()
    out = torch.zeros_like(q).cuda()
    pa.pa_prefill_window(q.cuda(), torch.tensor([0, rows], dtype=torch.int32).cuda(), rows, kp.cuda(), vp.cuda(),
                         bt.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), D ** -0.5, out, window=window,
                         sinks=sinks)
    assert pa.pa_device_errors(clear=True) == 0
    want, mean_abs = ref.attend(q, ks[0].double(), vs[0].double(), D ** -0.5, window, sinks)
    ok = _check(out, want, mean_abs, 2.0 ** -8)
    assert not ok.all() and ok.any(), "the case has nothing to show"


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_window_every_row_of_values_spoiled_once(pa, D):
    # one column of every token is NaN, inf or -inf in turn: every output knows its own window
    g = torch.Generator().manual_seed(D)
    n, rows, Hq, Hkv = 400, 150, 4, 2
    ks, vs, kp, vp, bt = ref.bf16_batch(g, [n], Hkv, D)
    for h, t, d, bad in _spoil(vp, bt, n, g, range(n)):
        vs[0][h, t, d] = bad
    q = torch.randn((rows, Hq, D), generator=g).bfloat16()
    for window, sinks in ((1, 0), (10, 2), (90, 0)):
        out = torch.zeros_like(q).cuda()
        pa.pa_prefill_window(q.cuda(), torch.tensor([0, rows], dtype=torch.int32).cuda(), rows, kp.cuda(), vp.cuda(),
                             bt.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), D ** -0.5, out, window=window,
                             sinks=sinks)
        want, mean_abs = ref.attend(q, ks[0].double(), vs[0].double(), D ** -0.5, window, sinks)
        _check(out, want, mean_abs, 2.0 ** -8)


@pytest.mark.parametrize("D", [64, 128])
def test_decode_window_values_not_finite(pa, D):
    g = torch.Generator().manual_seed(D)
    n = 700
    ks, vs, kp, vp, bt = ref.bf16_batch(g, [n], 2, D)
    for h, t, d, bad in _spoil(vp, bt, n, g, [1, 5, 300, 599, 600, 601, 650, 699]):
        vs[0][h, t, d] = bad
    q = torch.randn((1, 8, D), generator=g).bfloat16()
    for window, sinks in ((100, 0), (100, 3), (1, 0), (ref.ALL, 0)):
        out = torch.zeros_like(q).cuda()
        pa.pa_decode_window(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                            D ** -0.5, out, window=window, sinks=sinks)
        want, mean_abs = ref.attend(q, ks[0].double(), vs[0].double(), D ** -0.5, window, sinks)
        _check(out, want, mean_abs, 2.0 ** -16)
