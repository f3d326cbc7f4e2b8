"""Values at the ends of what the 8-bit attention calls take: queries from the
smallest bf16 to large ones and far from zero mean, blocks of zero keys; and the
precision that the calls state, bounded element by element.  Against the definition in 64
bits, with the bounds of the arithmetic that the kernels use."""
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

# |out - definition| <= 2^-8 |out| for its rounding to bf16, plus this part of the
# weighted mean of |V|: weights as f16 (2^-11 each) against a sum of unrounded ones.
MULTI = 2.0 ** -11


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_kv_attention_36_b200 import binding
    binding.pa_device_errors(clear=True)
    return binding


def _multi(pa, q, cache, n, scale, window=ref.ALL, sinks=0):
    """The last q.shape[0] tokens of one sequence of n tokens."""
    out = torch.full_like(q, float("nan")).cuda()
    k, v, ks, vs, bt = [t.cuda() for t in cache]
    pa.pa_prefill_i8(q.cuda(), torch.tensor([0, q.shape[0]], dtype=torch.int32).cuda(), q.shape[0], k, v, ks, vs, bt,
                     torch.tensor([n], dtype=torch.int32).cuda(), scale, out, window=window, sinks=sinks)
    assert pa.pa_device_errors(clear=True) == 0
    return out


def _want(q, cache, n, scale, window=ref.ALL, sinks=0):
    k, v, ks, vs, bt = cache
    return ref.attend(q, *ref.values_i8(k, v, ks, vs, bt[0], n), scale, window, sinks)


TINY = 2.0 ** -133  # bf16's smallest


@pytest.mark.parametrize("n,rows", [(300, 40), (4000, 3)])  # a tile a CTA, a tile a cluster
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [TINY, 2.0 ** -128, 2.0 ** -126, 1e-30, 1e-6, 1e5, 1e30])
def test_prefill_i8_query_sizes(pa, size, D, n, rows):
    g = torch.Generator().manual_seed(D)
    cache = ref.i8_batch(g, [n], 2, D)
    q = torch.randn((rows, 8, D), generator=g)
    if size < 1e-37:  # a few steps of the smallest value, zeros among them
        q = q.clamp(-3, 3).round()
    q = (q.double() * size).bfloat16()
    assert (q[0] != 0).any()
    scale = min(D ** -0.5 / size, 1e38)  # logits of size 1, or none to speak of
    want, mean_abs = _want(q, cache, n, scale)
    ref.assert_attention(_multi(pa, q, cache, n, scale), want, mean_abs, MULTI)


@pytest.mark.parametrize("n,rows", [(300, 40), (4000, 3)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [TINY, 2.0 ** -127, 1e-30, 1e-15])
def test_prefill_i8_tiny_queries_and_zero_keys(pa, size, D, n, rows):
    # blocks of zero keys have a scale of 0; the row's own page and the window's first are seen in part
    g = torch.Generator().manual_seed(D + 1)
    k, v, ks, vs, bt = ref.i8_batch(g, [n], 2, D)
    for page in range(0, (n + 15) // 16, 2):
        k[int(bt[0, page])] = 0
        ks[int(bt[0, page])] = 0.0
    q = (torch.randn((rows, 8, D), generator=g).clamp(-3, 3).round().double() * size).bfloat16()
    for window in (ref.ALL, 165):
        want, mean_abs = _want(q, (k, v, ks, vs, bt), n, 0.125, window)
        ref.assert_attention(_multi(pa, q, (k, v, ks, vs, bt), n, 0.125, window), want, mean_abs, MULTI)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_i8_queries_far_from_zero_mean(pa, D):
    # every row sees two tokens with values +1 and -1, so out = tanh of half the logits' difference.
    # Queries are 256 but for 8 columns of 258, keys sum to zero over the columns: a logit is the small
    # difference of large products.  Column pairs cancel but for 2 code, so a partial sum of whole pairs
    # is below 2^11, and one within 16 columns below 2^18: D / 16 roundings of 2^-24 of that are at most
    # 0.13 of a logit's unit (q times code), of which 413 make a logit of 1.  The difference of two logits
    # is off by 2^-10.6 at most, out by half of that: inside the 2^-11 + 2^-12 of the check.
    g = torch.Generator().manual_seed(D)
    n = 90
    k, v, ks, vs, bt = ref.i8_batch(g, [n], 2, D)
    half = torch.randint(-127, 128, (k.shape[0], 2, 16, D // 2), generator=g).to(torch.int8)
    k = torch.stack([half, -half], dim=-1).flatten(-2).contiguous()
    ks.fill_(1.0)
    by_byte = torch.empty(16, dtype=torch.int8)
    by_byte[torch.tensor(ref.V_BYTES)] = torch.tensor([127 - 254 * (t % 2) for t in range(16)], dtype=torch.int8)
    v = by_byte.expand(v.shape).contiguous()
    vs.fill_(1 / 127)
    q = torch.full((n, 8, D), 256.0)
    q[..., : 16: 2] = 258.0
    q = q.bfloat16()
    want, mean_abs = _want(q, (k, v, ks, vs, bt), n, 1 / 413, 2)
    ref.assert_attention(_multi(pa, q, (k, v, ks, vs, bt), n, 1 / 413, 2), want, mean_abs, MULTI)


# ---- the precision that the calls state -------------------------------------------

def _bounds(q, cache, b, n, scale, window, sinks, weight_step, weight_relative, query_step):
    """The definition of one sequence's last q.shape[0] rows and what the kernels may be off by:
      2^-8 |out|, its rounding to bf16;
      each weight times its V scale: weight_step of the row's heaviest and weight_relative of itself;
      the queries: query_step of the row's largest value, which moves a logit by up to that times
      |scale| sum |K|, and so every weight and their sum by as much (twice);
      2^-15 of the mean |V| for 32-bit logits, exponents and sums."""
    k, v, ks, vs, bt = cache
    keys, values = ref.values_i8(k, v, ks, vs, bt[b], n)
    rows, Hq, D = q.shape
    Hkv = keys.shape[0]
    G = Hq // Hkv
    blocks = bt[b, torch.arange(n) // 16].long()
    unit = vs.double()[blocks].t()  # [Hkv][n]
    out, tol = (torch.zeros((rows, Hq, D), dtype=torch.float64) for _ in range(2))
    for i in range(rows):
        see = ref.visible(n, n - rows + i, window, sinks)
        x = q[i].double().view(Hkv, G, D)
        s = torch.einsum("gjd,gtd->gjt", x, keys[:, see]) * scale
        w = torch.exp(s - s.amax(-1, keepdim=True))
        l = w.sum(-1, keepdim=True)
        mean = torch.einsum("gjt,gtd->gjd", w, values[:, see]) / l
        mean_abs = torch.einsum("gjt,gtd->gjd", w, values[:, see].abs()) / l
        heaviest = (w * unit[:, None, see]).amax(-1, keepdim=True)
        codes = (values[:, see].abs() / unit[:, see, None]).sum(1)[:, None]  # sum of |code|
        logit = abs(scale) * query_step * x.abs().amax(-1, keepdim=True) * keys[:, see].abs().sum(-1).amax(-1)[:, None, None]
        err = 2.0 ** -8 * mean.abs() + weight_step * heaviest * codes / l + \
            (weight_relative + 2 * logit + 2.0 ** -15) * mean_abs
        out[i], tol[i] = mean.reshape(Hq, D), err.reshape(Hq, D)
    return out, tol + 1e-30


def _within(got, want, tol):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), "output not finite"
    worst = ((got - want).abs() / tol).max().item()
    assert worst <= 1.0, f"error {worst:.2f} times its bound"


@pytest.mark.parametrize("sharp", [0.3, 1.0, 3.0])
@pytest.mark.parametrize("window,sinks", [(ref.ALL, 0), (100, 5)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (8, 1, 64), (16, 4, 128), (3, 3, 128)])
def test_decode_i8_within_its_stated_precision(pa, Hq, Hkv, D, window, sinks, sharp):
    # 16-bit fixed point: weights to 2^-17 of the heaviest (of their step, so of the row at most),
    # queries to half of 1 / 32512 of the row's largest value
    g = torch.Generator().manual_seed(Hq + D)
    lens = [1, 16, 40, 64, 200, 777]
    cache = k, v, ks, vs, bt = ref.i8_batch(g, lens, Hkv, D)
    q = torch.randn((len(lens), Hq, D), generator=g).bfloat16()
    scale = sharp * D ** -0.5
    out = torch.full_like(q, float("nan")).cuda()
    pa.pa_decode_i8(q.cuda(), *[t.cuda() for t in cache], torch.tensor(lens, dtype=torch.int32).cuda(), scale, out,
                    window=window, sinks=sinks)
    for b, n in enumerate(lens):
        want, tol = _bounds(q[b:b + 1], cache, b, n, scale, window, sinks, 2.0 ** -17, 0.0, 0.5 / 32512)
        _within(out[b:b + 1], want, tol)


@pytest.mark.parametrize("D", [64, 128])
def test_decode_i8_one_query_channel_far_above_the_rest(pa, D):
    # a channel 1000 times the others where keys are small: the others keep 2^-16 of that one
    g = torch.Generator().manual_seed(D)
    lens = [300, 70]
    k, v, ks, vs, bt = ref.i8_batch(g, lens, 2, D)
    k[..., 7] = k[..., 7] // 100
    q = torch.randn((2, 8, D), generator=g)
    q[..., 7] *= 1000
    q = q.bfloat16()
    out = torch.full_like(q, float("nan")).cuda()
    pa.pa_decode_i8(q.cuda(), *[t.cuda() for t in (k, v, ks, vs, bt)], torch.tensor(lens, dtype=torch.int32).cuda(),
                    0.02, out)
    for b, n in enumerate(lens):
        want, tol = _bounds(q[b:b + 1], (k, v, ks, vs, bt), b, n, 0.02, ref.ALL, 0, 2.0 ** -17, 0.0, 0.5 / 32512)
        _within(out[b:b + 1], want, tol)
    multi = _multi(pa, q[:1], (k, v, ks, vs, bt[:1]), lens[0], 0.02)
    want, tol = _bounds(q[:1], (k, v, ks, vs, bt), 0, lens[0], 0.02, ref.ALL, 0, 2.0 ** -31, MULTI, 2.0 ** -25)
    _within(multi, want, tol)


@pytest.mark.parametrize("sharp", [0.3, 1.0, 3.0])
@pytest.mark.parametrize("window,sinks", [(ref.ALL, 0), (100, 5)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (8, 1, 64), (16, 4, 128), (3, 3, 128)])
def test_prefill_i8_within_its_stated_precision(pa, Hq, Hkv, D, window, sinks, sharp):
    # f16 weights, lifted: 2^-11 of each, 2^-31 of the heaviest; queries as f16 of less than 4
    g = torch.Generator().manual_seed(Hq + D)
    scale = sharp * D ** -0.5
    for n, rows in ((90, 90), (777, 30), (2500, 2)):
        cache = ref.i8_batch(g, [n], Hkv, D)
        q = torch.randn((rows, Hq, D), generator=g).bfloat16()
        want, tol = _bounds(q, cache, 0, n, scale, window, sinks, 2.0 ** -31, MULTI, 2.0 ** -25)
        _within(_multi(pa, q, cache, n, scale, window, sinks), want, tol)
