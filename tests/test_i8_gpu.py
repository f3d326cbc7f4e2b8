"""The 8-bit cache with a scale for each (block, kv head): appended codes and
scales equal the definition's bit by bit, attention over them against the
definition in 64 bits (unread blocks hold noise and scales of NaN)."""
import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

DECODE_WEIGHTS = 2.0 ** -11   # softmax weights as f16
PREFILL_WEIGHTS = 2.0 ** -8   # softmax weights as bf16


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_kv_attention_36_b200 import binding
    binding.pa_device_errors(clear=True)
    return binding


def _append_both(pa, k_rows, v_rows, slots, caches):
    gpu = [t.cuda() for t in caches]
    pa.pa_cache_append_i8(k_rows.cuda(), v_rows.cuda(), torch.tensor(slots, dtype=torch.int32).cuda(), *gpu)
    ref.append_i8(k_rows.float(), v_rows.float(), slots, caches)
    for name, a, b in zip(("k codes", "v codes", "k scales", "v scales"), gpu, caches):
        assert torch.equal(a.cpu().nan_to_num(-3), b.nan_to_num(-3)), name + " differ from the definition"


def _rows(gen, T, Hkv, D, size=1.0):
    return (torch.randn((T, Hkv, D), generator=gen) * size).bfloat16()


@pytest.mark.parametrize("Hkv,D", [(1, 64), (2, 128), (5, 64), (8, 128), (16, 64)])
def test_append_whole_blocks_any_order(pa, Hkv, D):
    g = torch.Generator().manual_seed(Hkv + D)
    caches = ref.fresh_i8(12, Hkv, D, junk=g)
    slots = torch.randperm(12 * 16, generator=g)[:150].tolist()
    slots[3], slots[77] = -1, -100  # padding
    _append_both(pa, _rows(g, 150, Hkv, D), _rows(g, 150, Hkv, D), slots, caches)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_append_token_by_token_grows_scales(pa, D):
    # the decode's way: one row a call, larger and smaller ones in turn
    g = torch.Generator().manual_seed(D)
    caches = ref.fresh_i8(3, 2, D, junk=g)
    for t in range(40):
        size = [0.1, 1.0, 3.0, 0.5, 0.0][t % 5] * (1 + t / 8)
        _append_both(pa, _rows(g, 1, 2, D, size), _rows(g, 1, 2, D, size), [t], caches)


def test_append_chunks_that_start_inside_blocks(pa):
    g = torch.Generator().manual_seed(3)
    caches = ref.fresh_i8(40, 4, 128, junk=g)
    at = [0, 200, 400]
    for step in (1, 7, 16, 30, 1, 5):
        slots = [a + i for a in at for i in range(step)]
        order = torch.randperm(len(slots), generator=g).tolist()
        _append_both(pa, _rows(g, len(slots), 4, 128, 1 + step / 4), _rows(g, len(slots), 4, 128), 
                     [slots[i] for i in order], caches)
        at = [a + step for a in at]


def test_append_same_slot_twice_last_lands(pa):
    g = torch.Generator().manual_seed(8)
    caches = ref.fresh_i8(2, 2, 64, junk=g)
    _append_both(pa, _rows(g, 6, 2, 64), _rows(g, 6, 2, 64), [5, 20, 5, 6, 20, 5], caches)


def test_append_ties_zeros_and_edges(pa):
    # 254 halves: every tie rounds to even; an all-zero row; the largest bf16 values
    D = 128
    caches = ref.fresh_i8(4, 1, D)
    k = (torch.arange(D) - 63.5).bfloat16().view(1, 1, D).repeat(4, 1, 1)
    k[0, 0, 0] = 127.0
    k[1] = 0
    k[2] *= 1e36
    v = k.flip(2).contiguous()
    _append_both(pa, k, v, [0, 16, 32, 50], caches)
    _append_both(pa, torch.zeros_like(k), torch.zeros_like(v), [1, 17, 33, 51], caches)


def test_append_nonfinite_poisons_its_block_only(pa):
    g = torch.Generator().manual_seed(2)
    k, v = _rows(g, 3, 2, 64), _rows(g, 3, 2, 64)
    k[1, 0, 5] = float("nan")
    v[1, 1, 9] = float("inf")
    gpu = [t.cuda() for t in ref.fresh_i8(3, 2, 64)]
    slots = torch.tensor([0, 16, 32], dtype=torch.int32).cuda()
    pa.pa_cache_append_i8(k.cuda(), v.cuda(), slots, *gpu)
    bad_k, bad_v = ~torch.isfinite(gpu[2]).cpu(), ~torch.isfinite(gpu[3]).cpu()
    assert bad_k.tolist() == [[False, False], [True, False], [False, False]]
    assert bad_v.tolist() == [[False, False], [False, True], [False, False]]
    pa.pa_cache_append_i8(k[:1].cuda(), v[:1].cuda(), slots[1:2], *gpu)  # row 0 again: anew
    assert torch.isfinite(gpu[2]).all() and torch.isfinite(gpu[3]).all()


def test_append_slot_errors_and_many_tokens(pa):
    g = torch.Generator().manual_seed(1)
    caches = ref.fresh_i8(300, 1, 64, junk=g)
    T = 4700
    slots = torch.randperm(300 * 16, generator=g)[:T].tolist()
    slots[17] = 300 * 16
    slots[4000] = 0x7FFFFFFF
    _append_both(pa, _rows(g, T, 1, 64), _rows(g, T, 1, 64), slots, caches)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_SLOT


def _decode_i8(pa, q, batch, lens, scale, **kw):
    k, v, ks, vs, bt = batch
    out = torch.full_like(q, float("nan")).cuda()
    pa.pa_decode_i8(q.cuda(), k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(),
                    torch.tensor(lens, dtype=torch.int32).cuda(), scale, out, **kw)
    assert pa.pa_device_errors(clear=True) == 0
    return out


def _check_decode(pa, q, batch, lens, scale, window, sinks):
    out = _decode_i8(pa, q, batch, lens, scale, window=window, sinks=sinks)
    k, v, ks, vs, bt = batch
    for b, n in enumerate(lens):
        want, mean_abs = ref.attend(q[b:b + 1], *ref.values_i8(k, v, ks, vs, bt[b], n), scale, window, sinks)
        ref.assert_attention(out[b:b + 1], want, mean_abs, DECODE_WEIGHTS)
    return out


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 1, 128), (4, 2, 64), (3, 3, 128), (16, 4, 64), (20, 5, 128),
                                      (48, 6, 64), (7, 7, 64), (32, 8, 64), (64, 8, 128), (16, 16, 128), (80, 20, 64)])
def test_decode_i8_head_layouts(pa, Hq, Hkv, D):
    g = torch.Generator().manual_seed(Hq + Hkv + D)
    lens = [0, 1, 16, 17, 700, 90, 31, 2100]
    q = torch.randn((len(lens), Hq, D), generator=g).bfloat16()
    _check_decode(pa, q, ref.i8_batch(g, lens, Hkv, D), lens, D ** -0.5, ref.ALL, 0)


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (100, 21), (7, 600), (333, 0)])
def test_decode_i8_window(pa, window, sinks):
    g = torch.Generator().manual_seed(window)
    lens = [1, 17, 0, 64, 500, 1000, 115]
    q = torch.randn((len(lens), 16, 64), generator=g).bfloat16()
    _check_decode(pa, q, ref.i8_batch(g, lens, 4, 64), lens, 0.125, window, sinks)


def test_decode_i8_many_and_long_repeats(pa):
    g = torch.Generator().manual_seed(13)
    lens = torch.randint(0, 50, (800,), generator=g).tolist()
    lens[3] = 33333
    batch = ref.i8_batch(g, lens, 2, 64)
    q = torch.randn((len(lens), 8, 64), generator=g).bfloat16()
    out = _check_decode(pa, q, batch, lens, 0.125, ref.ALL, 0)
    assert torch.equal(out, _decode_i8(pa, q, batch, lens, 0.125)), "repeated calls differ"


def test_decode_i8_scales_far_apart(pa):
    # one block in ten has scales 1000 times larger, one in ten values of zero, one in ten a scale of zero
    g = torch.Generator().manual_seed(21)
    lens = [700, 160, 40]
    k, v, ks, vs, bt = ref.i8_batch(g, lens, 2, 128)
    pick = torch.randint(0, 10, ks.shape, generator=g)
    ks = torch.where(pick == 0, ks * 8, ks)
    vs = torch.where(pick == 1, vs * 1000, vs)
    vs = torch.where(pick == 2, 0.0, vs)
    q = torch.randn((3, 8, 128), generator=g).bfloat16()
    _check_decode(pa, q, (k, v, ks, vs, bt), lens, 0.09, ref.ALL, 0)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e5, 1e30])
def test_decode_i8_query_sizes(pa, size):
    # queries far from 1: the scale brings the logits back
    g = torch.Generator().manual_seed(5)
    lens = [300, 20]
    batch = ref.i8_batch(g, lens, 2, 64)
    q = (torch.randn((2, 8, 64), generator=g) * size).bfloat16()
    _check_decode(pa, q, batch, lens, 0.125 / size, ref.ALL, 0)


@pytest.mark.parametrize("window,sinks", [(ref.ALL, 0), (40, 3), (1, 0), (333, 21)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (4, 4, 128), (16, 2, 128), (3, 3, 64)])
def test_prefill_i8(pa, window, sinks, Hq, Hkv, D):
    g = torch.Generator().manual_seed(window % 999 + D + Hq)
    q_lens = [0, 1, 5, 64, 130, 1, 200]
    lens = [9, 1, 5, 300, 130, 517, 900]
    batch = k, v, ks, vs, bt = ref.i8_batch(g, lens, Hkv, D)
    q = torch.randn((sum(q_lens) + 2, Hq, D), generator=g).bfloat16()
    cu = torch.tensor([0] + torch.tensor(q_lens).cumsum(0).tolist(), dtype=torch.int32)
    out = torch.full_like(q, 7.0).cuda()
    pa.pa_prefill_i8(q.cuda(), cu.cuda(), max(q_lens), k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(),
                     torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5, out, window=window, sinks=sinks)
    assert pa.pa_device_errors(clear=True) == 0
    assert (out[sum(q_lens):] == 7.0).all(), "rows behind the last sequence changed"
    for b, n in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        want, mean_abs = ref.attend(q[rows], *ref.values_i8(k, v, ks, vs, bt[b], n), D ** -0.5, window, sinks)
        ref.assert_attention(out[rows], want, mean_abs, PREFILL_WEIGHTS)


@pytest.mark.parametrize("window,sinks", [(ref.ALL, 0), (700, 0), (300, 600), (2400, 4)])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 128), (8, 1, 64), (3, 3, 128)])
def test_prefill_i8_few_rows_long_contexts(pa, window, sinks, Hq, Hkv, D):
    # a tile's keys are shared by the CTAs of a cluster; some have no key that a row sees
    g = torch.Generator().manual_seed(window % 1000 + sinks + D)
    q_lens = [1, 3, 0, 20, 129, 2]
    lens = [4001, 2500, 7, 257, 1100, 513]
    k, v, ks, vs, bt = ref.i8_batch(g, lens, Hkv, D)
    q = torch.randn((sum(q_lens), Hq, D), generator=g).bfloat16()
    cu = torch.tensor([0] + torch.tensor(q_lens).cumsum(0).tolist(), dtype=torch.int32)
    args = (q.cuda(), cu.cuda(), max(q_lens), k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5)
    out = torch.full_like(q, float("nan")).cuda()
    pa.pa_prefill_i8(*args, out, window=window, sinks=sinks)
    assert pa.pa_device_errors(clear=True) == 0
    for b, n in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        want, mean_abs = ref.attend(q[rows], *ref.values_i8(k, v, ks, vs, bt[b], n), D ** -0.5, window, sinks)
        ref.assert_attention(out[rows], want, mean_abs, PREFILL_WEIGHTS)
    again = torch.full_like(out, float("nan"))
    pa.pa_prefill_i8(*args, again, window=window, sinks=sinks)
    assert torch.equal(again, out), "repeated calls differ"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefill_i8_few_rows_nonfinite_scale_reaches_who_sees_it(pa, D, which, bad):
    # windows of rows 0, 1, 2 start at tokens 1998, 1999, 2000; the block of 1984-1999 has a bad scale
    g = torch.Generator().manual_seed(D)
    k, v, ks, vs, bt = ref.i8_batch(g, [3000], 2, D)
    q = torch.randn((3, 4, D), generator=g).bfloat16()
    want, mean_abs = ref.attend(q, *ref.values_i8(k, v, ks, vs, bt[0], 3000), D ** -0.5, 1000, 0)
    (ks if which == "k" else vs)[int(bt[0, 1999 // 16])] = bad
    out = torch.zeros_like(q).cuda()
    pa.pa_prefill_i8(q.cuda(), torch.tensor([0, 3], dtype=torch.int32).cuda(), 3, k.cuda(), v.cuda(), ks.cuda(),
                     vs.cuda(), bt.cuda(), torch.tensor([3000], dtype=torch.int32).cuda(), D ** -0.5, out,
                     window=1000, sinks=0)
    if bad != bad:
        assert torch.isnan(out[:2]).all(), "a NaN scale was dropped"
    ref.assert_attention(out[2:], want[2:], mean_abs[2:], PREFILL_WEIGHTS)


def test_prefill_i8_scales_far_apart(pa):
    g = torch.Generator().manual_seed(22)
    k, v, ks, vs, bt = ref.i8_batch(g, [400], 2, 64)
    pick = torch.randint(0, 10, ks.shape, generator=g)
    vs = torch.where(pick == 1, vs * 1000, vs)
    vs = torch.where(pick == 2, 0.0, vs)
    q = torch.randn((90, 8, 64), generator=g).bfloat16()
    for scale in (0.125, -0.125, 0.0):
        out = torch.full_like(q, float("nan")).cuda()
        pa.pa_prefill_i8(q.cuda(), torch.tensor([0, 90], dtype=torch.int32).cuda(), 90, k.cuda(), v.cuda(), ks.cuda(),
                         vs.cuda(), bt.cuda(), torch.tensor([400], dtype=torch.int32).cuda(), scale, out)
        want, mean_abs = ref.attend(q, *ref.values_i8(k, v, ks, vs, bt[0], 400), scale, ref.ALL, 0)
        ref.assert_attention(out, want, mean_abs, PREFILL_WEIGHTS)


def test_i8_device_errors(pa):
    g = torch.Generator().manual_seed(6)
    k, v, ks, vs, bt = [t.cuda() for t in ref.i8_batch(g, [100], 2, 64)]
    q = torch.randn((1, 4, 64), generator=g).bfloat16().cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    bad = bt.clone()
    bad[0, 2] = 1 << 20
    for table, n, bits in ((bad, 100, pa.PA_DEVERR_BLOCK_ID), (bt, 113, pa.PA_DEVERR_CONTEXT),
                           (bt, -1, pa.PA_DEVERR_CONTEXT)):
        cl = torch.tensor([n], dtype=torch.int32).cuda()
        pa.pa_decode_i8(q, k, v, ks, vs, table, cl, 0.1, out)
        assert pa.pa_device_errors(clear=True) == bits
        pa.pa_prefill_i8(q, cu, 1, k, v, ks, vs, table, cl, 0.1, out)
        assert pa.pa_device_errors(clear=True) == bits


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nonfinite_scale_poisons_who_sees_it_only(pa, D, which):
    # block 1 (tokens 16-31) of kv head 1 has a NaN scale: that head's queries
    # that see it are NaN, its other queries and the other head are untouched
    g = torch.Generator().manual_seed(D)
    k, v, ks, vs, bt = ref.i8_batch(g, [100], 2, D)
    clean = (ks.clone(), vs.clone())
    (ks if which == "k" else vs)[bt[0, 1].long(), 1] = float("nan")
    q = torch.randn((100, 8, D), generator=g).bfloat16()
    cu = torch.tensor([0, 100], dtype=torch.int32).cuda()
    cl = torch.tensor([100], dtype=torch.int32).cuda()
    cache = [t.cuda() for t in (k, v, ks, vs, bt)]
    want, mean_abs = ref.attend(q, *ref.values_i8(k, v, *clean, bt[0], 100), 0.1, 10, 3)
    sees = torch.stack([ref.visible(100, p, 10, 3)[16:32].any() for p in range(100)])
    out = torch.empty_like(q).cuda()
    pa.pa_prefill_i8(q.cuda(), cu, 100, *cache, cl, 0.1, out, window=10, sinks=3)
    got = out.cpu()
    assert torch.isnan(got[sees][:, 4:]).all()
    ref.assert_attention(got[:, :4], want[:, :4], mean_abs[:, :4], PREFILL_WEIGHTS)
    ref.assert_attention(got[~sees][:, 4:], want[~sees][:, 4:], mean_abs[~sees][:, 4:], PREFILL_WEIGHTS)
    for n, poisoned in ((30, True), (60, False)):
        one = torch.empty_like(q[:1]).cuda()
        pa.pa_decode_i8(q[n - 1:n].cuda(), *cache, torch.tensor([n], dtype=torch.int32).cuda(), 0.1, one, window=10,
                        sinks=3)
        ref.assert_attention(one[:, :4], want[n - 1:n, :4], mean_abs[n - 1:n, :4], DECODE_WEIGHTS)
        if poisoned:
            assert torch.isnan(one[:, 4:]).all()
        else:
            ref.assert_attention(one[:, 4:], want[n - 1:n, 4:], mean_abs[n - 1:n, 4:], DECODE_WEIGHTS)


def test_decode_i8_zero_queries_and_scales(pa):
    # all-zero queries, a scale of zero and a negative one
    g = torch.Generator().manual_seed(31)
    lens = [70, 5]
    batch = ref.i8_batch(g, lens, 2, 64)
    q = torch.randn((2, 8, 64), generator=g).bfloat16()
    q[0, 3] = 0
    for scale in (0.125, 0.0, -0.3):
        _check_decode(pa, q, batch, lens, scale, ref.ALL, 0)
