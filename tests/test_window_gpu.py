"""Sliding-window attention with sinks against the definition in 64 bits:
windows and sinks that end inside a page, that touch, that leave pages
unread (their table entries and rows are poisoned), empty and one-token
contexts, long contexts split over CTAs, every head layout."""
import pytest
import torch

from tests import paging, serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_kv_attention_36_b200 import binding
    binding.pa_device_errors(clear=True)
    return binding


def _forget(kp, vp, bt, lens, oldest, window, sinks):
    """Poisons what no query of the batch sees: rows, and the table entries of
    whole pages.  oldest[b] = position of b's first query."""
    for b, n in enumerate(lens):
        if n == 0:
            continue
        seen = torch.zeros(((n + 15) // 16) * 16, dtype=torch.bool)
        for p in range(oldest[b], n):
            seen[:n] |= ref.visible(n, p, window, sinks)
        for j in range(0, len(seen) // 16):
            blk = int(bt[b, j])
            gone = ~seen[16 * j: 16 * j + 16]
            for pool in (kp, vp):
                pool[blk].view(torch.int16)[:, gone] = paging.NAN_BITS
            if gone.all():
                bt[b, j] = ref.PAD_BLOCK
    return kp, vp, bt


def _decode_ref(q, ks, vs, lens, scale, window, sinks):
    pairs = [ref.attend(q[b:b + 1], ks[b].double(), vs[b].double(), scale, window, sinks) for b in range(len(lens))]
    return torch.cat([o for o, _ in pairs]), torch.cat([a for _, a in pairs])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 0), (64, 4), (100, 21), (333, 40), (50, 400),
                                          (ref.ALL, 0), (ref.ALL, ref.ALL), (5, ref.ALL)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (8, 8, 128)])
def test_decode_window(pa, window, sinks, Hq, Hkv, D):
    g = torch.Generator().manual_seed(window % 1000 + sinks % 1000 + D)
    lens = [0, 1, 15, 16, 17, 33, 64, 65, 100, 257, 340, 1000]
    ks, vs, kp, vp, bt = ref.bf16_batch(g, lens, Hkv, D)
    kp, vp, bt = _forget(kp, vp, bt, lens, [n - 1 for n in lens], window, sinks)
    q = torch.randn((len(lens), Hq, D), generator=g).bfloat16()
    want, mean_abs = _decode_ref(q, ks, vs, lens, D ** -0.5, window, sinks)
    out = torch.full_like(q, float("nan")).cuda()
    pa.pa_decode_window(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                        D ** -0.5, out, window=window, sinks=sinks)
    assert pa.pa_device_errors(clear=True) == 0
    ref.assert_attention(out, want, mean_abs, 2.0 ** -16)


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (2, 1, 128), (3, 3, 64), (20, 5, 128), (32, 4, 64), (14, 7, 128),
                                      (64, 16, 128), (24, 24, 64)])
def test_decode_window_head_layouts(pa, Hq, Hkv, D):
    g = torch.Generator().manual_seed(Hq * 100 + Hkv)
    lens = [700, 3, 0, 90, 2000]
    ks, vs, kp, vp, bt = ref.bf16_batch(g, lens, Hkv, D)
    q = torch.randn((len(lens), Hq, D), generator=g).bfloat16()
    want, mean_abs = _decode_ref(q, ks, vs, lens, D ** -0.5, 200, 5)
    out = torch.full_like(q, float("nan")).cuda()
    pa.pa_decode_window(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                        D ** -0.5, out, window=200, sinks=5)
    assert pa.pa_device_errors(clear=True) == 0
    ref.assert_attention(out, want, mean_abs, 2.0 ** -16)


def test_decode_window_many_and_long(pa):
    # more sequences than a CTA has threads, and one context whose window is cut over CTAs
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 60, (700,), generator=g).tolist()
    lens[350] = 40000
    ks, vs, kp, vp, bt = ref.bf16_batch(g, lens, 2, 64)
    q = torch.randn((len(lens), 4, 64), generator=g).bfloat16()
    want, mean_abs = _decode_ref(q, ks, vs, lens, 0.125, 30011, 7)
    out = torch.full_like(q, float("nan")).cuda()
    args = (q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.125)
    pa.pa_decode_window(*args, out, window=30011, sinks=7)
    assert pa.pa_device_errors(clear=True) == 0
    ref.assert_attention(out, want, mean_abs, 2.0 ** -16)
    again = torch.empty_like(out)
    pa.pa_decode_window(*args, again, window=30011, sinks=7)
    assert torch.equal(out, again), "repeated calls differ"


def test_decode_window_of_everything_is_decode(pa):
    g = torch.Generator().manual_seed(4)
    lens = [5, 900, 64, 0]
    _, _, kp, vp, bt = ref.bf16_batch(g, lens, 4, 128)
    q = torch.randn((4, 16, 128), generator=g).bfloat16().cuda()
    args = (q, kp.cuda(), vp.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.09)
    a, b = torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode(*args, a)
    pa.pa_decode_window(*args, b, window=None)
    assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-6)


def test_window_negative_and_zero_scale(pa):
    g = torch.Generator().manual_seed(5)
    lens = [40, 300]
    ks, vs, kp, vp, bt = ref.bf16_batch(g, lens, 2, 64)
    q = torch.randn((2, 8, 64), generator=g).bfloat16()
    cl = torch.tensor(lens, dtype=torch.int32)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32)
    for scale in (-0.2, 0.0):
        want, mean_abs = _decode_ref(q, ks, vs, lens, scale, 33, 2)
        for multi in (False, True):
            out = torch.full_like(q, float("nan")).cuda()
            if multi:
                pa.pa_prefill_window(q.cuda(), cu.cuda(), 1, kp.cuda(), vp.cuda(), bt.cuda(), cl.cuda(), scale, out,
                                     window=33, sinks=2)
            else:
                pa.pa_decode_window(q.cuda(), kp.cuda(), vp.cuda(), bt.cuda(), cl.cuda(), scale, out, window=33,
                                    sinks=2)
            ref.assert_attention(out, want, mean_abs, 2.0 ** -8 if multi else 2.0 ** -16)


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 1), (16, 16), (63, 0), (64, 4), (65, 70), (333, 21),
                                          (20, 300), (ref.ALL, 0)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (4, 4, 128), (16, 2, 128)])
def test_prefill_window(pa, window, sinks, Hq, Hkv, D):
    g = torch.Generator().manual_seed(window % 1000 + 7 * (sinks % 1000) + D)
    q_lens = [0, 1, 5, 64, 130, 1, 200]
    lens = [9, 1, 5, 300, 130, 517, 900]
    ks, vs, kp, vp, bt = ref.bf16_batch(g, lens, Hkv, D)
    kp, vp, bt = _forget(kp, vp, bt, lens, [n - c for n, c in zip(lens, q_lens)], window, sinks)
    q = torch.randn((sum(q_lens) + 3, Hq, D), generator=g).bfloat16()  # 3 rows behind the last sequence
    cu = torch.tensor([0] + torch.tensor(q_lens).cumsum(0).tolist(), dtype=torch.int32)
    out = torch.full_like(q, 7.0).cuda()
    pa.pa_prefill_window(q.cuda(), cu.cuda(), max(q_lens), kp.cuda(), vp.cuda(), bt.cuda(),
                         torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5, out, window=window, sinks=sinks)
    assert pa.pa_device_errors(clear=True) == 0
    assert (out[sum(q_lens):] == 7.0).all(), "rows behind the last sequence changed"
    for b, n in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        want, mean_abs = ref.attend(q[rows], ks[b].double(), vs[b].double(), D ** -0.5, window, sinks)
        ref.assert_attention(out[rows], want, mean_abs, 2.0 ** -8)


def test_prefill_window_head_layouts(pa):
    for Hq, Hkv, D in ((1, 1, 64), (3, 3, 128), (32, 8, 64), (8, 1, 128)):
        g = torch.Generator().manual_seed(Hq + D)
        q_lens, lens = [33, 70], [33, 260]
        ks, vs, kp, vp, bt = ref.bf16_batch(g, lens, Hkv, D)
        q = torch.randn((sum(q_lens), Hq, D), generator=g).bfloat16()
        cu = torch.tensor([0, 33, 103], dtype=torch.int32)
        out = torch.full_like(q, float("nan")).cuda()
        pa.pa_prefill_window(q.cuda(), cu.cuda(), 70, kp.cuda(), vp.cuda(), bt.cuda(),
                             torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5, out, window=50, sinks=3)
        for b in range(2):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            want, mean_abs = ref.attend(q[rows], ks[b].double(), vs[b].double(), D ** -0.5, 50, 3)
            ref.assert_attention(out[rows], want, mean_abs, 2.0 ** -8)


@pytest.mark.parametrize("window,sinks", [(ref.ALL, 0), (700, 0), (1500, 100), (300, 600), (60, 2000), (2400, 4)])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 128), (8, 1, 64), (3, 3, 128)])
def test_prefill_window_few_rows_long_contexts(pa, window, sinks, Hq, Hkv, D):
    # a tile's keys are shared by the CTAs of a cluster; some have no key that a row sees
    g = torch.Generator().manual_seed(window % 1000 + sinks + D)
    q_lens = [1, 3, 0, 20, 129, 2]
    lens = [4001, 2500, 7, 257, 1100, 513]
    ks, vs, kp, vp, bt = ref.bf16_batch(g, lens, Hkv, D)
    kp, vp, bt = _forget(kp, vp, bt, lens, [n - c for n, c in zip(lens, q_lens)], window, sinks)
    q = torch.randn((sum(q_lens), Hq, D), generator=g).bfloat16()
    cu = torch.tensor([0] + torch.tensor(q_lens).cumsum(0).tolist(), dtype=torch.int32)
    out = torch.full_like(q, float("nan")).cuda()
    args = (q.cuda(), cu.cuda(), max(q_lens), kp.cuda(), vp.cuda(), bt.cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5)
    pa.pa_prefill_window(*args, out, window=window, sinks=sinks)
    assert pa.pa_device_errors(clear=True) == 0
    for b, n in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        want, mean_abs = ref.attend(q[rows], ks[b].double(), vs[b].double(), D ** -0.5, window, sinks)
        ref.assert_attention(out[rows], want, mean_abs, 2.0 ** -8)
    again = torch.full_like(out, float("nan"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prefill_window(*args, again, window=window, sinks=sinks)
        pa.pa_prefill_window(*args, again, window=window, sinks=sinks)
    graph.replay()
    assert torch.equal(again, out), "a replayed call differs"


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_window_few_rows_nan_key_reaches_who_sees_it(pa, D):
    # windows of rows 0, 1, 2 start at tokens 1998, 1999, 2000; key 1999 is NaN
    g = torch.Generator().manual_seed(D)
    ks, vs, kp, vp, bt = ref.bf16_batch(g, [3000], 2, D)
    blk = int(bt[0, 1999 // 16])
    q = torch.randn((3, 4, D), generator=g).bfloat16()
    args = (bt.cuda(), torch.tensor([3000], dtype=torch.int32).cuda(), D ** -0.5)
    kp[blk, :, 1999 % 16] = float("nan")
    out = torch.zeros_like(q).cuda()
    pa.pa_prefill_window(q.cuda(), torch.tensor([0, 3], dtype=torch.int32).cuda(), 3, kp.cuda(), vp.cuda(), *args, out,
                         window=1000, sinks=0)
    assert torch.isnan(out[:2]).all(), "a NaN key was dropped"
    want, mean_abs = ref.attend(q, ks[0].double(), vs[0].double(), D ** -0.5, 1000, 0)
    ref.assert_attention(out[2:], want[2:], mean_abs[2:], 2.0 ** -8)


def test_window_device_errors(pa):
    # a bad block id inside the window is reported; one outside it is never read
    g = torch.Generator().manual_seed(6)
    _, _, kp, vp, bt = ref.bf16_batch(g, [200], 2, 64)
    q = torch.randn((1, 4, 64), generator=g).bfloat16().cuda()
    cl = torch.tensor([200], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    for entry, bits in ((3, 0), (11, pa.PA_DEVERR_BLOCK_ID)):
        bad = bt.clone()
        bad[0, entry] = -5
        pa.pa_decode_window(q, kp.cuda(), vp.cuda(), bad.cuda(), cl, 0.1, out, window=64, sinks=16)
        assert pa.pa_device_errors(clear=True) == bits
        pa.pa_prefill_window(q, cu, 1, kp.cuda(), vp.cuda(), bad.cuda(), cl, 0.1, out, window=64, sinks=16)
        assert pa.pa_device_errors(clear=True) == bits
    long = torch.tensor([5000], dtype=torch.int32).cuda()
    full = torch.zeros_like(bt).cuda()
    pa.pa_decode_window(q, kp.cuda(), vp.cuda(), full, long, 0.1, out, window=64)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_CONTEXT
    pa.pa_prefill_window(q, cu, 1, kp.cuda(), vp.cuda(), full, long, 0.1, out, window=64)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_CONTEXT
