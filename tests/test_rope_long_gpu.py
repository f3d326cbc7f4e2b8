"""The appends of calls long enough to take several rows a thread: groups of rows
that cross from queries to keys to values, odd row counts, padding, queries in
place; and 8-bit appends whose warps take more than one tile of a block."""
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


def _long_enough(T, rows, D):
    """Rows a thread go up once every SM's 2048 threads have four of 16 values (csrc/pa_serving.cu)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return T * rows * (D // 16) >= 4 * 2048 * sms


def _close(got, x, cos_sin, positions, interleaved):
    """One rounding to bf16 (2^-8), products and sums in 32 bits (3 * 2^-24 of the pair's size)."""
    want = ref.rotate(x.double(), cos_sin.double(), positions, interleaved)
    size = x.double().abs().amax(-1, keepdim=True) * 2
    return ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * size).all()


def _inputs(g, T, Hq, Hkv, D, rd, spare):
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=g).bfloat16().cuda()
    nb = T // 16 + spare
    slots = torch.randperm(nb * 16, generator=g)[:T].to(torch.int32)
    positions = torch.randint(0, 4000, (T,), generator=g).to(torch.int32)
    return x, nb, slots, positions, ref.table(4000, rd).cuda()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rd,interleaved", [(22001, 5, 1, 128, 128, False), (22001, 5, 1, 128, 64, True),
                                                       (14501, 7, 7, 64, 64, True), (14501, 7, 7, 64, 32, False),
                                                       (31003, 6, 2, 64, 48, False)])
def test_rope_append_rows_in_fours(pa, T, Hq, Hkv, D, rd, interleaved, in_place):
    assert _long_enough(T, Hq + 2 * Hkv, D)
    g = torch.Generator().manual_seed(T + rd)
    x, nb, slots, positions, cos_sin = _inputs(g, T, Hq, Hkv, D, rd, 9)
    slots[::17] = -1 - torch.arange(len(slots[::17]), dtype=torch.int32)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    kc, vc = (torch.full((nb, Hkv, 16, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q_in = q.contiguous() if in_place else q
    q_out = q_in if in_place else torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_append(q_in, k, v, positions.cuda(), cos_sin, slots.cuda(), q_out, kc, vc, interleaved=interleaved)
    assert pa.pa_device_errors(clear=True) == 0
    live = (slots >= 0).cuda()
    at = positions.cuda()[live]
    assert _close(q_out[live], q[live], cos_sin, at, interleaved)
    kept = q[~live] if in_place else torch.full_like(q[~live], 9.0)
    assert torch.equal(q_out[~live], kept), "a padding token's q row changed"
    s = slots.cuda()[live].long()
    assert _close(kc[s // 16, :, s % 16], k[live], cos_sin, at, interleaved)
    assert torch.equal(vc[s // 16, :, s % 16], v[live])
    kc[s // 16, :, s % 16] = 5.0
    vc[s // 16, :, s % 16] = 5.0
    assert (kc == 5.0).all() and (vc == 5.0).all(), "other rows changed"


@pytest.mark.parametrize("T,Hq,Hkv,D,rd,interleaved", [(22001, 7, 1, 128, 128, False), (22001, 7, 1, 128, 32, True),
                                                       (28001, 11, 1, 64, 64, True),
                                                       (590, 3, 16, 64, 64, False), (590, 2, 16, 128, 64, True),
                                                       (1500, 2, 20, 64, 0, False)])
def test_rope_append_i8_long(pa, T, Hq, Hkv, D, rd, interleaved):
    assert Hkv > 1 or _long_enough(T, Hq, D)
    g = torch.Generator().manual_seed(T + D + rd)
    x, nb, slots, positions, cos_sin = _inputs(g, T, Hq, Hkv, D, rd, 9)
    slots[5], slots[T - 3] = -1, -7
    caches = ref.fresh_i8(nb, Hkv, D, junk=g)
    gpu = [t.cuda() for t in caches]
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    q_out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_append_i8(q, k, v, positions.cuda(), cos_sin, slots.cuda(), q_out, *gpu, interleaved=interleaved)
    assert pa.pa_device_errors(clear=True) == 0
    live = (slots >= 0).cuda()
    assert _close(q_out[live], q[live], cos_sin, positions.cuda()[live], interleaved)
    assert (q_out[~live] == 9.0).all(), "a padding token's q row changed"
    rows = ref.rotate(k.cpu().float(), cos_sin.cpu(), positions, interleaved)
    ref.append_i8(rows, v.cpu().float(), slots.tolist(), caches)
    for name, a, b in zip(("k codes", "v codes", "k scales", "v scales"), gpu, caches):
        assert torch.equal(a.cpu(), b), name + " differ from the definition"
