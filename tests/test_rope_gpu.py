"""The append with rotation against the definition: bf16 rows within their
rounding, 8-bit codes and scales bit by bit; both pairings, partial
rotation, strided rows, in-place queries, padding and far positions."""
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


def _fused(gen, T, Hq, Hkv, D):
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=gen).bfloat16()
    return x, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _assert_turned(got, x, cos_sin, positions, interleaved):
    """One rounding to bf16 (2^-8 relative), products and sums in 32 bits (3 * 2^-24 of the pair's size)."""
    want = ref.rotate(x.double(), cos_sin.double(), positions, interleaved)
    size = ref.rotate(x.double().abs(), cos_sin.double().abs(), positions, interleaved).abs() + \
        x.double().abs().amax(-1, keepdim=True)
    err = (got.double().cpu() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * size).all(), f"max error {err.max():.3g}"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rd", [(1, 1, 1, 64, 64), (7, 8, 2, 64, 32), (33, 32, 8, 128, 128), (5, 6, 3, 128, 64),
                                           (64, 20, 5, 64, 16), (9, 4, 4, 96, 48), (300, 16, 8, 128, 0), (2, 3, 1, 256, 256)])
def test_rope_append(pa, T, Hq, Hkv, D, rd, interleaved):
    g = torch.Generator().manual_seed(T + D + rd)
    nb = T // 16 + 5
    x, q, k, v = _fused(g, T, Hq, Hkv, D)
    slots = torch.randperm(nb * 16, generator=g)[:T].to(torch.int32)
    pad = T > 4
    if pad:
        slots[T // 2] = -1
    positions = torch.randint(0, 5000, (T,), generator=g).to(torch.int32)
    cos_sin = ref.table(5000, rd)
    kc = torch.randn((nb, Hkv, 16, D), generator=g).bfloat16()
    vc = torch.randn((nb, Hkv, 16, D), generator=g).bfloat16()
    gkc, gvc, gx = kc.cuda(), vc.cuda(), x.cuda()
    q_out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_append(gx[:, :Hq], gx[:, Hq:Hq + Hkv], gx[:, Hq + Hkv:], positions.cuda(), cos_sin.cuda(),
                      slots.cuda(), q_out, gkc, gvc, interleaved=interleaved)
    assert pa.pa_device_errors(clear=True) == 0
    live = slots >= 0
    blk, off = slots[live].long() // 16, slots[live].long() % 16
    _assert_turned(q_out[live.cuda()], q[live], cos_sin, positions[live], interleaved)
    assert (q_out[(~live).cuda()] == 9.0).all(), "a padding token's q row changed"
    _assert_turned(gkc.cpu()[blk, :, off], k[live], cos_sin, positions[live], interleaved)
    assert torch.equal(gvc.cpu()[blk, :, off], v[live])
    # nothing else changed
    kc[blk, :, off], vc[blk, :, off] = gkc.cpu()[blk, :, off], v[live]
    assert torch.equal(gkc.cpu(), kc) and torch.equal(gvc.cpu(), vc)


def test_rope_append_in_place_without_queries_and_other_block_sizes(pa):
    g = torch.Generator().manual_seed(1)
    T, Hq, Hkv, D = 40, 8, 2, 64
    _, q, k, v = _fused(g, T, Hq, Hkv, D)
    cos_sin, positions = ref.table(64, D), torch.arange(T, dtype=torch.int32)
    slots = torch.arange(T, dtype=torch.int32).flip(0).contiguous()
    for bs in (16, 32, 5):
        kc = torch.zeros((9, Hkv, bs, D), dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        gq = q.contiguous().cuda()
        pa.pa_rope_append(gq, k.contiguous().cuda(), v.contiguous().cuda(), positions.cuda(), cos_sin.cuda(),
                          slots.cuda(), gq, kc, vc)
        _assert_turned(gq, q, cos_sin, positions, False)
        s = slots.long()
        _assert_turned(kc.cpu()[s // bs, :, s % bs], k, cos_sin, positions, False)
        kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
        pa.pa_rope_append(None, k.contiguous().cuda(), v.contiguous().cuda(), positions.cuda(), cos_sin.cuda(),
                          slots.cuda(), None, kc2, vc2)
        assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_rope_far_positions(pa):
    # angles of a million tokens come from the table, so position costs no precision
    g = torch.Generator().manual_seed(2)
    T, D = 6, 64
    _, q, k, v = _fused(g, T, 2, 1, D)
    cos_sin = ref.table(1 << 20, 32)
    positions = torch.tensor([0, 1, 65535, 131071, 999999, (1 << 20) - 1], dtype=torch.int32)
    kc = torch.zeros((1, 1, 16, D), dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty((T, 2, D), dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_append(q.cuda(), k.cuda(), v.cuda(), positions.cuda(), cos_sin.cuda(),
                      torch.arange(T, dtype=torch.int32).cuda(), q_out, kc, kc.clone())
    _assert_turned(q_out, q, cos_sin, positions, False)


def test_rope_device_errors(pa):
    g = torch.Generator().manual_seed(3)
    _, q, k, v = _fused(g, 2, 2, 1, 64)
    cos_sin = ref.table(10, 64).cuda()
    kc = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    i8 = [t.cuda() for t in ref.fresh_i8(1, 1, 64)]
    q_out = torch.empty((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for positions, slots, bits in (([0, 10], [0, 1], pa.PA_DEVERR_POSITION), ([-1, 9], [0, 1], pa.PA_DEVERR_POSITION),
                                   ([0, 9], [0, 16], pa.PA_DEVERR_SLOT), ([0, 77], [0, -1], 0)):
        args = (q.cuda(), k.cuda(), v.cuda(), torch.tensor(positions, dtype=torch.int32).cuda(), cos_sin,
                torch.tensor(slots, dtype=torch.int32).cuda(), q_out)
        pa.pa_rope_append(*args, kc, kc.clone())
        assert pa.pa_device_errors(clear=True) == bits
        pa.pa_rope_append_i8(*args, *i8)
        assert pa.pa_device_errors(clear=True) == bits


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rd", [(1, 1, 1, 64, 64), (70, 8, 2, 64, 32), (130, 32, 8, 128, 128), (50, 6, 3, 128, 48),
                                           (90, 4, 4, 64, 16), (40, 8, 8, 128, 0)])
def test_rope_append_i8(pa, T, Hq, Hkv, D, rd, interleaved):
    g = torch.Generator().manual_seed(T + D + rd)
    nb = T // 16 + 4
    x, q, k, v = _fused(g, T, Hq, Hkv, D)
    positions = torch.randint(0, 3000, (T,), generator=g).to(torch.int32)
    cos_sin = ref.table(3000, rd)
    # a chunk that starts inside a block, then loose slots in any order
    slots = list(range(21, 21 + T // 2))
    rest = [s for s in torch.randperm(nb * 16, generator=g).tolist() if s not in set(slots)]
    slots = slots + rest[: T - len(slots)]
    caches = ref.fresh_i8(nb, Hkv, D, junk=g)
    gpu, gx = [t.cuda() for t in caches], x.cuda()
    q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_append_i8(gx[:, :Hq], gx[:, Hq:Hq + Hkv], gx[:, Hq + Hkv:], positions.cuda(), cos_sin.cuda(),
                         torch.tensor(slots, dtype=torch.int32).cuda(), q_out, *gpu, interleaved=interleaved)
    assert pa.pa_device_errors(clear=True) == 0
    _assert_turned(q_out, q, cos_sin, positions, interleaved)
    ref.append_i8(ref.rotate(k.float(), cos_sin, positions, interleaved), v.float(), slots, caches)
    for name, a, b in zip(("k codes", "v codes", "k scales", "v scales"), gpu, caches):
        assert torch.equal(a.cpu(), b), name + " differ from the definition"
