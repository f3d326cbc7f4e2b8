"""What a call reads is what the calls before it on its stream wrote, though its
kernel may start before theirs end: a rotating append into the same cache over
and over, each time followed at once by an attention call that reads the turned
queries, rows, codes and scales.  The same call on the settled tensors gives the
same bits."""
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


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("multi", [False, True])
@pytest.mark.parametrize("B,n,Hq,Hkv,D", [(64, 33, 8, 8, 64), (3, 500, 8, 2, 128), (1, 1, 4, 4, 128), (40, 70, 16, 4, 64)])
def test_attention_sees_the_append_before_it(pa, i8, multi, B, n, Hq, Hkv, D):
    g = torch.Generator().manual_seed(B + n)
    bt, nb = ref.tables(g, [n] * B)
    if i8:
        cache = [t.cuda() for t in ref.fresh_i8(nb, Hkv, D)]
    else:
        cache = [torch.zeros((nb, Hkv, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    T, table = B * n, bt.cuda()
    slots = torch.tensor([s for b in range(B) for s in ref.slots_of(bt, b, 0, n)], dtype=torch.int32).cuda()
    pos = torch.arange(n, dtype=torch.int32).repeat(B).cuda()
    cos_sin, cl = ref.table(n, D).cuda(), torch.full((B,), n, dtype=torch.int32, device="cuda")
    q_rot = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    q_in = q_rot if multi else q_rot[:B]
    outs = [torch.zeros_like(q_in) for _ in range(2)]
    append = pa.prepare_rope_append_i8 if i8 else pa.prepare_rope_append
    if multi:
        cu = (torch.arange(B + 1, dtype=torch.int32) * n).cuda()
        attend = pa.prepare_prefill_i8 if i8 else pa.prepare_prefill_window
        calls = [attend(q_in, cu, n, *cache, table, cl, D ** -0.5, o, window=None) for o in outs]
    else:
        attend = pa.prepare_decode_i8 if i8 else pa.prepare_decode_window
        ws = pa.alloc_workspace(pa.make_dims(q_in, cache[0], bt))
        calls = [attend(q_in, *cache, table, cl, D ** -0.5, o, ws, window=None) for o in outs]
    steps = [torch.randn((T, Hq + 2 * Hkv, D), generator=g).bfloat16().cuda() * s for s in (1.0, 0.01, 3.0)]
    appends = [append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos, cos_sin, slots, q_rot, *cache) for x in steps]
    torch.cuda.synchronize()
    for i in range(30):
        appends[i % 3]()
        appends[(i + 1) % 3]()
        calls[0]()
        torch.cuda.synchronize()
        calls[1]()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]), f"step {i}: the attention read what the append had not written yet"
    assert torch.isfinite(outs[0]).all() and pa.pa_device_errors(clear=True) == 0
