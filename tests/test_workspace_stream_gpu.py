"""Decodes on a side stream without a workspace, while the default stream
allocates and fills memory of the workspace's size: contexts cut over many CTAs
come out as they do with a workspace of the caller's."""
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


@pytest.mark.parametrize("what", ["pa_decode", "pa_decode_window", "pa_decode_i8"])
def test_workspace_of_a_call_on_a_side_stream(pa, what):
    g = torch.Generator().manual_seed(3)
    lens, Hq, Hkv, D = [20000, 9000, 5], 8, 2, 128
    q = torch.randn((3, Hq, D), generator=g).bfloat16().cuda()
    if what == "pa_decode_i8":
        k, v, ks, vs, bt = [t.cuda() for t in ref.i8_batch(g, lens, Hkv, D)]
        cache = (k, v, ks, vs)
    else:
        _, _, k, v, bt = ref.bf16_batch(g, lens, Hkv, D)
        bt, cache = bt.cuda(), (k.cuda(), v.cuda())
    args = (q, *cache, bt, torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5)
    kw = {} if what == "pa_decode" else dict(window=None)
    call = getattr(pa, what)
    want = torch.empty_like(q)
    ws = pa.alloc_workspace(pa.make_dims(q, cache[0], bt))
    call(*args, want, workspace=ws, **kw)
    side = torch.cuda.Stream()
    outs = [torch.zeros_like(q) for _ in range(30)]
    torch.cuda.synchronize()
    for out in outs:
        call(*args, out, stream=side, **kw)
        torch.full((ws.numel(),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)
    assert pa.pa_device_errors(clear=True) == 0
