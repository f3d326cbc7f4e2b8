"""Without a GPU: the windowed, 8-bit and rotating-append calls refuse bad
arguments before any CUDA call, the window's page lists and segment cuts hold
under brute force, and the test-side 64-bit definitions agree with torch."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from tests import serving_ref as ref

HERE = os.path.dirname(os.path.abspath(__file__))
OK, NULL, SHAPE, UNSUPPORTED, ALIGN = 0, -1, -2, -3, -4


@pytest.fixture(scope="module")
def binding():
    from paged_kv_attention_36_b200 import build
    build.build()
    from paged_kv_attention_36_b200 import binding
    return binding


def test_window_lists_and_cuts_brute_force(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "window_check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", os.path.join(HERE, "window_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.startswith("ok"), out.stdout + out.stderr


# ---- the definitions ------------------------------------------------------------

@pytest.mark.parametrize("window,sinks", [(ref.ALL, 0), (1, 0), (7, 3), (20, 50)])
def test_definition_of_attention_against_torch(window, sinks):
    g = torch.Generator().manual_seed(window % 100 + sinks)
    L, n, Hq, Hkv, D = 40, 9, 6, 2, 16
    q = torch.randn((n, Hq, D), generator=g, dtype=torch.float64)
    k, v = (torch.randn((Hkv, L, D), generator=g, dtype=torch.float64) for _ in range(2))
    mask = torch.stack([ref.visible(L, L - n + i, window, sinks) for i in range(n)])
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.repeat_interleave(3, 0), v.repeat_interleave(3, 0), attn_mask=mask, scale=0.3)
    got, mean_abs = ref.attend(q, k, v, 0.3, window, sinks)
    assert torch.allclose(got, want.transpose(0, 1), atol=1e-12)
    assert (mean_abs >= got.abs() - 1e-12).all()


def test_definition_of_the_8bit_append():
    caches = ref.fresh_i8(2, 1, 64)
    x = torch.zeros((1, 1, 64))
    x[0, 0, :3] = torch.tensor([127.0, -2.5, 3.5])
    ref.append_i8(x, x, [0], caches)  # scale 1: ties to even
    assert caches[2][0, 0] == 1.0 and caches[0][0, 0, 0, :3].tolist() == [127, -2, 4]
    assert caches[1][0, 0, :3, ref.v_byte(0)].tolist() == [127, -2, 4]
    ref.append_i8(2 * x, 2 * x, [3], caches)  # twice as large: the scale doubles, row 0 is rounded again
    assert caches[2][0, 0] == 2.0 and caches[0][0, 0, 0, :3].tolist() == [64, -1, 2]
    ref.append_i8(x, x, [0], caches)  # row 0 again: the block starts anew
    assert caches[2][0, 0] == 1.0 and caches[0][0, 0, 3].abs().max() == 0


def test_definition_of_rotation_keeps_lengths():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((5, 2, 32), generator=g, dtype=torch.float64)
    t = ref.table(50, 16).double()
    pos = torch.tensor([0, 1, 7, 30, 49])
    for interleaved in (False, True):
        y = ref.rotate(x, t, pos, interleaved)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-6) and torch.equal(y[..., 16:], x[..., 16:])
        assert torch.allclose(y[0], x[0])


# ---- refusals of the C ABI --------------------------------------------------------

def _dims(binding, **kw):
    d = dict(num_seqs=4, num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=16, num_blocks=64,
             max_blocks_per_seq=7)
    d.update(kw)
    return binding.pa_dims(*[d[n] for n, _ in binding.pa_dims._fields_])


def _attend(binding, what, dims, window=64, sinks=4, mq=8, ks=16, vs=16, cu=16, **ptr):
    vp = ctypes.c_void_p
    p = dict(q=16, k=16, v=16, bt=16, cl=16, out=16, ws=16, ws_bytes=0)
    p.update(ptr)
    head = [vp(p["q"])] + ([vp(cu), mq] if "prefill" in what else []) + [vp(p["k"]), vp(p["v"])]
    if what.endswith("i8"):
        head += [vp(ks), vp(vs)]
    tail = [vp(p["ws"]), p["ws_bytes"]] if "decode" in what else []
    return getattr(binding.lib, what)(*head, vp(p["bt"]), vp(p["cl"]), 0.1, window, sinks, vp(p["out"]),
                                      ctypes.byref(dims) if dims is not None else None, *tail, vp(0))


CALLS = ["pa_decode_window", "pa_prefill_window", "pa_decode_i8", "pa_prefill_i8"]


@pytest.mark.parametrize("what", CALLS)
def test_attention_refusals(binding, what):
    call = lambda dims=_dims(binding), **kw: _attend(binding, what, dims, **kw)  # noqa: E731
    assert call(None) == NULL
    assert call(window=0) == SHAPE and call(window=-5) == SHAPE and call(sinks=-1) == SHAPE
    assert call(_dims(binding, num_q_heads=6, num_kv_heads=4)) == SHAPE
    assert call(_dims(binding, num_q_heads=6, num_kv_heads=2)) == UNSUPPORTED  # three query heads per kv head
    assert call(_dims(binding, head_dim=96)) == UNSUPPORTED
    assert call(_dims(binding, block_size=32)) == UNSUPPORTED
    assert call(_dims(binding, num_blocks=0)) == SHAPE
    for name in ("q", "k", "v", "bt", "cl", "out"):
        assert call(**{name: 0}) == NULL, name
    for name in ("q", "k", "v", "out"):
        assert call(**{name: 24}) == ALIGN, name
    assert call(bt=18) == ALIGN and call(cl=18) == ALIGN
    assert call(_dims(binding, num_seqs=0)) == OK
    if "prefill" in what:
        assert call(mq=-1) == SHAPE and call(mq=0) == OK and call(cu=0) == NULL and call(cu=18) == ALIGN
        assert call(_dims(binding, num_seqs=1 << 30), mq=1 << 30) == SHAPE
        assert call(_dims(binding, num_blocks=1 << 28)) == SHAPE
        if what.endswith("i8"):  # decode calls need a device to get this far
            assert call(ks=0) == NULL and call(vs=0) == NULL and call(ks=18) == ALIGN


def _append(binding, i8, dims, T=3, q=16, q_stride=512, k=16, k_stride=128, v=16, v_stride=128, rd=64, max_position=10,
            positions=16, cos_sin=16, slots=16, q_out=1 << 20, kc=16, vc=16, ks=16, vs=16, rope=True):
    vp = ctypes.c_void_p
    r = ctypes.byref(binding.pa_rope(positions, cos_sin, max_position, rd, 0)) if rope else None
    args = [vp(q), q_stride, vp(k), k_stride, vp(v), v_stride, r, vp(slots), T, vp(q_out), vp(kc), vp(vc)]
    args += [vp(ks), vp(vs)] if i8 else []
    fn = binding.lib.pa_rope_append_i8 if i8 else binding.lib.pa_rope_append
    return fn(*args, ctypes.byref(dims) if dims is not None else None, vp(0))


@pytest.mark.parametrize("i8", [False, True])
def test_rotating_append_refusals(binding, i8):
    call = lambda dims=_dims(binding), **kw: _append(binding, i8, dims, **kw)  # noqa: E731
    assert call(None) == NULL
    assert call(T=-1) == SHAPE and call(T=0) == OK
    assert call(rd=-16) == SHAPE and call(rd=80) == SHAPE and call(rd=24) == UNSUPPORTED
    assert call(_dims(binding, head_dim=24), rd=16) == UNSUPPORTED
    assert call(_dims(binding, num_kv_heads=0)) == SHAPE
    assert call(k=0) == NULL and call(v=0) == NULL and call(slots=0) == NULL and call(kc=0) == NULL
    assert call(q_out=0) == NULL and call(positions=0) == NULL and call(cos_sin=0) == NULL
    assert call(max_position=0) == SHAPE
    assert call(k=24) == ALIGN and call(q=24) == ALIGN and call(cos_sin=20) == ALIGN and call(slots=18) == ALIGN
    assert call(q_stride=504) == SHAPE and call(k_stride=120) == SHAPE and call(v_stride=-128) == SHAPE
    assert call(q_stride=516) == ALIGN and call(k_stride=132) == ALIGN
    # q_out over q: only q itself, when it is dense
    assert call(q=1 << 20, q_stride=1024) == SHAPE
    assert call(q=(1 << 20) + 1024) == SHAPE and call(q=(1 << 20) - 1024) == SHAPE
    assert call(_dims(binding, num_blocks=1 << 28)) == SHAPE
    if i8:
        assert call(_dims(binding, head_dim=96)) == UNSUPPORTED and call(_dims(binding, block_size=32)) == UNSUPPORTED
        assert call(ks=0) == NULL and call(vs=0) == NULL and call(ks=18) == ALIGN


def test_append_i8_refusals(binding):
    vp = ctypes.c_void_p
    f = binding.lib.pa_cache_append_i8

    def call(dims=_dims(binding), T=3, k=16, v=16, slots=16, kc=16, vc=16, ks=16, vs=16):
        return f(vp(k), vp(v), vp(slots), T, vp(kc), vp(vc), vp(ks), vp(vs),
                 ctypes.byref(dims) if dims is not None else None, vp(0))
    assert call(None) == NULL and call(T=-1) == SHAPE and call(T=0) == OK
    assert call(_dims(binding, head_dim=32)) == UNSUPPORTED and call(_dims(binding, block_size=8)) == UNSUPPORTED
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert call(**{name: 0}) == NULL, name
    for name in ("k", "v", "kc", "vc"):
        assert call(**{name: 24}) == ALIGN, name


# ---- refusals of the binding -------------------------------------------------------

def test_binding_refusals(binding):
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    kc = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    bt, cl = torch.zeros((2, 1), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    out = torch.empty_like(q)
    for bad in (dict(window=0), dict(window=-1), dict(window=1 << 31), dict(window=4, sinks=-1)):
        with pytest.raises(ValueError, match="window"):
            binding.pa_decode_window(q, kc, kc, bt, cl, 0.1, out, **bad)
    with pytest.raises(ValueError, match="CUDA"):
        binding.pa_decode_window(q, kc, kc, bt, cl, 0.1, out, window=4)
    with pytest.raises(ValueError, match="CUDA"):
        binding.pa_prefill_window(q, cl, 2, kc, kc, bt, cl, 0.1, out, window=None)
    k8 = torch.zeros((3, 2, 16, 64), dtype=torch.int8)
    s = torch.zeros((3, 2))
    with pytest.raises(TypeError):
        binding.pa_decode_i8(q.float(), k8, k8, s, s, bt, cl, 0.1, out)
    with pytest.raises(ValueError, match="CUDA"):
        binding.pa_cache_append_i8(q, q, cl, k8, k8, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        binding.pa_rope_append(q, q, q, cl, s, cl, out, kc, kc)
