"""The new calls together, as a layer of a serving engine uses them: chunked
prefill and decode steps over one cache (append with rotation, then windowed
or 8-bit attention), captured into graphs and replayed, on other streams, two
at once, with tensors aligned to 4 bytes only, and far into a large pool."""
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


class Layer:
    """One attention layer's cache (bf16 or 8-bit) and its calls."""

    def __init__(self, pa, gen, i8, B, pages, Hq, Hkv, D, window, sinks):
        self.pa, self.gen, self.i8 = pa, gen, i8
        self.B, self.Hq, self.Hkv, self.D, self.window, self.sinks = B, Hq, Hkv, D, window, sinks
        self.bt, nb = ref.tables(gen, [pages * 16] * B)
        if i8:
            self.cache = [t.cuda() for t in ref.fresh_i8(nb, Hkv, D, junk=gen)]
        else:
            self.cache = [torch.full((nb, Hkv, 16, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                          for _ in range(2)]
        self.cos_sin = ref.table(pages * 16, D).cuda()
        self.lens = [0] * B

    def step(self, chunks, decode):
        """Appends chunks[b] new tokens to sequence b, attends with their queries; returns (q rotated, out)."""
        pa, T = self.pa, sum(chunks)
        x = torch.randn((T, self.Hq + 2 * self.Hkv, self.D), generator=self.gen).bfloat16().cuda()
        q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
        positions, slots = [], []
        for b, c in enumerate(chunks):
            positions += range(self.lens[b], self.lens[b] + c)
            slots += ref.slots_of(self.bt, b, self.lens[b], self.lens[b] + c)
            self.lens[b] += c
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        q_rot = torch.empty((T, self.Hq, self.D), dtype=torch.bfloat16, device="cuda")
        append = pa.pa_rope_append_i8 if self.i8 else pa.pa_rope_append
        append(q, k, v, ints(positions), self.cos_sin, ints(slots), q_rot, *self.cache)
        out = torch.full_like(q_rot, float("nan"))
        tail = (self.bt.cuda(), ints(self.lens), self.D ** -0.5, out)
        kw = dict(window=self.window, sinks=self.sinks)
        if decode:
            (pa.pa_decode_i8 if self.i8 else pa.pa_decode_window)(q_rot, *self.cache, *tail, **kw)
        else:
            cu = ints([0] + torch.tensor(chunks).cumsum(0).tolist())
            (pa.pa_prefill_i8 if self.i8 else pa.pa_prefill_window)(q_rot, cu, max(chunks), *self.cache, *tail, **kw)
        return q_rot, out

    def check(self, chunks, q_rot, out, weight_error):
        """Attention over what the cache holds now, in 64 bits."""
        cache, row = [t.cpu() for t in self.cache], 0
        for b, (c, n) in enumerate(zip(chunks, self.lens)):
            if self.i8:
                k, v = ref.values_i8(*cache, self.bt[b], n)
            else:
                blocks = self.bt[b, : (n + 15) // 16].long()
                k, v = (t[blocks].permute(1, 0, 2, 3).reshape(self.Hkv, -1, self.D)[:, :n].double() for t in cache)
            want, mean_abs = ref.attend(q_rot[row:row + c].cpu(), k, v, self.D ** -0.5,
                                        ref.ALL if self.window is None else self.window, self.sinks)
            ref.assert_attention(out[row:row + c], want, mean_abs, weight_error)
            row += c


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,window,sinks", [(8, 2, 64, 40, 4), (8, 8, 128, 100, 0), (16, 4, 128, None, 0)])
def test_prefill_then_decode_steps(pa, i8, Hq, Hkv, D, window, sinks):
    g = torch.Generator().manual_seed(D + Hq)
    layer = Layer(pa, g, i8, 3, 12, Hq, Hkv, D, window, sinks)
    for chunks in ([50, 1, 17], [33, 70, 5]):
        q, out = layer.step(chunks, decode=False)
        layer.check(chunks, q, out, 2.0 ** -8)
    for _ in range(4):
        q, out = layer.step([1, 1, 1], decode=True)
        layer.check([1, 1, 1], q, out, 2.0 ** -11)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("i8", [False, True])
def test_step_in_a_graph(pa, i8):
    # one captured step (append, decode, multi-query call), replayed on new inputs, against eager calls
    g = torch.Generator().manual_seed(11)
    B, Hq, Hkv, D, pages = 3, 8, 2, 64, 9
    bt, nb = ref.tables(g, [pages * 16] * B)
    lens = [100, 37, 140]
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    positions = (cl - 1).contiguous()
    slots = torch.tensor([ref.slots_of(bt, b, n - 1, n)[0] for b, n in enumerate(lens)], dtype=torch.int32).cuda()
    cu = torch.arange(B + 1, dtype=torch.int32).cuda()
    cos_sin = ref.table(256, D).cuda()
    if i8:
        start = [t.cuda() for t in ref.fresh_i8(nb, Hkv, D, junk=g)]
    else:
        start = [torch.randn((nb, Hkv, 16, D), generator=g).bfloat16().cuda() for _ in range(2)]
    cache = [t.clone() for t in start]
    x = torch.empty((B, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    q_rot = torch.empty((B, Hq, D), dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty_like(q_rot) for _ in range(2)]
    ws = pa.alloc_workspace(pa.make_dims(q_rot, cache[0], bt))
    table = bt.cuda()

    def calls():
        append = pa.prepare_rope_append_i8 if i8 else pa.prepare_rope_append
        decode = pa.prepare_decode_i8 if i8 else pa.prepare_decode_window
        multi = pa.prepare_prefill_i8 if i8 else pa.prepare_prefill_window
        kw = dict(window=50, sinks=3)
        append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], positions, cos_sin, slots, q_rot, *cache)()
        decode(q_rot, *cache, table, cl, 0.125, outs[0], ws, **kw)()
        multi(q_rot, cu, 1, *cache, table, cl, 0.125, outs[1], **kw)()

    inputs = [torch.randn(x.shape, generator=g).bfloat16().cuda() * s for s in (1.0, 3.0, 0.5)]
    eager = []
    for inp in inputs:
        for c, s in zip(cache, start):
            c.copy_(s)
        x.copy_(inp)
        calls()
        eager.append([t.clone() for t in (*outs, q_rot, *cache)])
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()  # loads everything before the capture
    side.synchronize()
    with torch.cuda.graph(graph):
        calls()
    for inp, want in zip(inputs, eager):
        for c, s in zip(cache, start):
            c.copy_(s)
        x.copy_(inp)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((*outs, q_rot, *cache), want):
            assert torch.equal(got, w), "a replay differs from the eager calls"
    assert pa.pa_device_errors(clear=True) == 0


def test_two_decodes_at_once_on_other_streams(pa):
    # two streams, a workspace each, many calls in flight: nothing is shared between them
    g = torch.Generator().manual_seed(5)
    lens = [700, 3, 1500, 90]
    batch = ref.i8_batch(g, lens, 4, 128)
    k, v, ks, vs, bt = [t.cuda() for t in batch]
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [torch.randn((4, 16, 128), generator=g).bfloat16().cuda() for _ in range(2)]
    want = [torch.empty_like(q) for q in qs]
    for q, w in zip(qs, want):
        pa.pa_decode_i8(q, k, v, ks, vs, bt, cl, 0.09, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(10)] for q in qs]
    spaces = [pa.alloc_workspace(pa.make_dims(q, k, bt)) for q in qs]
    torch.cuda.synchronize()
    for i in range(10):
        for s, q, o, ws in zip(streams, qs, outs, spaces):
            pa.pa_decode_i8(q, k, v, ks, vs, bt, cl, 0.09, o[i], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)
    assert pa.pa_device_errors(clear=True) == 0


def test_append_then_attend_back_to_back(pa):
    # each kernel may start while the one before it ends: it must still see that one's writes
    g = torch.Generator().manual_seed(6)
    B, Hq, Hkv, D, n = 64, 8, 8, 64, 33
    bt, nb = ref.tables(g, [48] * B)
    cache = [t.cuda() for t in ref.fresh_i8(nb, Hkv, D)]
    ws = None
    for step in range(20):
        rows = torch.randn((B * n, Hkv, D), generator=g).bfloat16().cuda()
        slots = torch.tensor([s for b in range(B) for s in ref.slots_of(bt, b, 0, n)], dtype=torch.int32).cuda()
        q = torch.randn((B, Hq, D), generator=g).bfloat16().cuda()
        cl, table = torch.full((B,), n, dtype=torch.int32, device="cuda"), bt.cuda()
        out, again = torch.empty_like(q), torch.empty_like(q)
        if ws is None:
            ws = pa.alloc_workspace(pa.make_dims(q, cache[0], bt))
        torch.cuda.synchronize()
        pa.pa_cache_append_i8(rows, rows, slots, *cache)
        pa.pa_decode_i8(q, *cache, table, cl, 0.125, out, workspace=ws)
        torch.cuda.synchronize()
        pa.pa_decode_i8(q, *cache, table, cl, 0.125, again, workspace=ws)
        assert torch.equal(out, again), f"step {step}: the decode ran ahead of the append"


def test_tensors_aligned_to_four_bytes(pa):
    # scales, tables, lengths and slots need 4-byte alignment only
    g = torch.Generator().manual_seed(7)
    lens = [100, 17]
    k, v, ks, vs, bt = ref.i8_batch(g, lens, 8, 64)

    def off(t):  # the same values, one element into an allocation
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.reshape(-1).cuda()
        return flat[1:].view(t.shape)
    q = torch.randn((2, 16, 64), generator=g).bfloat16()
    cl = torch.tensor(lens, dtype=torch.int32)
    out = torch.empty_like(q).cuda()
    pa.pa_decode_i8(q.cuda(), k.cuda(), v.cuda(), off(ks), off(vs), off(bt), off(cl), 0.125, out)
    for b, n in enumerate(lens):
        want, mean_abs = ref.attend(q[b:b + 1], *ref.values_i8(k, v, ks, vs, bt[b], n), 0.125, ref.ALL, 0)
        ref.assert_attention(out[b:b + 1], want, mean_abs, 2.0 ** -11)
    caches = ref.fresh_i8(8, 8, 64, junk=g)
    gpu = [caches[0].cuda(), caches[1].cuda(), off(caches[2]), off(caches[3])]
    rows = torch.randn((61, 8, 64), generator=g).bfloat16()
    slots = torch.randperm(128, generator=g)[:61].to(torch.int32)
    pa.pa_cache_append_i8(rows.cuda(), rows.cuda(), off(slots), *gpu)
    ref.append_i8(rows.float(), rows.float(), slots.tolist(), caches)
    for a, b in zip(gpu, caches):
        assert torch.equal(a.cpu(), b)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("i8", [False, True])
def test_far_into_a_large_pool(pa, i8):
    # byte offsets past 2^32, blocks at both ends of the pool
    g = torch.Generator().manual_seed(8)
    Hkv, D, NB = 8, 128, 300_000 if i8 else 150_000
    n, Hq = 40, 8
    ends = [NB - 1, 0, NB - 2]
    bt = torch.tensor([ends], dtype=torch.int32).cuda()
    if i8:
        cache = [torch.empty((NB, Hkv, 16, D), dtype=torch.int8, device="cuda"),
                 torch.empty((NB, Hkv, D, 16), dtype=torch.int8, device="cuda"),
                 torch.empty((NB, Hkv), device="cuda"), torch.empty((NB, Hkv), device="cuda")]
    else:
        cache = [torch.empty((NB, Hkv, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x = torch.randn((n, Hq + 2 * Hkv, D), generator=g).bfloat16().cuda()
    slots = torch.tensor(ref.slots_of(bt.cpu(), 0, 0, n), dtype=torch.int32).cuda()
    q_rot = torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(n, dtype=torch.int32).cuda()
    append = pa.pa_rope_append_i8 if i8 else pa.pa_rope_append
    append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos, ref.table(64, D).cuda(), slots, q_rot, *cache)
    small = [t[ends].cpu() for t in cache]
    here = torch.arange(3)
    if i8:
        k, v = ref.values_i8(*small, here, n)
    else:
        k, v = (t.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n].double() for t in small)
    cl = torch.tensor([n], dtype=torch.int32).cuda()
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    out, last = torch.empty_like(q_rot), torch.empty_like(q_rot[:1])
    multi = pa.pa_prefill_i8 if i8 else pa.pa_prefill_window
    decode = pa.pa_decode_i8 if i8 else pa.pa_decode_window
    multi(q_rot, cu, n, *cache, bt, cl, 0.09, out, window=30, sinks=2)
    decode(q_rot[-1:].contiguous(), *cache, bt, cl, 0.09, last, window=30, sinks=2)
    want, mean_abs = ref.attend(q_rot.cpu(), k, v, 0.09, 30, 2)
    ref.assert_attention(out, want, mean_abs, 2.0 ** -8)
    ref.assert_attention(last, want[-1:], mean_abs[-1:], 2.0 ** -11)
    assert pa.pa_device_errors(clear=True) == 0


def test_wrong_device_and_shapes_are_refused(pa):
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    k8 = torch.zeros((3, 2, 16, 64), dtype=torch.int8, device="cuda")
    v8 = torch.zeros((3, 2, 64, 16), dtype=torch.int8, device="cuda")
    s = torch.zeros((3, 2), device="cuda")
    bt, cl = torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    with pytest.raises(ValueError):
        pa.pa_decode_i8(q, k8, k8, s, s, bt, cl, 0.1, out)              # v not transposed
    with pytest.raises(ValueError):
        pa.pa_decode_i8(q, k8, v8, s[0], s, bt, cl, 0.1, out)           # one scale per head
    with pytest.raises(ValueError):
        pa.pa_decode_i8(q[:1], k8, v8, s, s, bt, cl, 0.1, out[:1])      # fewer queries than sequences
    with pytest.raises(ValueError):
        pa.pa_prefill_i8(q, cl, 2, k8, v8, s, s, bt, cl, 0.1, out)      # cu_q_lens one short
    with pytest.raises(ValueError):
        pa.pa_decode_window(q.transpose(0, 1), kc, kc, bt, cl, 0.1, out, window=4)
    with pytest.raises(pa.PaError) as e:
        pa.pa_decode_window(q, kc, kc, bt, cl, 0.1, out, window=4, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -5
    rows = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((4, 64), device="cuda")
    with pytest.raises(ValueError):
        pa.pa_rope_append(q, rows.transpose(1, 2).contiguous().transpose(1, 2), rows, cl, table, cl, out, kc, kc)
    with pytest.raises(ValueError):
        pa.pa_rope_append(q, rows, rows[:1], cl, table, cl, out, kc, kc)
    with pytest.raises(pa.PaError) as e:
        pa.pa_rope_append(q, rows, rows, cl, torch.zeros((4, 40), device="cuda"), cl, out, kc, kc)
    assert e.value.code == -3
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("B", [32, 33, 70])
def test_multi_query_many_sequences(pa, i8, B):
    # up to 32 sequences are taken from the longest on, more in their order; some bring nothing
    g = torch.Generator().manual_seed(B)
    Hq, Hkv, D = 4, 2, 64
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    chunks = [min(n, int(c)) for n, c in zip(lens, torch.randint(0, 60, (B,), generator=g))]
    lens[5] = lens[6] = lens[7] = 64  # equal lengths
    chunks[5], chunks[6], chunks[7] = 64, 0, 1
    if i8:
        k, v, ks, vs, bt = ref.i8_batch(g, lens, Hkv, D)
        cache, seqs = (k, v, ks, vs), [ref.values_i8(k, v, ks, vs, bt[b], n) for b, n in enumerate(lens)]
    else:
        keys, values, kp, vp, bt = ref.bf16_batch(g, lens, Hkv, D)
        cache, seqs = (kp, vp), [(a.double(), b.double()) for a, b in zip(keys, values)]
    q = torch.randn((sum(chunks), Hq, D), generator=g).bfloat16()
    cu = [0] + torch.tensor(chunks).cumsum(0).tolist()
    out = torch.full_like(q, float("nan")).cuda()
    call = pa.pa_prefill_i8 if i8 else pa.pa_prefill_window
    call(q.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), max(chunks), *[t.cuda() for t in cache], bt.cuda(),
         torch.tensor(lens, dtype=torch.int32).cuda(), 0.125, out, window=77, sinks=9)
    assert pa.pa_device_errors(clear=True) == 0
    for b in range(B):
        rows = slice(cu[b], cu[b + 1])
        want, mean_abs = ref.attend(q[rows], *seqs[b], 0.125, 77, 9)
        ref.assert_attention(out[rows], want, mean_abs, 2.0 ** -8)
