"""What the serving operators over the paged cache are measured on.

Six calls, in three sets that a serving step runs together:

  * attention with a sliding window and a few first tokens that stay visible
    (sinks), over the bf16 paged cache: one query token per sequence
    (``decode_window``) and the last tokens of each sequence
    (``prefill_window``);
  * attention over a paged cache held in 8-bit integers with one scale for
    each (block of 16 tokens, kv head), with or without a window: one query
    token per sequence (``decode_i8``) and the last tokens of each sequence
    (``prefill_i8``);
  * the step's append with the position rotation applied on the way, into
    the bf16 cache (``rope_append``) and into the 8-bit one
    (``rope_append_i8``).

``run`` computes them in plain torch (32-bit sums and products), or, with
``own``, through paged_kv_attention_36_b200.binding.
"""
import math
import random

import torch

own = False

BLOCK = 16  # tokens of a cache block
FULL = 0    # a case's window: 0 = the whole context

# order of the 16 tokens in a row of the transposed 8-bit V tile:
# token t sits at byte 4*((t % 8) / 2) + 2*(t / 8) + t % 2
V_BYTE = [4 * ((t % 8) // 2) + 2 * (t // 8) + t % 2 for t in range(BLOCK)]


def listed():
    return [
        # the smallest decode step of a few chats: latency alone counts
        dict(name="decode_window few short", op="decode_window", seqs=4, q_heads=8, kv_heads=2, head_dim=64,
             shortest=17, longest=257, one_long=0, window=64, sinks=4, lens_seed=1),
        # a full decode batch of a windowed layer: most of each context is out of the window
        dict(name="decode_window batch", op="decode_window", seqs=128, q_heads=32, kv_heads=8, head_dim=64,
             shortest=512, longest=4096, one_long=0, window=1024, sinks=4, lens_seed=2),
        # chunked prefill of a windowed layer, 512-token chunks behind long contexts
        dict(name="prefill_window chunks", op="prefill_window", seqs=16, q_heads=32, kv_heads=8, head_dim=64,
             chunk_lo=512, chunk_hi=512, past_lo=0, past_hi=3500, window=1024, sinks=4, lens_seed=3),
        # ragged chunks, odd window and sinks that end inside a block, wide heads
        dict(name="prefill_window ragged", op="prefill_window", seqs=13, q_heads=16, kv_heads=8, head_dim=128,
             chunk_lo=1, chunk_hi=700, past_lo=0, past_hi=5000, window=333, sinks=21, lens_seed=4),
        # the smallest decode step over the 8-bit cache
        dict(name="decode_i8 few short", op="decode_i8", seqs=4, q_heads=8, kv_heads=2, head_dim=64,
             shortest=1, longest=100, one_long=0, window=FULL, sinks=0, lens_seed=5),
        # a full decode batch over the 8-bit cache
        dict(name="decode_i8 batch", op="decode_i8", seqs=128, q_heads=32, kv_heads=8, head_dim=64,
             shortest=512, longest=4096, one_long=0, window=FULL, sinks=0, lens_seed=6),
        # one very long sequence among short ones: the split over a context
        dict(name="decode_i8 one long", op="decode_i8", seqs=64, q_heads=32, kv_heads=8, head_dim=128,
             shortest=1024, longest=1024, one_long=131072, window=FULL, sinks=0, lens_seed=7),
        # chunked prefill over the 8-bit cache
        dict(name="prefill_i8 chunks", op="prefill_i8", seqs=16, q_heads=32, kv_heads=8, head_dim=128,
             chunk_lo=512, chunk_hi=512, past_lo=0, past_hi=3500, window=FULL, sinks=0, lens_seed=8),
        # a decode step's append: one token per sequence, rows cut from a fused projection
        dict(name="rope_append step", op="rope_append", seqs=128, q_heads=32, kv_heads=8, head_dim=64,
             chunk_lo=1, chunk_hi=1, past_lo=511, past_hi=4095, rotary_dim=64, interleaved=False, lens_seed=9),
        # a prefill step's append: whole chunks
        dict(name="rope_append chunks", op="rope_append", seqs=16, q_heads=32, kv_heads=8, head_dim=128,
             chunk_lo=512, chunk_hi=512, past_lo=0, past_hi=3500, rotary_dim=128, interleaved=False, lens_seed=10),
        # the same step into the 8-bit cache: blocks grow by a row, scales with them
        dict(name="rope_append_i8 step", op="rope_append_i8", seqs=128, q_heads=32, kv_heads=8, head_dim=64,
             chunk_lo=1, chunk_hi=1, past_lo=511, past_hi=4095, rotary_dim=64, interleaved=False, lens_seed=11),
        # ragged chunks into the 8-bit cache, interleaved pairs over a part of the head
        dict(name="rope_append_i8 ragged", op="rope_append_i8", seqs=24, q_heads=32, kv_heads=8, head_dim=128,
             chunk_lo=1, chunk_hi=600, past_lo=0, past_hi=3500, rotary_dim=64, interleaved=True, lens_seed=12),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode_window", "prefill_window", "decode_i8", "prefill_i8", "rope_append", "rope_append_i8"])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 8])
    case = dict(op=op, q_heads=kv_heads * rng.choice([1, 2, 4, 4, 8]), kv_heads=kv_heads,
                head_dim=rng.choice([64, 128]), lens_seed=rng.randrange(1 << 30))
    if op.startswith("decode"):
        seqs = _spread(rng, 1, 200)
        longest = _spread(rng, 1, min(20000, 400000 // seqs))
        case.update(seqs=seqs, shortest=rng.randint(0, longest), longest=longest,
                    one_long=rng.choice([0, 0, _spread(rng, 1000, 100000)]))
    else:
        seqs = _spread(rng, 1, 24)
        chunk = _spread(rng, 1, min(1500, 6000 // seqs))
        case.update(seqs=seqs, chunk_lo=rng.randint(1, chunk), chunk_hi=chunk, past_lo=0,
                    past_hi=_spread(rng, 1, 4000))
    if op.startswith("rope"):
        case.update(rotary_dim=rng.choice([case["head_dim"], case["head_dim"], case["head_dim"] // 2, 32]),
                    interleaved=rng.random() < 0.5)
    else:
        windowed = op.endswith("window") or rng.random() < 0.25
        case.update(window=_spread(rng, 1, 4000) if windowed else FULL,
                    sinks=rng.choice([0, 1, 4, 16, rng.randint(0, 100)]) if windowed else 0)
    return case


# ---- sizes -------------------------------------------------------------------

def _lengths(case):
    """(query tokens, cached tokens with them) of each sequence."""
    r = random.Random(case["lens_seed"])
    if case["op"].startswith("decode"):
        lens = [r.randint(case["shortest"], case["longest"]) for _ in range(case["seqs"])]
        if case["one_long"]:
            lens[r.randrange(len(lens))] = case["one_long"]
        return [1] * len(lens), lens
    chunks = [r.randint(case["chunk_lo"], case["chunk_hi"]) for _ in range(case["seqs"])]
    return chunks, [c + r.randint(case["past_lo"], case["past_hi"]) for c in chunks]


def _seen(case, position):
    """How many cached tokens the query at `position` attends to."""
    if not case["window"]:
        return position + 1
    first = max(0, position + 1 - case["window"])
    return position + 1 - first + min(case["sinks"], first)


def work(case):
    """Bytes: the rows that some query sees once (codes and scales for the 8-bit cache), the queries and outputs
    once; for an append the new rows read and written once. Operations: the two products of attention over what each
    query sees; three for each rotated value."""
    chunks, lens = _lengths(case)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    tokens = sum(chunks)
    if case["op"].startswith("rope"):
        wide = 1 if case["op"].endswith("i8") else 2  # bytes of a cached value
        moved = tokens * d * (2 * hq * 2 + 2 * hkv * (2 + wide)) + tokens * (case["rotary_dim"] * 4 + 8)
        if wide == 1:
            blocks = sum((n - 1) // BLOCK - (n - c) // BLOCK + 1 for c, n in zip(chunks, lens))
            moved += blocks * hkv * 2 * 4
        return {"bytes": moved, "flops": 3 * tokens * (hq + hkv) * case["rotary_dim"]}
    rows = pairs = 0
    for c, n in zip(chunks, lens):
        if n == 0:
            continue
        first = max(0, n - c + 1 - case["window"]) if case["window"] else 0
        rows += n - first + min(case["sinks"], first)
        pairs += sum(_seen(case, p) for p in range(n - c, n))
    wide = 1 if case["op"].endswith("i8") else 2
    moved = rows * hkv * d * 2 * wide + 2 * tokens * hq * d * 2 + (rows // BLOCK) * 4
    if wide == 1:
        moved += rows // BLOCK * hkv * 2 * 4
    return {"bytes": moved, "flops": 4 * pairs * hq * d}


# ---- inputs ------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _tables(gen, pages, spare):
    """Block tables over a shuffled pool, entries past a sequence's pages far out of range."""
    total = sum(pages)
    pool = total + spare
    order = torch.randperm(pool, generator=gen, device="cuda")[:total].to(torch.int32)
    table = torch.full((len(pages), max(1, max(pages))), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


def _quantized(x):
    """x [blocks][heads][16][D] as 8-bit codes with a scale for each (block, head)."""
    top = x.abs().amax(dim=(2, 3))
    scale = top / torch.full_like(top, 127.0)
    return torch.round(x / scale[:, :, None, None]).to(torch.int8), scale


def _transposed(codes):
    """[blocks][heads][16][D] -> [blocks][heads][D][16] in the stored token order."""
    out = torch.empty(codes.shape[0], codes.shape[1], codes.shape[3], BLOCK, dtype=codes.dtype, device=codes.device)
    out[..., torch.tensor(V_BYTE, device=codes.device)] = codes.transpose(2, 3)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    chunks, lens = _lengths(case)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    tokens, i8 = sum(chunks), case["op"].endswith("i8")
    ints = dict(dtype=torch.int32, device="cuda")
    s = dict(case=dict(case), chunks=chunks, lens=lens)
    if case["op"].startswith("rope"):
        pages = [(n - 1) // BLOCK - (n - c) // BLOCK + 1 for c, n in zip(chunks, lens)]
    else:
        pages = [-(-n // BLOCK) for n in lens]
    table, pool = _tables(gen, pages, 8 + sum(pages) // 4)
    # keys have channels of their own size, values do not
    key_size = 0.5 + 1.5 * torch.rand((hkv, 1, d), generator=gen, device="cuda")
    k, v = _normal(gen, pool, hkv, BLOCK, d) * key_size, _normal(gen, pool, hkv, BLOCK, d)
    if i8:
        s["k_cache"], s["k_scale"] = _quantized(k)
        codes, s["v_scale"] = _quantized(v)
        s["v_cache"] = _transposed(codes)
    else:
        s["k_cache"], s["v_cache"] = k.bfloat16(), v.bfloat16()
    del k, v
    if case["op"].startswith("rope"):
        # q, k and v rows as slices of one projection's output
        fused = _normal(gen, tokens, hq + 2 * hkv, d).bfloat16()
        s["q"], s["k_new"], s["v_new"] = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
        at = torch.cat([torch.arange(n - c, n, **ints) for c, n in zip(chunks, lens)])
        page = torch.cat([torch.arange(n - c, n, **ints) // BLOCK - (n - c) // BLOCK for c, n in zip(chunks, lens)])
        seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(chunks, device="cuda"))
        s["positions"] = at
        s["slots"] = table[seq, page.long()] * BLOCK + at % BLOCK
        rd = case["rotary_dim"]
        turn = torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None] * \
            500000.0 ** (-torch.arange(0, rd, 2, device="cuda", dtype=torch.float64) / rd)
        s["cos_sin"] = torch.cat([turn.cos(), turn.sin()], dim=1).float()
        s["q_out"] = torch.empty(tokens, hq, d, dtype=torch.bfloat16, device="cuda")
        if i8:  # the values that the caches stand for, read back after the append
            s["k_value"] = torch.empty(s["k_cache"].shape, dtype=torch.bfloat16, device="cuda")
            s["v_value"] = torch.empty(s["v_cache"].shape, dtype=torch.bfloat16, device="cuda")
    else:
        s["q"] = _normal(gen, tokens, hq, d).bfloat16()
        s["out"] = torch.empty_like(s["q"])
        s["tables"], s["context"] = table, torch.tensor(lens, **ints)
        starts = [0]
        for c in chunks:
            starts.append(starts[-1] + c)
        s["starts"] = torch.tensor(starts, **ints)
        s["scale"] = d ** -0.5
    if own:
        s["call"] = _bind(s)
    return s


def _bind(s):
    """The framework's call with its arguments bound once, as a serving loop keeps it."""
    from paged_kv_attention_36_b200 import binding as pa
    case, op = s["case"], s["case"]["op"]
    caches = (s["k_cache"], s["v_cache"]) + ((s["k_scale"], s["v_scale"]) if op.endswith("i8") else ())
    if op.startswith("rope"):
        bind = pa.prepare_rope_append_i8 if op.endswith("i8") else pa.prepare_rope_append
        return bind(s["q"], s["k_new"], s["v_new"], s["positions"], s["cos_sin"], s["slots"], s["q_out"], *caches,
                    interleaved=case["interleaved"])
    window = case["window"] if case["window"] else pa.PA_WINDOW_ALL
    if op.startswith("decode"):
        bind = pa.prepare_decode_i8 if op.endswith("i8") else pa.prepare_decode_window
        return bind(s["q"], *caches, s["tables"], s["context"], s["scale"], s["out"],
                    pa.alloc_workspace(pa.make_dims(s["q"], s["k_cache"], s["tables"])), window=window,
                    sinks=case["sinks"])
    bind = pa.prepare_prefill_i8 if op.endswith("i8") else pa.prepare_prefill_window
    return bind(s["q"], s["starts"], max(s["chunks"]), *caches, s["tables"], s["context"], s["scale"], s["out"],
                window=window, sinks=case["sinks"])


# ---- the plain forms ---------------------------------------------------------

def _visible(case, key, query):
    """Which of the positions `key` the positions `query` attend to (both broadcast)."""
    see = key <= query
    if case["window"]:
        see = see & ((key > query - case["window"]) | (key < case["sinks"]))
    return see


def _blocks(s, block, which):
    """Cached blocks [n][heads][16][D] in 32 bits."""
    rows = s[which + "_cache"][block]
    if "k_scale" not in s:
        return rows.float()
    if which == "v":
        rows = rows.transpose(2, 3)[:, :, torch.tensor(V_BYTE, device="cuda")]
    return rows.float() * s[which + "_scale"][block][:, :, None, None]


def _plain_decode(s):
    """Every block of every context in one list: scores, a softmax by sequence, weighted sums added by sequence."""
    case = s["case"]
    hkv, d = case["kv_heads"], case["head_dim"]
    b, g = case["seqs"], case["q_heads"] // hkv
    context = s["context"].long()
    count = (context + BLOCK - 1) // BLOCK
    total = sum(-(-n // BLOCK) for n in s["lens"])
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), count, output_size=total)
    page = torch.arange(total, device="cuda") - (torch.cumsum(count, 0) - count)[seq]
    see = _visible(case, page[:, None] * BLOCK + torch.arange(BLOCK, device="cuda"), context[seq][:, None] - 1)
    if case["window"]:
        some = see.any(1)
        seq, page, see = seq[some], page[some], see[some]
    block = s["tables"][seq, page].long()
    q = s["q"].float().view(b, hkv, g, d)
    score = (q[seq] @ _blocks(s, block, "k").transpose(2, 3)) * s["scale"]  # [blocks][hkv][g][16]
    score = score.masked_fill(~see[:, None, None], -math.inf)
    top = torch.full((b, hkv, g), -math.inf, device="cuda")
    top.scatter_reduce_(0, seq[:, None, None].expand(-1, hkv, g), score.amax(-1), "amax")
    weight = torch.exp(score - top[seq][..., None])
    norm = torch.zeros((b, hkv, g), device="cuda").index_add_(0, seq, weight.sum(-1))
    out = torch.zeros((b, hkv, g, d), device="cuda").index_add_(0, seq, weight @ _blocks(s, block, "v"))
    return torch.where(norm[..., None] > 0, out / norm[..., None], 0.0).view(b, hkv * g, d).bfloat16()


def _plain_prefill(s):
    """Padded batches: scores of all queries with all cached tokens, masked, a softmax, weighted sums."""
    case = s["case"]
    hkv, d = case["kv_heads"], case["head_dim"]
    b, g = case["seqs"], case["q_heads"] // hkv
    most = max(s["chunks"])
    starts, context = s["starts"].long(), s["context"].long()
    chunk = starts[1:] - starts[:-1]
    page = torch.arange(s["tables"].shape[1], device="cuda")
    longest = page.numel() * BLOCK
    pos = torch.arange(longest, device="cuda")
    block = torch.where(page * BLOCK < context[:, None], s["tables"], 0).long().reshape(-1)
    k = _blocks(s, block, "k").view(b, -1, hkv, BLOCK, d).transpose(1, 2).reshape(b, hkv, longest, d)
    v = _blocks(s, block, "v").view(b, -1, hkv, BLOCK, d).transpose(1, 2).reshape(b, hkv, longest, d)
    i = torch.arange(most, device="cuda")
    row = torch.minimum(starts[:-1, None] + i, starts[1:, None] - 1)
    q = s["q"][row].float().view(b, most, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * most, d)
    see = _visible(case, pos[None, None, :], (context - chunk)[:, None, None] + i[None, :, None])
    score = (q @ k.transpose(2, 3)).view(b, hkv, g, most, longest) * s["scale"]
    score = score.masked_fill(~see[:, None, None], -math.inf)
    weight = torch.exp(score - score.amax(-1, keepdim=True))
    out = (weight.view(b, hkv, g * most, longest) @ v).view(b, hkv, g, most, d) / weight.sum(-1, keepdim=True)
    out = out.permute(0, 3, 1, 2, 4).reshape(b, most, hkv * g, d).bfloat16()
    tokens = s["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), chunk, output_size=tokens)
    return out[seq, torch.arange(tokens, device="cuda") - starts[seq]]


def _rotated(s, x):
    """x [T][heads][D] in 32 bits, its first rotary_dim values turned by the angles of the tokens' positions."""
    case = s["case"]
    rd = case["rotary_dim"]
    turn = s["cos_sin"][s["positions"].long()][:, None, :]
    c, sn = turn[..., :rd // 2], turn[..., rd // 2:]
    x = x.float()
    if case["interleaved"]:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        y = torch.cat([a * c - b * sn, b * c + a * sn], dim=-1)
    return torch.cat([y, x[..., rd:]], dim=-1)


def _plain_rope(s):
    block, offset = s["slots"].long() // BLOCK, s["slots"].long() % BLOCK
    s["q_out"].copy_(_rotated(s, s["q"]))
    s["k_cache"][block, :, offset] = _rotated(s, s["k_new"]).bfloat16()
    s["v_cache"][block, :, offset] = s["v_new"]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_requantize(rows, codes, scale, block, byte_of, offset):
    """rows [T][heads][D] into codes (a view [blocks][heads][16][D]): a block whose first row is written starts
    anew; one whose new rows pass 127 scales takes a larger scale and its old codes are rounded again."""
    top = torch.zeros_like(scale).scatter_reduce_(0, block[:, None].expand(-1, rows.shape[1]), rows.abs().amax(-1),
                                                  "amax")
    new = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda")
    new[block[offset == 0]] = True
    old = torch.where(new[:, None], 0.0, scale)
    now = torch.maximum(old, top / torch.full_like(top, 127.0))
    grown = now > old
    touched = torch.unique(block)
    at = codes[touched].float()
    again = torch.round(at * old[touched][:, :, None, None] / now[touched][:, :, None, None])
    codes[touched] = torch.where(grown[touched][:, :, None, None], again, at).to(torch.int8)
    scale.copy_(now)
    step = now[block][:, :, None]
    codes[block, :, byte_of] = torch.where(step > 0, torch.round(rows / step), 0.0).to(torch.int8)


def _plain_rope_i8(s):
    block, offset = s["slots"].long() // BLOCK, s["slots"].long() % BLOCK
    s["q_out"].copy_(_rotated(s, s["q"]))
    _plain_requantize(_rotated(s, s["k_new"]), s["k_cache"], s["k_scale"], block, offset, offset)
    byte = torch.tensor(V_BYTE, device="cuda")[offset]
    _plain_requantize(s["v_new"].float(), s["v_cache"].transpose(2, 3), s["v_scale"], block, byte, offset)


def _values(s):
    """What the 8-bit caches stand for, in their stored order."""
    torch.mul(s["k_cache"], s["k_scale"][:, :, None, None], out=s["k_value"])
    torch.mul(s["v_cache"], s["v_scale"][:, :, None, None], out=s["v_value"])
    return s["q_out"], s["k_value"], s["v_value"]


def run(state):
    op = state["case"]["op"]
    if own:
        state["call"]()
        if op == "rope_append":
            return state["q_out"], state["k_cache"], state["v_cache"]
        return _values(state) if op == "rope_append_i8" else state["out"]
    if op == "rope_append":
        return _plain_rope(state)
    if op == "rope_append_i8":
        _plain_rope_i8(state)
        return _values(state)
    return _plain_decode(state) if op.startswith("decode") else _plain_prefill(state)


# ---- the definition in 64 bits -------------------------------------------------

def _exact_attention(case, s):
    """Sequence by sequence from the definition: softmax over the tokens that each query sees."""
    hkv, g = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    order = torch.argsort(torch.tensor(V_BYTE, device="cuda"))  # token at each stored byte
    for b, (c, n) in enumerate(zip(s["chunks"], s["lens"])):
        if n:
            blocks = s["tables"][b, : (n + BLOCK - 1) // BLOCK].long()
            k, v = s["k_cache"][blocks].double(), s["v_cache"][blocks].double()
            if "k_scale" in s:
                k = k * s["k_scale"][blocks].double()[..., None, None]
                v = v * s["v_scale"][blocks].double()[..., None, None]
                by_token = torch.empty_like(v)
                by_token[..., order] = v
                v = by_token.transpose(2, 3)
            k = k.permute(1, 0, 2, 3).reshape(hkv, -1, k.shape[-1])[:, :n]
            v = v.permute(1, 0, 2, 3).reshape(hkv, -1, v.shape[-1])[:, :n]
            query = s["q"][row:row + c].double().reshape(c, hkv, g, -1)
            last = torch.arange(n - c, n, device="cuda")[:, None]
            token = torch.arange(n, device="cuda")[None, :]
            hidden = token > last
            if case["window"]:
                hidden |= (last - token >= case["window"]) & (token >= case["sinks"])
            for h in range(hkv):
                z = torch.einsum("cgd,td->gct", query[:, h], k[h]) * s["scale"]
                p = torch.softmax(z.masked_fill(hidden, -math.inf), dim=-1)
                out[row:row + c, h * g:(h + 1) * g] = torch.einsum("gct,td->cgd", p, v[h])
        row += c
    return out


def _exact_turn(case, s, x):
    """Pairs as complex numbers, multiplied by e^(i angle) of the table."""
    rd = case["rotary_dim"]
    at = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(at[:, :rd // 2], at[:, rd // 2:])[:, None]
    x = x.double().clone()
    pair = (slice(0, rd, 2), slice(1, rd, 2)) if case["interleaved"] else (slice(0, rd // 2), slice(rd // 2, rd))
    z = torch.complex(x[..., pair[0]].contiguous(), x[..., pair[1]].contiguous()) * turn
    x[..., pair[0]], x[..., pair[1]] = z.real, z.imag
    return x


def _exact_append(case, s):
    q, k, v = _exact_turn(case, s, s["q"]), _exact_turn(case, s, s["k_new"]), s["v_new"].double()
    slots = s["slots"].tolist()
    if case["op"] == "rope_append":
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        block = torch.tensor([x // BLOCK for x in slots], device="cuda")
        offset = torch.tensor([x % BLOCK for x in slots], device="cuda")
        k_cache[block, :, offset] = k
        v_cache[block, :, offset] = v
        return q, k_cache, v_cache
    # the 8-bit values depend on every earlier rounding: they have no value of their own in 64 bits
    return q, None, None


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    return _exact_append(case, s) if case["op"].startswith("rope") else _exact_attention(case, s)
