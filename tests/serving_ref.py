"""Test-side definitions, in 64 bits, of windowed attention, the 8-bit
block-scaled cache and the append with rotation, and random paged batches
for them.  Plain torch on the CPU, sequence by sequence."""
from __future__ import annotations

import math

import torch

from tests import paging

PAD_BLOCK = paging.PAD_BLOCK
ALL = 0x7FFFFFFF  # a window that holds every token


def v_byte(t: int) -> int:
    """Byte of token t in a row of the transposed 8-bit V tile (include/pa.h)."""
    return 4 * ((t % 8) // 2) + 2 * (t // 8) + t % 2


V_BYTES = [v_byte(t) for t in range(16)]


def visible(L: int, p: int, window: int, sinks: int) -> torch.Tensor:
    """[L] bools: the cached tokens a query at position p attends to."""
    t = torch.arange(L)
    return (t <= p) & ((t > p - window) | (t < sinks))


def attend(q, keys, values, scale, window, sinks):
    """The last q.shape[0] tokens' attention over keys/values [Hkv][L][D]
    (64 bits), and the weighted mean of |V| that a relative error of the
    weights multiplies.  Rows that see a token whose K or V is not finite
    come out as the arithmetic has them; unseen tokens never count."""
    n, Hq, D = q.shape
    Hkv, L, _ = keys.shape
    G = Hq // Hkv
    out = torch.zeros((n, Hq, D), dtype=torch.float64)
    mean_abs = torch.zeros((n, Hq, D), dtype=torch.float64)
    for i in range(n):
        see = visible(L, L - n + i, window, sinks)
        if not see.any():
            continue
        k, v = keys[:, see], values[:, see]
        s = torch.einsum("gjd,gtd->gjt", q[i].double().view(Hkv, G, D), k) * scale
        w = torch.exp(s - s.amax(-1, keepdim=True))
        w = w / w.sum(-1, keepdim=True)
        out[i] = torch.einsum("gjt,gtd->gjd", w, v).reshape(Hq, D)
        mean_abs[i] = torch.einsum("gjt,gtd->gjd", w, v.abs()).reshape(Hq, D)
    return out, mean_abs


def assert_attention(got, ref, mean_abs, weight_error):
    """|got - ref| <= 2^-8 |ref| (the output's rounding to bf16) + (weight_error
    + 2^-12) * mean |V|: the softmax weights' rounding, and 2^-12 for logits
    and sums in 32 bits (a logit is off by at most D * 2^-24 * |s| < 2^-13
    here, which moves a weight by as much, and its sum once more)."""
    got = got.double().cpu()
    assert torch.isfinite(got).all(), "output not finite"
    tol = 2.0 ** -8 * ref.abs() + (weight_error + 2.0 ** -12) * mean_abs + 1e-30
    err = (got - ref).abs()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.2f} times its bound"


# ---- 8-bit caches -------------------------------------------------------------

def fresh_i8(num_blocks, Hkv, D, junk=None):
    """Caches and scales (CPU); `junk`: a generator that fills them with noise."""
    k = torch.zeros((num_blocks, Hkv, 16, D), dtype=torch.int8)
    v = torch.zeros((num_blocks, Hkv, D, 16), dtype=torch.int8)
    ks, vs = torch.zeros((num_blocks, Hkv)), torch.zeros((num_blocks, Hkv))
    if junk is not None:
        k.random_(-127, 128, generator=junk)
        v.random_(-127, 128, generator=junk)
        ks.uniform_(0, 4, generator=junk)
        vs.uniform_(0, 4, generator=junk)
    return k, v, ks, vs


def append_i8(k_rows, v_rows, slots, caches):
    """The definition, block by block, in the 32-bit operations it names:
    k_rows, v_rows [T][Hkv][D] float32, slots a list; caches updated in place."""
    k_cache, v_cache, k_scale, v_scale = caches
    last = {}
    for t, s in enumerate(slots):
        if 0 <= s < k_cache.shape[0] * 16:
            last[s] = t  # of two tokens with one slot the later lands
    by_block = {}
    for s, t in last.items():
        by_block.setdefault(s // 16, {})[s % 16] = t
    for blk, rows in by_block.items():
        for g in range(k_cache.shape[1]):
            for is_v, src, tile, scale in ((False, k_rows, k_cache[blk, g], k_scale),
                                           (True, v_rows, v_cache[blk, g].t()[V_BYTES], v_scale)):
                offs = sorted(rows)
                x = torch.stack([src[rows[o], g] for o in offs])
                old = torch.tensor(0.0) if 0 in rows else scale[blk, g].clone()
                need = x.abs().max() / torch.tensor(127.0)
                now = torch.maximum(old, need)
                codes = tile.clone()
                if 0 in rows:
                    codes.zero_()
                elif now > old:
                    codes = torch.round(codes.float() * old / now).to(torch.int8)
                new = torch.round(x / now) if now > 0 else torch.zeros_like(x)
                codes[offs] = new.to(torch.int8)
                scale[blk, g] = now
                if is_v:
                    v_cache[blk, g][:, V_BYTES] = codes.t()
                else:
                    k_cache[blk, g] = codes


def values_i8(k, v, ks, vs, blocks, L):
    """[Hkv][L][D] keys and values (64 bits) of a sequence's blocks."""
    blocks = blocks[: (L + 15) // 16].long()
    kk = k[blocks].double() * ks[blocks].double()[..., None, None]
    vv = v[blocks][..., V_BYTES].transpose(2, 3).double() * vs[blocks].double()[..., None, None]

    def rows(x):
        return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :L]
    return rows(kk), rows(vv)


# ---- rotation -----------------------------------------------------------------

def table(max_position, rotary_dim, base=10000.0):
    """cos_sin [max_position][rotary_dim] fp32, from angles in 64 bits."""
    a = torch.arange(max_position, dtype=torch.float64)[:, None] * \
        base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / max(rotary_dim, 1))
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(x, cos_sin, positions, interleaved):
    """x [T][heads][D] turned, in x's own precision (one rounding per operation)."""
    rd = cos_sin.shape[1]
    at = cos_sin.to(x.dtype)[positions.long()][:, None]
    c, s = at[..., : rd // 2], at[..., rd // 2:]
    y = x.clone()
    lo = slice(0, rd, 2) if interleaved else slice(0, rd // 2)
    hi = slice(1, rd, 2) if interleaved else slice(rd // 2, rd)
    a, b = x[..., lo], x[..., hi]
    y[..., lo] = a * c - b * s
    y[..., hi] = b * c + a * s
    return y


# ---- paged batches --------------------------------------------------------------

def bf16_batch(gen, lens, Hkv, D, spare=3):
    """K and V of each sequence [Hkv][L][D] bf16, their NaN-poisoned pools and the block tables."""
    ks, vs = paging.random_seqs(gen, lens, Hkv, D), paging.random_seqs(gen, lens, Hkv, D)
    nb = sum((n + 15) // 16 for n in lens) + spare
    (kp, vp), bt = paging.page([ks, vs], lens, 16, nb, gen, poison=True)
    return ks, vs, kp, vp, bt


def tables(gen, lens, spare=3):
    """Shuffled block tables, padded with an id that must not be read; and the pool size."""
    pages = [(n + 15) // 16 for n in lens]
    nb = sum(pages) + spare
    order = torch.randperm(nb, generator=gen).to(torch.int32)
    bt = torch.full((len(lens), max(1, max(pages, default=0))), PAD_BLOCK, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = order[at: at + n]
        at += n
    return bt, nb


def slots_of(bt, b, start, stop):
    return [int(bt[b, t // 16]) * 16 + t % 16 for t in range(start, stop)]


def i8_batch(gen, lens, Hkv, D):
    """Random 8-bit pools, unread parts full of noise with scales of NaN."""
    bt, nb = tables(gen, lens)
    k, v, ks, vs = fresh_i8(nb, Hkv, D, junk=gen)
    ks = 0.002 + 0.02 * torch.rand(ks.shape, generator=gen)
    vs = 0.002 + 0.02 * torch.rand(vs.shape, generator=gen)
    used = torch.zeros(nb, dtype=torch.bool)
    for b, n in enumerate(lens):
        used[bt[b, : (n + 15) // 16].long()] = True
    ks[~used] = math.nan
    vs[~used] = math.nan
    return k, v, ks, vs, bt
