"""fp64 CPU definitions of the decode-step operators around the pre-projection.

TEST INFRASTRUCTURE ONLY, like dsnq_oracle.py: plain and slow, sharing no code
with the CUDA path.  bf16 values come in as uint16 bit patterns and results go
out in fp64, unrounded.
"""

from __future__ import annotations

import numpy as np

__all__ = ["decode_bf16", "extend_block_tables", "rope_rotate", "head_rmsnorm_rope", "latent_rows",
           "paged_latent_attention"]


def decode_bf16(bits) -> np.ndarray:
    """The values of bf16 bit patterns."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def extend_block_tables(seq_lens, new_tokens, free_pages, table, page_size, rows):
    """Request by request, token by token.  Returns (new_lens, row_starts,
    positions, slots, (pages taken, pages wanted), table)."""
    table = np.array(table, np.int64)
    B, width = table.shape
    cap = width * page_size
    free = [int(x) for x in free_pages]
    positions, slots = np.zeros(rows, np.int64), np.full(rows, -1, np.int64)
    new_lens, starts = [], []
    row = taken = wanted = 0
    for b in range(B):
        old = min(max(int(seq_lens[b]), 0), cap)
        n = 1 if new_tokens is None else max(int(new_tokens[b]), 0)
        starts.append(min(row, rows))
        length = old
        full = False
        for j in range(n):
            pos, r = old + j, row + j
            if r < rows:
                positions[r] = pos
            if r >= rows or pos >= cap:
                continue
            if pos % page_size == 0 or (j == 0 and pos // page_size >= -(-old // page_size)):
                # The token opens a page.
                wanted += 1
                if taken < len(free):
                    table[b, pos // page_size] = free[taken]
                    taken += 1
                else:
                    full = True
            if full:
                continue
            length = pos + 1
            page = table[b, pos // page_size]
            if page >= 0:
                slots[r] = page * page_size + pos % page_size
        new_lens.append(length)
        row += n
    starts.append(min(row, rows))
    return (np.array(new_lens, np.int64), np.array(starts, np.int64), positions, slots,
            np.array([taken, wanted], np.int64), table)


def _inverse_turn(bits):
    """floor(2^bits / (2 pi)), from Machin's pi = 16 atan(1/5) - 4 atan(1/239)."""
    one = 1 << (2 * bits)

    def atan_inverse(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    return (one << bits) // (2 * (16 * atan_inverse(5) - 4 * atan_inverse(239)))


_TURN_BITS = 1300                        # beyond the exponents of fp64 frequencies and positions
_PER_TURN = _inverse_turn(_TURN_BITS)


def _angle(position, freq):
    """position * freq modulo one turn: the exact product's fraction of a turn
    (Python integers), rounded to fp64 once."""
    num, den = float(freq).as_integer_ratio()
    scale = den << _TURN_BITS
    return int(position) * num * _PER_TURN % scale / scale * (2.0 * np.pi)


def rope_rotate(x, positions, inv_freq, layout, scale=1.0, inverse=False):
    """x [..., tokens on axis 0, ..., R] with its pairs rotated, fp64."""
    x = np.asarray(x, np.float64)
    ang = np.array([[_angle(p, f) for f in inv_freq] for p in positions]).reshape(len(positions), len(inv_freq))
    c, s = np.cos(ang) * scale, np.sin(ang) * scale * (-1.0 if inverse else 1.0)
    shape = (len(positions),) + (1,) * (x.ndim - 2) + (len(inv_freq),)
    c, s = c.reshape(shape), s.reshape(shape)
    out = np.empty_like(x)
    if layout == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        out[..., 0::2], out[..., 1::2] = a * c - b * s, b * c + a * s
    else:
        h = x.shape[-1] // 2
        a, b = x[..., :h], x[..., h:]
        out[..., :h], out[..., h:] = a * c - b * s, b * c + a * s
    return out


def head_rmsnorm_rope(x, positions, inv_freq, gamma=None, eps=1e-6, normalize=True, rope_offset=0, layout="interleaved",
                      rope_scale=1.0, inverse=False):
    """x [M, H, D] fp64 -> fp64, unrounded."""
    x = np.array(x, np.float64)
    if normalize:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if gamma is not None:
            x = x * np.asarray(gamma, np.float64)
    lo, hi = rope_offset, rope_offset + 2 * len(inv_freq)
    if hi > lo:
        x[..., lo:hi] = rope_rotate(x[..., lo:hi], positions, inv_freq, layout, rope_scale, inverse)
    return x


def latent_rows(kv, pe, positions, inv_freq, gamma=None, eps=1e-6, normalize=False, rope_offset=0, layout="interleaved",
                rope_scale=1.0):
    """The rows [kv | pe] as they go into the cache, fp64."""
    kv = np.array(kv, np.float64)
    if normalize:
        kv = kv / np.sqrt((kv * kv).mean(-1, keepdims=True) + eps)
        if gamma is not None:
            kv = kv * np.asarray(gamma, np.float64)
    row = kv if pe is None else np.concatenate([kv, np.asarray(pe, np.float64)], -1)
    lo, hi = rope_offset, rope_offset + 2 * len(inv_freq)
    if hi > lo:
        row[:, lo:hi] = rope_rotate(row[:, lo:hi], positions, inv_freq, layout, rope_scale)
    return row


def paged_latent_attention(q, cache, table, lens, v_dim, scale):
    """q [B,H,DK], cache [pages, page, DK] (fp64).  Returns (out, lse, weight,
    reach): weight[b,h,d] = sum_j softmax_j |v_jd| and reach[b,h] = the
    largest scale * sum_d |q_d k_jd|, which the error bounds are made of."""
    B, H, _ = q.shape
    page = cache.shape[1]
    out, weight = np.zeros((B, H, v_dim)), np.zeros((B, H, v_dim))
    lse, reach = np.full((B, H), -np.inf), np.zeros((B, H))
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        k = np.stack([cache[table[b][j // page], j % page] for j in range(n)])
        z = scale * q[b] @ k.T
        reach[b] = (scale * np.abs(q[b]) @ np.abs(k).T).max(-1)
        m = z.max(-1, keepdims=True)
        p = np.exp(z - m)
        total = p.sum(-1, keepdims=True)
        lse[b] = (m + np.log(total))[:, 0]
        out[b] = p / total @ k[:, :v_dim]
        weight[b] = p / total @ np.abs(k[:, :v_dim])
    return out, lse, weight, reach
