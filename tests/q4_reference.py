"""64-bit reference of the 4-bit pools, the attention over them, the tables and the rotation,
written from the definitions (numpy only)."""
import numpy as np

CH = 64
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)], np.float64)[:127]      # byte 127 is NaN


def _nearest_even(x, table):
    """Index of the table entry nearest to each x >= 0; halfway goes to the even index; saturates."""
    i = np.clip(np.searchsorted(table, x, side="right") - 1, 0, len(table) - 1)
    j = np.minimum(i + 1, len(table) - 1)
    lo, hi = x - table[i], table[j] - x
    up = (hi < lo) | ((hi == lo) & (i % 2 == 1))
    return np.where((j > i) & up, j, i)


def quantise(x, g=1.0):
    """float64 rows [..., W] -> (codes [..., W] 0..15, scale bytes [..., W / 16])."""
    grp = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    amax = np.abs(grp).max(-1)
    sb = _nearest_even(np.minimum(amax / (6.0 * g), 448.0), E4M3)
    s = E4M3[sb][..., None] * g
    y = np.divide(np.abs(grp), s, out=np.zeros_like(grp), where=s > 0)
    code = _nearest_even(y, E2M1) + 8 * (np.signbit(grp) & (s > 0))
    return code.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def values(codes, scales, g=1.0):
    v = E2M1[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    s = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])[scales]
    return (v.reshape(v.shape[:-1] + (-1, 16)) * s[..., None]).reshape(v.shape) * g


def pack(codes, scales):
    """codes [n_slots, heads, 64, W], scales [n_slots, heads, 64, W / 16] -> pool bytes."""
    n, h, _, W = codes.shape
    c = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return np.concatenate([c.reshape(n, h, 32 * W), scales.reshape(n, h, 4 * W)], -1)


def unpack(pool):
    n, h, nb = pool.shape
    W = nb // 36
    c = pool[:, :, :32 * W].reshape(n, h, CH, W // 2)
    codes = np.empty((n, h, CH, W), np.uint8)
    codes[..., 0::2], codes[..., 1::2] = c & 15, c >> 4
    return codes, pool[:, :, 32 * W:].reshape(n, h, CH, W // 16)


def pool_values(pool, g=1.0):
    return values(*unpack(pool), g)


def row_set(b, table, topk_idx, topk_count, start, length, n_slots):
    """(slot, row) of the attended rows of sequence b."""
    pos = [] if topk_idx is None else list(topk_idx[b, :max(0, min(topk_count[b], topk_idx.shape[1]))])
    if start[b] >= 0:
        pos += list(range(start[b], start[b] + max(length[b], 0)))
    out = []
    for p in pos:
        if p < 0 or p // CH >= table.shape[1]:
            continue
        s = table[b, p // CH]
        if 0 <= s < n_slots:
            out.append((s, p % CH))
    return np.array(out, np.int64).reshape(-1, 2)


def attend(q, kv, vv, dv, rows, scale):
    """One sequence: q [Hq, dqk], kv / vv [n_slots, heads, 64, W] values (vv None: latent).
    Returns o [Hq, dv], lse [Hq], and for error bounds: sum_j p_j |v_j| [Hq, dv], and the largest
    scale * sum_i |q_i k_ji| over the rows [Hq], and sum_j |v_j| [Hq, dv]."""
    Hq, dqk = q.shape
    heads = kv.shape[1]
    G = Hq // heads
    o, spread, flat = np.zeros((Hq, dv)), np.zeros((Hq, dv)), np.zeros((Hq, dv))
    lse, mag = np.full(Hq, -np.inf), np.zeros(Hq)
    if len(rows):
        for h in range(heads):
            k = kv[rows[:, 0], h, rows[:, 1]]
            v = k[:, :dv] if vv is None else vv[rows[:, 0], h, rows[:, 1]]
            qs = q[h * G:(h + 1) * G]
            s = qs @ k.T * scale
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            t = p.sum(-1, keepdims=True)
            sl = slice(h * G, (h + 1) * G)
            o[sl], spread[sl] = p @ v / t, p @ np.abs(v) / t
            flat[sl] = np.abs(v).sum(0)
            lse[sl] = (np.log(t) + m)[:, 0]
            mag[sl] = (np.abs(qs) @ np.abs(k).T).max(-1) * scale
    return o, lse, spread, mag, flat


def tables(table, cached, new, n_slots, max_new):
    """(table_next, slot_map, position, new_offset, n_free), request by request."""
    B, stride = table.shape
    cached = np.maximum(cached, 0)
    new = np.minimum(np.maximum(new, 0), 2 ** 31 - 1 - cached)        # positions are int32
    nxt = np.full((B, stride), -1, np.int32)
    have = [min(-(-int(c) // CH), stride) for c in cached]
    need = [min(-(-int(c + n) // CH), stride) for c, n in zip(cached, new)]
    used = set()
    for b in range(B):
        for c in range(have[b]):
            if 0 <= table[b, c] < n_slots:
                nxt[b, c] = table[b, c]
                used.add(int(table[b, c]))
    free = [s for s in range(n_slots) if s not in used]
    taken = 0
    for b in range(B):
        for c in range(have[b], need[b]):
            if taken < len(free):
                nxt[b, c] = free[taken]
            taken += 1
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    slot_map, position = np.full(max_new, -1, np.int64), np.full(max_new, -1, np.int32)
    for b in range(B):
        for i in range(int(new[b])):
            at, pos = int(off[b]) + i, int(cached[b]) + i
            if at >= max_new:
                break
            position[at] = pos
            if pos // CH < stride and nxt[b, pos // CH] >= 0:
                slot_map[at] = int(nxt[b, pos // CH]) * CH + pos % CH
    return nxt, slot_map, position, off.astype(np.int32), max(len(free) - taken, 0)


def norm_rope(x, weight, width, position, inv_freq, rot_offset, interleaved, eps):
    """float64 rows [T, H, D]."""
    y = x.astype(np.float64).copy()
    if width:
        y[..., :width] /= np.sqrt((y[..., :width] ** 2).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y[..., :width] *= weight
    half = len(inv_freq)
    a = position.astype(np.float64)[:, None, None] * inv_freq.astype(np.float64)
    i = np.arange(half)
    iu, iv = (rot_offset + 2 * i, rot_offset + 2 * i + 1) if interleaved else (rot_offset + i, rot_offset + half + i)
    u, v = y[..., iu].copy(), y[..., iv].copy()
    y[..., iu], y[..., iv] = u * np.cos(a) - v * np.sin(a), v * np.cos(a) + u * np.sin(a)
    return y
