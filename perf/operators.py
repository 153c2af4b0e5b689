"""Workloads of the serving operators around the 4-bit KV pools, with their plain forms.

Four operators, in the order in which a decode or prefill step uses them:

  tables   request lengths -> chunk table, slot map, positions of the new tokens
  rope     RMS norm of queries and keys for each head and position rotation, in one pass
  cache    rows written in 4 bits through the slot map, and read back
  attend   decode attention over 4-bit pools: top-k rows plus a window (or the whole context)

The 4-bit format: groups of 16 consecutive values of a row; each value is an e2m1 code (0, 0.5, 1,
1.5, 2, 3, 4, 6 and a sign), each group has one e4m3 scale, and the pool one fp32 scale g, so a value
is e2m1 * e4m3 * g.  A pool is [n_slots, heads, 36 * width] bytes: per slot and head, 64 rows of
width / 2 code bytes (low nibble: even element), then 64 rows of width / 16 scale bytes.
"""
import math

import torch

own = False

CHUNK = 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases ----

def listed():
    return [
        # one decode step of 32 sequences with contexts of 16K to 512K: almost nothing to assign, latency counts
        dict(name="tables_decode_b32", op="tables", B=32, ctx_lo=16384, ctx_hi=524288, new_lo=1, new_hi=1, idle=1),
        # prompts of 64 requests enter next to cached prefixes of any length
        dict(name="tables_prefill_b64", op="tables", B=64, ctx_lo=1, ctx_hi=131072, new_lo=64, new_hi=4096, idle=4),
        # 8 decoded tokens of the latent layout: 128 query rows rotated only, the latent row normalised and rotated
        dict(name="rope_decode_latent_b8", op="rope", T=8, Hq=128, Hk=1, D=576, q_norm=0, k_norm=512, rot_offset=512,
             rot=64, interleaved=True, dtype="bf16", pos_hi=524288, pad=0),
        # a prefill batch with grouped heads, the last rows padding
        dict(name="rope_prefill_gqa", op="rope", T=8192, Hq=32, Hk=8, D=128, q_norm=128, k_norm=128, rot_offset=0,
             rot=128, interleaved=False, dtype="bf16", pos_hi=131072, pad=37),
        # odd head counts and widths in fp32
        dict(name="rope_odd_f32", op="rope", T=777, Hq=12, Hk=3, D=80, q_norm=80, k_norm=80, rot_offset=0,
             rot=32, interleaved=False, dtype="f32", pos_hi=524288, pad=5),
        # the decoded latent rows of 32 sequences
        dict(name="cache_decode_latent_b32", op="cache", T=32, H=1, W=576, two=False, dtype="bf16", g=1.0, pad=1),
        # K and V rows of a prefill batch, 8 heads
        dict(name="cache_prefill_gqa", op="cache", T=16384, H=8, W=128, two=True, dtype="bf16", g=0.5, pad=100),
        # one 16K context, 16 heads over one K/V head, top-k 512 plus the 8000-token window
        dict(name="attend_16k_b1_h16", op="attend", B=1, Hq=16, Hkv=1, dqk=128, dv=128, latent=False, k=512,
             window=8000, ctx_lo=16384, ctx_hi=16384, idle=0, dtype="bf16"),
        # ragged short contexts attended whole, grouped heads, two requests idle
        dict(name="attend_dense_gqa_b16", op="attend", B=16, Hq=32, Hkv=8, dqk=128, dv=128, latent=False, k=0,
             window=16384, ctx_lo=1, ctx_hi=16384, idle=2, dtype="bf16"),
        # 8 contexts of 128K, latent rows, 128 heads
        dict(name="attend_128k_b8_latent", op="attend", B=8, Hq=128, Hkv=1, dqk=576, dv=512, latent=True, k=2048,
             window=8000, ctx_lo=131072, ctx_hi=131072, idle=0, dtype="bf16"),
        # 32 ragged contexts, latent rows, 64 heads
        dict(name="attend_ragged_b32_latent", op="attend", B=32, Hq=64, Hkv=1, dqk=576, dv=512, latent=True, k=2048,
             window=8000, ctx_lo=16384, ctx_hi=524288, idle=0, dtype="bf16"),
        # one context of 512K attended whole: the split axis is long and there are few rows
        dict(name="attend_dense_512k_b1", op="attend", B=1, Hq=32, Hkv=4, dqk=128, dv=128, latent=False, k=0,
             window=524288, ctx_lo=524288, ctx_hi=524288, idle=0, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "cache", "attend", "attend"])
    if op == "tables":
        b = _log(rng, 1, 256)
        return dict(op="tables", B=b, ctx_lo=_log(rng, 1, 4096), ctx_hi=_log(rng, 4096, 131072),
                    new_lo=1, new_hi=_log(rng, 1, 131072 // b), idle=rng.randint(0, b // 4))
    if op == "rope":
        dtype = rng.choice(["bf16", "f16", "f32"])
        if rng.random() < 0.3:
            return dict(op="rope", T=_log(rng, 1, 512), Hq=rng.choice([16, 64, 128]), Hk=1, D=576, q_norm=0, k_norm=512,
                        rot_offset=512, rot=64, interleaved=True, dtype=dtype, pos_hi=_log(rng, 64, 524288), pad=0)
        D = rng.choice([48, 64, 80, 96, 128, 192, 256])
        rot = rng.choice([D, D // 2])
        return dict(op="rope", T=_log(rng, 1, 4096), Hq=rng.randint(1, 40), Hk=rng.randint(1, 8), D=D,
                    q_norm=rng.choice([0, D]), k_norm=rng.choice([0, D]), rot_offset=rng.choice([0, D - rot]), rot=rot,
                    interleaved=rng.random() < 0.5, dtype=dtype, pos_hi=_log(rng, 64, 524288), pad=0)
    if op == "cache":
        if rng.random() < 0.4:
            return dict(op="cache", T=_log(rng, 2, 16384), H=1, W=576, two=False, dtype=rng.choice(["bf16", "f16"]),
                        g=rng.choice([1.0, 0.25]), pad=rng.randint(0, 1))
        return dict(op="cache", T=_log(rng, 2, 16384), H=rng.randint(1, 8), W=rng.choice([64, 128]), two=True,
                    dtype=rng.choice(["bf16", "f16", "f32"]), g=rng.choice([1.0, 0.5, 2.0]), pad=rng.randint(0, 1))
    if rng.random() < 0.5:
        b = _log(rng, 1, 16)
        lo = _log(rng, 1, 65536)
        return dict(op="attend", B=b, Hq=rng.choice([8, 16, 64, 128]), Hkv=1, dqk=576, dv=512, latent=True,
                    k=rng.choice([0, 100, 512, 2048]), window=_log(rng, 64, 8000), ctx_lo=lo, ctx_hi=_log(rng, lo, 131072),
                    idle=rng.randint(0, b // 4), dtype=rng.choice(["bf16", "f16"]))
    hkv, b = rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 32)
    lo = _log(rng, 1, 16384)
    hi = _log(rng, lo, max(lo, 1000000 // (b * hkv)))
    return dict(op="attend", B=b, Hq=hkv * rng.choice([1, 2, 4, 5, 7, 8, 16]), Hkv=hkv, dqk=rng.choice([64, 128]), dv=0,
                latent=False, k=rng.choice([0, 0, 77, 512]), window=_log(rng, 64, 131072), ctx_lo=lo, ctx_hi=hi,
                idle=rng.randint(0, b // 4), dtype=rng.choice(["bf16", "f16"]))


def _spread(lo, hi, n, idle):
    """n lengths from lo to hi, evenly on a logarithmic scale and out of order; the last `idle` are 0."""
    live = n - idle
    at = [(7 * i) % live if live % 7 else i for i in range(live)]
    return [int(round(lo * (hi / lo) ** (i / max(live - 1, 1)))) if live > 1 else hi for i in at] + [0] * idle


def _lengths(c):
    """(tk, window start, window length) of each sequence of an attend case."""
    rows = []
    for n in _spread(c["ctx_lo"], c["ctx_hi"], c["B"], c["idle"]):
        start = max(0, n - c["window"]) // CHUNK * CHUNK
        rows.append((min(c["k"], start), start, n - start))
    return rows


def work(c):
    if c["op"] == "tables":
        ctx, new = _spread(c["ctx_lo"], c["ctx_hi"], c["B"], c["idle"]), _spread(c["new_lo"], c["new_hi"], c["B"], c["idle"])
        have = sum(-(-x // CHUNK) for x in ctx)
        total = sum(new)
        return {"bytes": 4 * have + 4 * c["B"] * _stride(c) + 12 * total + 12 * c["B"], "flops": 0}
    size = {"bf16": 2, "f16": 2, "f32": 4}[c["dtype"]]
    if c["op"] == "rope":
        n = (c["T"] - c["pad"]) * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 2 * size * n + 4 * c["T"], "flops": 6 * n}
    if c["op"] == "cache":
        n = (c["T"] - c["pad"]) * c["H"] * c["W"] * (2 if c["two"] else 1)
        return {"bytes": int((size + 0.5625 + 0.5625 + 2) * n) + 8 * c["T"], "flops": 4 * n}
    rows = sum(t + w for t, _, w in _lengths(c))
    dv = c["dv"] or c["dqk"]
    width = c["dqk"] if c["latent"] else c["dqk"] + dv
    return {"bytes": int(rows * c["Hkv"] * width * 0.5625) + c["B"] * c["Hq"] * (2 * c["dqk"] + 2 * dv + 4),
            "flops": 2 * rows * c["Hq"] * (c["dqk"] + dv)}


# -------------------------------------------------------------- prepare ----

def _stride(c):
    return -(-(c["ctx_hi"] + c["new_hi"]) // CHUNK) + 2


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _layout(pool, W):
    """The code bytes [slots, heads, 64, W / 2] and scales [slots, heads, 64, W / 16] of a pool, as views."""
    n, h = pool.shape[:2]
    return pool[:, :, :32 * W].view(n, h, CHUNK, W // 2), pool[:, :, 32 * W:].view(n, h, CHUNK, W // 16)


def _quantise(x, g):
    """fp32 rows [..., W] -> code bytes [..., W / 2] and scale bytes [..., W / 16]."""
    grp = x.unflatten(-1, (-1, 16))
    # the quotient in 64 bits: amax / 6 is often halfway between two e4m3 values
    s = (grp.abs().amax(-1).double() / (6.0 * g)).clamp(max=448.0).float().to(torch.float8_e4m3fn)
    sg = (s.float() * g).unsqueeze(-1)
    y = torch.where(sg > 0, grp.abs() / sg, torch.zeros_like(grp))
    # nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; halfway cases go to the even code
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = (code + 8 * torch.signbit(grp)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _values(codes, scales, g):
    """Code bytes [..., W / 2] and scale bytes [..., W / 16] -> fp32 values [..., W]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    s = scales.view(torch.float8_e4m3fn).float() * g
    return (v.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _random_pool(n_slots, heads, W, gen):
    """A pool of normal rows, each with a magnitude of its own."""
    pool = torch.empty(n_slots, heads, 36 * W, dtype=torch.uint8, device="cuda")
    codes, scales = _layout(pool, W)
    step = max(1, (1 << 26) // (heads * CHUNK * W))
    for a in range(0, n_slots, step):
        b = min(n_slots, a + step)
        x = torch.randn(b - a, heads, CHUNK, W, device="cuda", generator=gen)
        x *= torch.rand(b - a, heads, CHUNK, 1, device="cuda", generator=gen) + 0.5
        codes[a:b], scales[a:b] = _quantise(x, 1.0)
    return pool


def prepare(case, seed):
    c, gen = case, _gen(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    st = dict(c=c, status=torch.zeros(1, **i32))
    if c["op"] == "tables":
        ctx, new = _spread(c["ctx_lo"], c["ctx_hi"], c["B"], c["idle"]), _spread(c["new_lo"], c["new_hi"], c["B"], c["idle"])
        stride = _stride(c)
        have = torch.tensor([-(-x // CHUNK) for x in ctx], **i32)
        need = sum(-(-(x + y) // CHUNK) for x, y in zip(ctx, new))
        n_slots = need + need // 4 + 8
        # the cached chunks sit anywhere in the pool; entries past them are left over from earlier requests
        perm = torch.randperm(n_slots, device="cuda", generator=gen).int()
        left = torch.randint(-1, n_slots, (c["B"], stride), device="cuda", generator=gen, dtype=torch.int32)
        kept = torch.arange(stride, **i32)[None] < have[:, None]
        table = left
        table[kept] = perm[: int(have.sum())]
        st.update(table=table, cached=torch.tensor(ctx, **i32), new=torch.tensor(new, **i32), n_slots=n_slots,
                  max_new=sum(new) + 64)
        return st
    dt = DTYPES[c["dtype"]]
    if c["op"] == "rope":
        qkv = torch.randn(c["T"], c["Hq"] + c["Hk"], c["D"], device="cuda", generator=gen).to(dt)
        pos = torch.randint(0, c["pos_hi"], (c["T"],), device="cuda", generator=gen, dtype=torch.int32)
        if c["pad"]:
            pos[-c["pad"]:] = -1
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        st.update(q=qkv[:, :c["Hq"]], k=qkv[:, c["Hq"]:], pos=pos, inv=inv.float(), eps=1e-6,
                  wq=(1 + 0.1 * torch.randn(c["q_norm"], device="cuda", generator=gen)).to(dt) if c["q_norm"] else None,
                  wk=(1 + 0.1 * torch.randn(c["k_norm"], device="cuda", generator=gen)).to(dt) if c["k_norm"] else None,
                  q_out=torch.zeros(c["T"], c["Hq"], c["D"], device="cuda", dtype=dt),
                  k_out=torch.zeros(c["T"], c["Hk"], c["D"], device="cuda", dtype=dt))
        return st
    if c["op"] == "cache":
        n_slots = c["T"] // CHUNK + 8
        slots = torch.randperm(n_slots * CHUNK, device="cuda", generator=gen)[:c["T"]]
        if c["pad"]:
            slots[-c["pad"]:] = -1
        names = ("k", "v") if c["two"] else ("k",)
        for n in names:
            x = torch.randn(c["T"], c["H"], c["W"], device="cuda", generator=gen)
            x *= torch.exp(torch.randn(c["T"], c["H"], 1, device="cuda", generator=gen))
            st[n] = x.to(dt)
            st[n + "_pool"] = torch.zeros(n_slots, c["H"], 36 * c["W"], dtype=torch.uint8, device="cuda")
        st.update(slots=slots)
        return st
    rows, dv = _lengths(c), c["dv"] or c["dqk"]
    stride = -(-c["ctx_hi"] // CHUNK) + 1
    n_ch = [-(-(s + w) // CHUNK) for _, s, w in rows]
    n_slots = sum(n_ch) + 5
    perm = torch.randperm(n_slots, device="cuda", generator=gen).int()
    table = torch.full((c["B"], stride), -1, **i32)
    topk = torch.full((c["B"], c["k"]), -1, **i32)
    at = 0
    for b, (tk, start, _) in enumerate(rows):
        table[b, :n_ch[b]] = perm[at:at + n_ch[b]]
        at += n_ch[b]
        if tk:
            pick = torch.rand(start, device="cuda", generator=gen).topk(tk).indices
            topk[b, :tk] = pick.sort().values.int()
    st.update(q=torch.randn(c["B"], c["Hq"], c["dqk"], device="cuda", generator=gen).to(dt), table=table, topk=topk,
              count=torch.tensor([r[0] for r in rows], **i32), start=torch.tensor([r[1] for r in rows], **i32),
              length=torch.tensor([r[2] for r in rows], **i32), longest=max(max(r[2] for r in rows), 1), dv=dv,
              scale=c["dqk"] ** -0.5, k_pool=_random_pool(n_slots, c["Hkv"], c["dqk"], gen),
              v_pool=None if c["latent"] else _random_pool(n_slots, c["Hkv"], dv, gen))
    return st


# ------------------------------------------------------------------ run ----

def run(st):
    op = st["c"]["op"]
    return _own(st, op) if own else {"tables": _tables, "rope": _rope, "cache": _cache, "attend": _attend}[op](st)


def _own(st, op):
    from learned_sparse_kv_b200 import lsa
    c, status = st["c"], st["status"]
    if op == "tables":
        return lsa.build_tables(st["table"], st["cached"], st["new"], st["n_slots"], st["max_new"], status=status)
    if op == "rope":
        return lsa.qk_norm_rope(st["q"], st["k"], st["pos"], st["inv"], q_weight=st["wq"], k_weight=st["wk"],
                                q_norm_width=c["q_norm"], k_norm_width=c["k_norm"], eps=st["eps"],
                                rot_offset=c["rot_offset"], interleaved=c["interleaved"], q_out=st["q_out"],
                                k_out=st["k_out"])
    if op == "cache":
        two = c["two"]
        lsa.write_q4(st["k"], st["k_pool"], st["slots"], v=st["v"] if two else None,
                     v_pool=st["v_pool"] if two else None, k_scale=c["g"], v_scale=c["g"], status=status)
        k = lsa.read_q4(st["k_pool"], st["slots"], scale=c["g"], status=status)
        return (k, lsa.read_q4(st["v_pool"], st["slots"], scale=c["g"], status=status)) if two else (k,)
    return lsa.sparse_decode_q4(st["q"], st["k_pool"], st["v_pool"], st["table"], st["topk"], st["count"], st["start"],
                                st["length"], st["longest"], st["dv"], st["scale"], out_dtype=st["q"].dtype,
                                status=status)


def _tables(st):
    """Kept chunks keep their slots, new chunks take the free slots in order, new tokens get slot and position."""
    table, cached, new, n_slots = st["table"], st["cached"], st["new"], st["n_slots"]
    B, stride = table.shape
    dev = table.device
    c = torch.arange(stride, device=dev)[None]
    have, need = (cached + 63)[:, None] // CHUNK, (cached + new + 63)[:, None] // CHUNK
    kept = c < have
    used = torch.zeros(n_slots + 1, dtype=torch.int32, device=dev)
    used[torch.where(kept, table, n_slots).flatten().long()] = 1
    free = torch.sort(used[:n_slots], stable=True).indices
    n_free = n_slots - used[:n_slots].sum()
    wants = (c >= have) & (c < need)
    rank = (torch.cumsum(wants.flatten().int(), 0) - 1).view(B, stride)
    fresh = torch.where(rank < n_free, free[rank.clamp(0, n_slots - 1)], -1).int()
    nxt = torch.where(kept, table, torch.where(wants, fresh, -1)).int()
    offset = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0)).int()
    i = torch.arange(st["max_new"], device=dev)
    b = torch.searchsorted(offset[1:].contiguous(), i, right=True).clamp(max=B - 1)
    pos = cached[b] + i - offset[b]
    slot = nxt[b, (pos // CHUNK).clamp(0, stride - 1)].long()
    live = i < offset[B]
    slots = torch.where(live & (slot >= 0), slot * CHUNK + pos % CHUNK, -1)
    left = (n_free - wants.sum()).clamp(min=0).int().reshape(1)
    return nxt, slots, torch.where(live, pos, -1).int(), offset, left


def _norm_rotate(x, weight, width, st, out):
    c = st["c"]
    y = x.float()
    if width:
        part = y[..., :width]
        part = part * torch.rsqrt((part * part).mean(-1, keepdim=True) + st["eps"])
        if weight is not None:
            part = part * weight.float()
        y = torch.cat([part, y[..., width:]], -1)
    a = c["rot_offset"]
    angle = st["pos"].double()[:, None] * st["inv"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = y[..., a:a + c["rot"]]
    if c["interleaved"]:
        u, v = r[..., 0::2], r[..., 1::2]
        r = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    else:
        u, v = r.chunk(2, -1)
        r = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    y = torch.cat([y[..., :a], r, y[..., a + c["rot"]:]], -1).to(x.dtype)
    return torch.where((st["pos"] >= 0)[:, None, None], y, out)


def _rope(st):
    c = st["c"]
    return (_norm_rotate(st["q"], st["wq"], c["q_norm"], st, st["q_out"]),
            _norm_rotate(st["k"], st["wk"], c["k_norm"], st, st["k_out"]))


def _store_load(x, pool, slots, g):
    codes, scales = _layout(pool, x.shape[-1])
    live = slots >= 0
    at, row = slots.clamp(min=0) // CHUNK, slots.clamp(min=0) % CHUNK
    qc, qs = _quantise(x.float(), g)
    # a padded row stores what its slot holds: it changes nothing
    keep = live[:, None, None]
    first = torch.argmax(live.int())
    at, row = torch.where(live, at, at[first]), torch.where(live, row, row[first])
    codes[at, :, row] = torch.where(keep, qc, qc[first][None])
    scales[at, :, row] = torch.where(keep, qs, qs[first][None])
    return torch.where(keep, _values(codes[at, :, row], scales[at, :, row], g), 0.0).to(torch.bfloat16)


def _cache(st):
    g = st["c"]["g"]
    k = _store_load(st["k"], st["k_pool"], st["slots"], g)
    return (k, _store_load(st["v"], st["v_pool"], st["slots"], g)) if st["c"]["two"] else (k,)


def _row_set(st):
    """Pool slot, row in it, and presence of each attended row, [B, rows]."""
    w = torch.arange(st["longest"], device="cuda")[None]
    pos = torch.cat([st["topk"].clamp(min=0), (st["start"][:, None] + w)], 1)
    n = st["topk"].shape[1]
    there = torch.cat([torch.arange(n, device="cuda")[None] < st["count"][:, None], w < st["length"][:, None]], 1)
    pos = torch.where(there, pos, 0).long()
    slot = torch.gather(st["table"], 1, pos // CHUNK).clamp(min=0).long()
    return slot, pos % CHUNK, there


def _gathered(pool, W, slot, row):
    codes, scales = _layout(pool, W)
    return _values(codes[slot, :, row], scales[slot, :, row], 1.0)   # [B, rows, heads, W]


def _attend(st):
    q, dv = st["q"].float(), st["dv"]
    B, Hq, dqk = q.shape
    slot, row, there = _row_set(st)
    k = _gathered(st["k_pool"], dqk, slot, row)
    v = k[..., :dv] if st["v_pool"] is None else _gathered(st["v_pool"], dv, slot, row)
    Hkv = k.shape[2]
    qg = q.view(B, Hkv, Hq // Hkv, dqk)
    s = torch.matmul(qg, k.permute(0, 2, 3, 1)) * st["scale"]
    s = s.masked_fill(~there[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + m
    return o.reshape(B, Hq, dv).to(st["q"].dtype), lse.reshape(B, Hq)


# ---------------------------------------------------------------- exact ----

def _e4m3(t):
    """t >= 0 rounded to the nearest e4m3 value (halfway to even), at most 448, in 64 bits."""
    t = t.clamp(max=448.0)
    e = ((t.view(torch.int64) >> 52) - 1023).clamp(min=-6)   # floor(log2 t), subnormal below 2^-6
    u = ((e - 3 + 1023) << 52).view(torch.float64)           # the step at t: 2^(e - 3)
    return torch.round(t / u) * u


def _e2m1(y):
    """y >= 0 rounded to the nearest e2m1 value (halfway to even), in 64 bits."""
    u = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    return (torch.round(y / u) * u).clamp(max=6.0)


def _decode64(pool, W, slot, row):
    """float64 rows of a pool: the sign, exponent and mantissa bits of every code, written out."""
    n, h = pool.shape[:2]
    flat = pool.reshape(n * h, 36 * W)
    unit = slot[..., None] * h + torch.arange(h, device=pool.device)                    # [B, rows, heads]
    j = torch.arange(W, device=pool.device)
    byte = flat[unit[..., None], row[..., None, None] * (W // 2) + j // 2].long()
    code = (byte >> (4 * (j % 2))) & 15
    e, m = (code >> 1) & 3, code & 1
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e - 1).double())
    sb = flat[unit[..., None], 32 * W + row[..., None, None] * (W // 16) + j // 16].long()
    se, sm = (sb >> 3) & 15, (sb & 7).double()
    scale = torch.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8) * 2.0 ** (se - 7).double())
    return mag * scale * torch.where(code >= 8, -1.0, 1.0)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "tables":
        return None   # whole numbers only
    if c["op"] == "rope":
        outs = []
        for x, w, width, buf in ((st["q"], st["wq"], c["q_norm"], st["q_out"]), (st["k"], st["wk"], c["k_norm"], st["k_out"])):
            y = x.double().clone()
            if width:
                ms = y[..., :width].pow(2).sum(-1, keepdim=True) / width
                y[..., :width] = y[..., :width] / (ms + st["eps"]).sqrt() * (1.0 if w is None else w.double())
            half, a = c["rot"] // 2, c["rot_offset"]
            i = torch.arange(half, device=y.device)
            iu, iv = (a + 2 * i, a + 2 * i + 1) if c["interleaved"] else (a + i, a + half + i)
            z = torch.complex(y[..., iu], y[..., iv])
            turn = st["pos"].double()[:, None] * st["inv"].double()[None]
            z = z * torch.polar(torch.ones_like(turn), turn)[:, None]
            y[..., iu], y[..., iv] = z.real, z.imag
            y[st["pos"] < 0] = buf[st["pos"] < 0].double()
            outs.append(y)
        return tuple(outs)
    if c["op"] == "cache":
        outs = []
        for n in ("k", "v") if c["two"] else ("k",):
            x = st[n].double().unflatten(-1, (-1, 16))
            s = _e4m3(x.abs().amax(-1, keepdim=True) / 6 / c["g"]) * c["g"]
            y = torch.where(s > 0, x.abs() / s.clamp(min=1e-300), 0.0)
            val = (_e2m1(y) * s * x.sign()).flatten(-2)
            val[st["slots"] < 0] = 0
            outs.append(val)
        return tuple(outs)
    Hq, Hkv, dv = c["Hq"], c["Hkv"], st["dv"]
    G = Hq // Hkv
    o = torch.zeros(c["B"], Hq, dv, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (tk, start, n) in enumerate(_lengths(c)):
        if tk + n == 0:
            continue
        pos = torch.cat([st["topk"][b, :tk].long(), start + torch.arange(n, device="cuda")])
        slot = st["table"][b].long()[pos // CHUNK]
        for h in range(Hkv):
            kp = st["k_pool"][:, h:h + 1]
            k = _decode64(kp, c["dqk"], slot, pos % CHUNK)[:, 0]
            v = k[:, :dv] if st["v_pool"] is None else _decode64(st["v_pool"][:, h:h + 1], dv, slot, pos % CHUNK)[:, 0]
            s = st["q"][b, h * G:(h + 1) * G].double() @ k.T * st["scale"]
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
            o[b, h * G:(h + 1) * G] = torch.softmax(s, -1) @ v
    return o, lse
