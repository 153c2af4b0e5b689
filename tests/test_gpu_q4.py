"""GPU parity of the 4-bit pools and the attention over them with a 64-bit reference.

Stored codes and scales must match bit for bit.  Attention bounds, per element, with
A = sum_j p_j |v_j| and D = (dqk + 32) 2^-23 scale max_j sum_i |q_i k_ji| (fp32 accumulation of a
score, one rounding of at most 2^-23 a step) plus dqk 2^-25 scale max|q| max|k| (query entries below f16's range):
  every weight is off by at most 2^-11 (f16) + 2 D + 2^-20 (exp2, fp32 sums), the result is rounded
  once to its type (eps / 2), fp32 sums of n rows add n 2^-24 at the most:
  |o - ref| <= (2^-11 + 2 D + 2^-20 + n 2^-24) A + eps_out / 2 |ref| + 2^-31 sum_j |v_j|
(the last term: weights are held as f16 with the largest at 2^6 or more, so a weight below f16's normal range,
2^-20 of the largest, is off by half a step of its subnormals, 2^-25 / 2^6 = 2^-31 of the largest, and the
largest is at most the sum)
  |lse - ref| <= D + 2^-20 + 2^-22 |ref|
"""
import numpy as np
import pytest
import torch

from tests import q4_reference as R

pytestmark = pytest.mark.gpu
CH = 64
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def L():
    from learned_sparse_kv_b200 import lsa
    return lsa


def cu(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------- write, read --

def _rows(rng, T, H, W, dtype):
    x = rng.standard_normal((T, H, W)) * np.exp(2 * rng.standard_normal((T, H, 1)))
    x[:, :, ::7] *= 30.0
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,W,two,g", [(1, 1, 576, False, 1.0), (33, 2, 128, True, 0.5), (257, 3, 64, True, 4.0),
                                         (5, 1, 16, False, 1.0), (64, 5, 176, True, 0.25)])
def test_write_then_read_exact(L, dtype, T, H, W, two, g):
    rng = np.random.default_rng(T + W)
    n_slots = T // CH + 3
    slots = rng.permutation(n_slots * CH)[:T].astype(np.int64)
    slots[T // 2:T // 2 + 2] = -1 if T > 4 else slots[T // 2:T // 2 + 2]
    x = [_rows(rng, T, H, W, dtype) for _ in range(1 + two)]
    before = [rng.integers(0, 256, (n_slots, H, 36 * W), dtype=np.uint8) for _ in x]
    pools = [cu(p) for p in before]
    st = status()
    L.write_q4(x[0].cuda(), pools[0], cu(slots), v=x[1].cuda() if two else None, v_pool=pools[1] if two else None,
               k_scale=g, v_scale=g, status=st)
    live = slots >= 0
    for xi, pool, old in zip(x, pools, before):
        codes, scales = R.unpack(old)
        qc, qs = R.quantise(xi.double().numpy(), g)
        # written row by row; everything else keeps its bytes
        codes[slots[live] // CH, :, slots[live] % CH] = qc[live]
        scales[slots[live] // CH, :, slots[live] % CH] = qs[live]
        got = pool.cpu().numpy()
        gc, gs = R.unpack(got)
        np.testing.assert_array_equal(gs, scales)
        np.testing.assert_array_equal(gc, codes)
        for out_dtype in (torch.bfloat16, torch.float32):
            back = L.read_q4(pool, cu(slots), scale=g, out_dtype=out_dtype, status=st).double().cpu().numpy()
            ref = np.where(live[:, None, None], R.values(qc, qs, g), 0.0)
            np.testing.assert_array_equal(back, ref)   # 6 significant bits and a power of two: exact
    assert st.item() == 0


def test_write_special_values_and_strides(L):
    """Halfway cases, zeros, tiny and huge rows, infinities and NaN; rows that are a view of a fused buffer."""
    W = 64
    x = np.zeros((8, 2, W), np.float32)
    x[0, 0] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0], 4)
    x[1, 0, :16] = 1e-30
    x[1, 0, 16:32] = 3e38
    x[2, 0, 5] = np.inf
    x[2, 1, 7] = -np.inf
    x[2, 1, 8] = 1.0
    x[3, 0, 20] = np.nan
    x[4, 1] = 6 * 2.0 ** -10          # amax / 6 halfway between 0 and the smallest scale
    x[5, 1] = 6 * 3 * 2.0 ** -10
    x[6, 0] = 2688.0
    x[6, 1] = 3000.0
    x[7] = -0.0
    big = torch.zeros(8, 5, W, device="cuda")
    big[:, 1:3] = cu(x)
    pool = L.q4_pool(1, 2, W)
    slots = torch.arange(8, device="cuda") * 3
    L.write_q4(big[:, 1:3], pool, slots)
    got = L.read_q4(pool, slots, out_dtype=torch.float32).cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref = R.values(*R.quantise(np.where(np.isfinite(x), x, 0.0).astype(np.float64)))
    ref[2, 0, :16] = 0.0
    ref[2, 0, 5] = 2688.0
    ref[2, 1, :16] = 0.0
    ref[2, 1, 7] = -2688.0            # the scale saturates at 448: 1 / 448 rounds to 0
    ref[3, 0, 16:32] = np.nan
    np.testing.assert_array_equal(got, ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("g", [1.0, 2.0 ** -5, 0.75])
def test_write_every_significand(L, dtype, g):
    """Every value of the type over five octaves below the group's maximum, for each significand of the
    scale, halfway cases among them; and every significand of the maximum itself."""
    bits = np.arange(1 << 16, dtype=np.uint16).view(np.int16)
    every = torch.from_numpy(bits).view(dtype).double()
    groups = []
    for m in range(8):
        s = (1 + m / 8) * g
        top = 6.0 * s
        x = every[(every.abs() <= top) & (every.abs() >= top / 32)]
        x = torch.cat([x, torch.zeros(-len(x) % 15, dtype=torch.float64)]).view(-1, 15)
        groups.append(torch.cat([x, torch.full((len(x), 1), top, dtype=torch.float64)], 1))
    x = every[(every >= 1) & (every < 8)]
    groups.append(torch.cat([x[:, None], torch.zeros(len(x), 15, dtype=torch.float64)], 1))
    x = torch.cat(groups).to(dtype)
    x = torch.cat([x, torch.zeros(-len(x) % 4, 16, dtype=dtype)]).view(-1, 1, 64)
    T = len(x)
    pool = L.q4_pool(T // CH + 1, 1, 64)
    L.write_q4(x.cuda(), pool, torch.arange(T, device="cuda"), k_scale=g)
    codes, scales = R.unpack(pool.cpu().numpy())
    # g = 0.75: the product s g and the quotients are rounded to fp32 before the codes, as the definition has it
    qc, qs = R.quantise(x.double().numpy(), g) if g != 0.75 else _fp32_quantise(x.float().numpy(), np.float32(g))
    np.testing.assert_array_equal(scales.transpose(0, 2, 1, 3).reshape(-1, 1, 4)[:T], qs)
    np.testing.assert_array_equal(codes.transpose(0, 2, 1, 3).reshape(-1, 1, 64)[:T], qc)


def _fp32_quantise(x, g):
    """R.quantise with its two quotients and one product rounded to fp32."""
    grp = x.reshape(x.shape[:-1] + (-1, 16))
    t = np.minimum(np.abs(grp).max(-1) / (np.float32(6) * g), np.float32(448))
    sb = R._nearest_even(t.astype(np.float64), R.E4M3)
    sg = (R.E4M3[sb].astype(np.float32) * g)[..., None]
    y = np.divide(np.abs(grp), sg, out=np.zeros_like(grp), where=sg > 0)
    code = R._nearest_even(y.astype(np.float64), R.E2M1) + 8 * (np.signbit(grp) & (sg > 0))
    return code.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def test_write_skips_and_flags_slots_outside_the_pool(L):
    x = torch.ones(3, 1, 64, device="cuda")
    pool = L.q4_pool(2, 1, 64)
    st = status()
    L.write_q4(x, pool, torch.tensor([2 * CH, -2, 5], device="cuda"), status=st)
    assert st.item() == L.DEV_INDEX
    assert int((pool != 0).sum()) == 32 + 4           # row 5 alone
    st.zero_()
    out = L.read_q4(pool, torch.tensor([2 * CH, 5, -1], device="cuda"), status=st)
    assert st.item() == L.DEV_INDEX
    # 1 / 6 = 10.67 / 64 rounds to the scale 11 / 64, and 64 / 11 = 5.8 to the code 6: 66 / 64
    np.testing.assert_array_equal(out[:, 0, 0].float().cpu().numpy(), [0, 66 / 64, 0])


def test_write_of_nothing(L):
    pool = L.q4_pool(1, 2, 64)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    L.write_q4(torch.empty(0, 2, 64, device="cuda"), pool, none)
    assert L.read_q4(pool, none).shape == (0, 2, 64)


@pytest.mark.parametrize("two", [False, True])
def test_append_token(L, two):
    rng = np.random.default_rng(3)
    B, H, W, dl, n_slots = 5, 2, 128, 64, 9
    table = np.array([[0, 1], [2, 3], [4, -1], [5, 6], [7, 8]], np.int32)
    start = np.array([0, 0, 0, 64, 0], np.int32)
    length = np.array([0, 63, 64, 1, 127], np.int32)     # sequence 2 has no chunk for position 64
    k, v = (_rows(rng, B, H, W, torch.bfloat16) for _ in range(2))
    li = torch.randn(B, dl).bfloat16()
    kp, vp = L.q4_pool(n_slots, H, W), L.q4_pool(n_slots, H, W)
    lip = torch.zeros(n_slots, CH, dl, dtype=torch.bfloat16, device="cuda")
    wl, st = cu(length), status()
    L.append_token_q4(k.cuda(), v.cuda() if two else None, li.cuda(), kp, vp if two else None, lip, cu(table), cu(start),
                      wl, status=st)
    assert st.item() == L.DEV_TABLE
    np.testing.assert_array_equal(wl.cpu().numpy(), length + np.array([1, 1, 0, 1, 1]))
    pos = start + length
    for x, pool in ((k, kp), (v, vp))[:1 + two]:
        codes, scales = (np.zeros((n_slots, H, CH, W), np.uint8), np.zeros((n_slots, H, CH, W // 16), np.uint8))
        qc, qs = R.quantise(x.double().numpy())
        for b in (0, 1, 3, 4):
            codes[table[b, pos[b] // CH], :, pos[b] % CH] = qc[b]
            scales[table[b, pos[b] // CH], :, pos[b] % CH] = qs[b]
        np.testing.assert_array_equal(pool.cpu().numpy(), R.pack(codes, scales))
    for b in (0, 1, 3, 4):
        assert torch.equal(lip[table[b, pos[b] // CH], pos[b] % CH].cpu(), li[b])
    assert int((lip != 0).any(-1).sum()) == 4


# --------------------------------------------------------------- attention --

def _pool(rng, n_slots, heads, W, magnitude=1.0):
    x = rng.standard_normal((n_slots, heads, CH, W)) * rng.uniform(0.3, 2.0, (n_slots, heads, CH, 1)) * magnitude
    return R.pack(*R.quantise(x))


def _case(seed, B, Hq, heads, dqk, dv, latent, k, starts, lengths, q_std=1.0, dtype=torch.bfloat16, shift=0):
    """Sequences of any start and length; rows outside the sets hold NaN scales."""
    rng = np.random.default_rng(seed)
    start, length = np.array(starts, np.int32), np.array(lengths, np.int32)
    n_ch = [-(-int(s + w) // CH) for s, w in zip(start, length)]
    stride = max(max(n_ch), 1) + 1
    n_slots = sum(n_ch) + 3
    perm = rng.permutation(n_slots).astype(np.int32)
    table, at = np.full((B, stride), -1, np.int32), 0
    topk, count = np.full((B, max(k, 1)), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        table[b, :n_ch[b]] = perm[at:at + n_ch[b]]
        at += n_ch[b]
        count[b] = min(k, start[b])
        topk[b, :count[b]] = np.sort(rng.permutation(start[b])[:count[b]])
    kp = _pool(rng, n_slots, heads, dqk)
    vp = None if latent else _pool(rng, n_slots, heads, dv)
    wanted = np.zeros((n_slots, CH), bool)
    for b in range(B):
        r = R.row_set(b, table, topk, count, start, length, n_slots)
        wanted[r[:, 0], r[:, 1]] = True
    for p in (kp, vp):
        if p is not None:
            codes, scales = R.unpack(p)
            codes = codes.copy()
            scales = scales.copy()
            codes[~np.broadcast_to(wanted[:, None], codes.shape[:3])] = 0x0f
            scales[~np.broadcast_to(wanted[:, None], scales.shape[:3])] = 0x7f
            p[...] = R.pack(codes, scales)
    q = (torch.from_numpy(rng.standard_normal((B, Hq, dqk)) * q_std) + shift).to(dtype)
    return dict(q=q, kp=kp, vp=vp, table=table, topk=topk if k else None, count=count, start=start, length=length,
                dv=dv, scale=dqk ** -0.5)


def _run(L, c, out_dtype=torch.bfloat16, k_scale=1.0, v_scale=1.0, st=None, **kw):
    return L.sparse_decode_q4(c["q"].cuda(), cu(c["kp"]), None if c["vp"] is None else cu(c["vp"]), cu(c["table"]),
                              None if c["topk"] is None else cu(c["topk"]), None if c["topk"] is None else cu(c["count"]),
                              cu(c["start"]), cu(c["length"]), max(int(c["length"].max()), 0), c["dv"], c["scale"],
                              k_scale=k_scale, v_scale=v_scale, out_dtype=out_dtype, status=st, **kw)


def _bounds(q, kv, vv, dv, rows, scale, eps_out):
    """Reference and tolerance of one sequence's output and lse."""
    dqk = q.shape[-1]
    ro, rl, spread, mag, flat = R.attend(q, kv, vv, dv, rows, scale)
    kmax = np.abs(kv[rows[:, 0], :, rows[:, 1]]).max()
    D = (dqk + 32) * 2.0 ** -23 * mag + dqk * 2.0 ** -25 * scale * np.abs(q).max(-1) * kmax
    tol = ((2.0 ** -11 + 2 * D[:, None] + 2.0 ** -20 + len(rows) * 2.0 ** -24) * spread + eps_out * np.abs(ro) +
           2.0 ** -31 * flat)
    return ro, tol, rl, D + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl)


def _check(c, out, lse, k_scale=1.0, v_scale=1.0, heads=slice(None)):
    kv = R.pool_values(c["kp"], k_scale)
    vv = None if c["vp"] is None else R.pool_values(c["vp"], v_scale)
    q = c["q"].double().numpy()[:, heads]
    o, s = out.double().cpu().numpy()[:, heads], lse.double().cpu().numpy()[:, heads]
    for b in range(len(q)):
        rows = R.row_set(b, c["table"], c["topk"], c["count"], c["start"], c["length"], len(c["kp"]))
        if not len(rows):
            assert np.all(o[b] == 0) and np.all(np.isneginf(s[b]))
            continue
        ro, to, rl, tl = _bounds(q[b], kv, vv, c["dv"], rows, c["scale"], EPS[out.dtype])
        bad = np.abs(o[b] - ro) > to
        assert not bad.any(), (b, int(bad.sum()), np.abs(o[b] - ro).max(), to.min())
        assert np.all(np.abs(s[b] - rl) <= tl), (b, np.abs(s[b] - rl).max())


SHAPES = [(4, 4, 128, 128, False), (8, 1, 128, 128, False), (16, 1, 128, 128, False), (15, 3, 128, 128, False),
          (36, 1, 64, 64, False), (14, 2, 64, 64, False), (12, 4, 64, 64, False),
          (128, 1, 576, 512, True), (64, 1, 576, 512, True), (1, 1, 576, 512, True), (97, 1, 576, 512, True)]


@pytest.mark.parametrize("Hq,heads,dqk,dv,latent", SHAPES)
def test_attention_ragged_windows(L, Hq, heads, dqk, dv, latent):
    """Lengths of 0, 1, around a chunk and around a tile, windows that start inside a chunk, top-k rows."""
    starts = [0, 0, 0, 64, 63, 128, 0, 200, 640, 0]
    lengths = [0, 1, 64, 65, 2, 0, 127, 300, 129, 1000]
    c = _case(Hq + dqk, 10, Hq, heads, dqk, dv, latent, 100, starts, lengths)
    st = status()
    out, lse = _run(L, c, st=st)
    assert st.item() == 0
    _check(c, out, lse)


@pytest.mark.parametrize("Hq,heads,dqk,dv,latent", [(8, 2, 128, 128, False), (40, 2, 64, 64, False),
                                                    (128, 1, 576, 512, True)])
@pytest.mark.parametrize("q_dtype,out_dtype", [(torch.float16, torch.float16), (torch.bfloat16, torch.float32)])
def test_attention_types_scales_and_splits(L, Hq, heads, dqk, dv, latent, q_dtype, out_dtype):
    """One long sequence (many splits), pool scales that are no powers of two, peaked queries."""
    c = _case(5, 2, Hq, heads, dqk, dv, latent, 77, [2500, 0], [3001, 4097], q_std=3.0, dtype=q_dtype)
    out, lse = _run(L, c, out_dtype, k_scale=0.3, v_scale=1.7)
    _check(c, out, lse, 0.3, 0.3 if latent else 1.7)


@pytest.mark.parametrize("latent", [False, True])
def test_attention_query_magnitudes(L, latent):
    """Queries far outside f16's range, and a zero query, keep the softmax of the definition."""
    Hq, heads, dqk, dv = (128, 1, 576, 512) if latent else (8, 1, 128, 128)
    c = _case(9, 1, Hq, heads, dqk, dv, latent, 0, [0], [300])
    q = c["q"]
    for h, f in enumerate([2.0 ** 40, 2.0 ** -40, 0.0, 2.0 ** 17]):
        q[0, h] *= f
    c["scale"] = 2.0 ** -18
    out, lse = _run(L, c)
    assert bool(torch.isfinite(lse[0, 1:]).all())
    # the first head's scores differ by more than fp32 resolves: only the others are compared
    _check(c, out, lse, heads=slice(1, 8))


@pytest.mark.parametrize("latent", [False, True])
def test_attention_skips_and_flags_bad_pages(L, latent):
    Hq, heads, dqk, dv = (128, 1, 576, 512) if latent else (8, 2, 128, 128)
    c = _case(11, 3, Hq, heads, dqk, dv, latent, 70, [256, 256, 256], [200, 200, 200])
    c["table"][0, 5] = -1                       # a window chunk without a slot
    c["table"][1, 1] = len(c["kp"]) + 4         # a top-k chunk with one outside the pool
    st = status()
    out, lse = _run(L, c, st=st)
    assert st.item() == L.DEV_TABLE
    _check(c, out, lse)
    c["topk"][2, 3] = -7
    c["topk"][2, 4] = 64 * c["table"].shape[1] + 1
    st.zero_()
    out, lse = _run(L, c, st=st)
    assert st.item() == L.DEV_TABLE | L.DEV_INDEX
    _check(c, out, lse)
    c["start"][0] = -64                         # no window at all
    out, lse = _run(L, c, st=st)
    _check(c, out, lse)
    c["start"][:], c["count"][:] = -64, 0       # nothing anywhere
    st.zero_()
    out, lse = _run(L, c, st=st)
    assert st.item() == L.DEV_INDEX
    _check(c, out, lse)


@pytest.mark.parametrize("latent", [False, True])
def test_attention_all_equal_rows_and_growing_maximum(L, latent):
    """Scores that grow along the sequence move the reference maximum many times."""
    Hq, heads, dqk, dv = (70, 1, 576, 512) if latent else (5, 1, 128, 128)
    c = _case(13, 1, Hq, heads, dqk, dv, latent, 0, [0], [2048], shift=1.0)
    kp = np.zeros((len(c["kp"]), 1, CH, dqk))
    order = {int(s): i for i, s in enumerate(c["table"][0]) if s >= 0}
    for s, i in order.items():
        kp[s, 0] = (np.arange(CH)[:, None] + CH * i) / 2048.0 * 6.0
    c["kp"] = R.pack(*R.quantise(kp))
    c["q"] = torch.full_like(c["q"], 1.0)
    out, lse = _run(L, c)
    _check(c, out, lse)


@pytest.mark.parametrize("latent", [False, True])
def test_attention_in_graphs_and_on_streams(L, latent):
    """Two captured graphs with workspaces of their own, replayed on two streams at once, give what eager
    calls give, bit for bit; and so does a side stream."""
    Hq, heads, dqk, dv = (128, 1, 576, 512) if latent else (16, 2, 128, 128)
    cs = [_case(20 + i, 3, Hq, heads, dqk, dv, latent, 64, [640, 0, 64], [500 + 64 * i, 1, 900]) for i in range(2)]
    dev = [dict(q=c["q"].cuda(), kp=cu(c["kp"]), vp=None if latent else cu(c["vp"]), table=cu(c["table"]),
                topk=cu(c["topk"]), count=cu(c["count"]), start=cu(c["start"]), length=cu(c["length"])) for c in cs]

    def call(d, **kw):
        return L.sparse_decode_q4(d["q"], d["kp"], d["vp"], d["table"], d["topk"], d["count"], d["start"], d["length"],
                                  1000, dv, 0.1, **kw)
    eager = [call(d) for d in dev]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = call(dev[0], stream=side)
    side.synchronize()
    assert torch.equal(out[0], eager[0][0]) and torch.equal(out[1], eager[0][1])
    graphs, results = [], []
    for d in dev:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            results.append(call(d))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for r, e in zip(results, eager):
        assert torch.equal(r[0], e[0]) and torch.equal(r[1], e[1])


def test_latent_wait_that_runs_out(L):
    """The failure path: a wait on a barrier nothing arrives on returns with LSA_DEV_TIMEOUT, and the
    next call is as if nothing had happened."""
    c = _case(31, 2, 128, 1, 576, 512, True, 64, [640, 128], [700, 900])
    good = _run(L, c)
    st = status()
    L.test_stall_next_wait(L.TEST_STALL_ATTENTION_Q4)
    _run(L, c, st=st)
    torch.cuda.synchronize()
    assert st.item() & L.DEV_TIMEOUT
    st.zero_()
    again = _run(L, c, st=st)
    assert st.item() == 0
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


def test_latent_tails_with_cold_caches(L):
    """One to five tiles a split, gathered rows first or last, nothing in the caches: the kernel's warps reach its
    end far apart, and no wait may run out."""
    flush = torch.empty(2 ** 26, dtype=torch.int32, device="cuda")
    for n, (k, n_seq) in enumerate([(0, 74), (64, 74), (200, 74), (0, 37)]):
        rng = np.random.default_rng(n)
        starts = rng.integers(0, 400, n_seq) * (k > 0)
        lengths = rng.integers(0, 640, n_seq)
        c = _case(50 + n, n_seq, 128, 1, 576, 512, True, k, starts, lengths)
        st, first = status(), None
        for _ in range(4):
            flush.zero_()
            out, lse = _run(L, c, st=st)
            first = first or (out, lse)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        assert st.item() == 0
        _check(c, *first)


@pytest.mark.parametrize("Hq,heads,dqk,dv,latent", [(8, 2, 128, 128, False), (8, 1, 64, 64, False), (128, 1, 576, 512, True)])
def test_windows_longer_than_their_table_row(L, Hq, heads, dqk, dv, latent):
    """Rows behind the table row's last chunk do not exist: they are flagged and cost nothing, however many are asked for."""
    c = _case(71, 5, Hq, heads, dqk, dv, latent, 64, [64, 128, 0, 64 * 9, 192], [300, 200, 5, 1, 100])
    end = 64 * c["table"].shape[1]
    c["table"][c["table"] < 0] = c["table"][0, 0]          # the spare chunk has a slot
    real = dict(c, length=c["length"].copy(), start=c["start"].copy())
    c["length"][0], real["length"][0] = 2 ** 31 - 1, end - 64
    c["length"][1], real["length"][1] = end, end - 128
    c["start"][3], c["length"][3], real["length"][3] = 2 ** 31 - 1, 2 ** 31 - 1, 0
    c["start"][4], c["length"][4], real["length"][4] = end, 70, 0
    for name in ("kp", "vp"):        # rows that only the longer windows have hold NaN scales: give them values
        if c[name] is not None:
            codes, scales = (a.copy() for a in R.unpack(c[name]))
            scales[scales == 0x7f] = 0x30
            c[name][...] = R.pack(codes, scales)
    st = status()
    out, lse = L.sparse_decode_q4(c["q"].cuda(), cu(c["kp"]), None if latent else cu(c["vp"]), cu(c["table"]), cu(c["topk"]),
                                  cu(c["count"]), cu(c["start"]), cu(c["length"]), end, dv, c["scale"], status=st)
    assert st.item() == L.DEV_TABLE
    _check(dict(real, kp=c["kp"], vp=c["vp"]), out, lse)


@pytest.mark.parametrize("Hq,heads,dqk,dv,latent", [(8, 2, 128, 128, False), (40, 1, 64, 64, False), (16, 1, 576, 512, True)])
def test_many_short_sequences(L, Hq, heads, dqk, dv, latent):
    """More sequences than a block has threads, most of them empty or a few rows long, some with top-k rows alone."""
    rng = np.random.default_rng(Hq)
    B = 700
    starts = rng.integers(0, 3, B) * rng.integers(0, 100, B)
    lengths = rng.integers(0, 2, B) * rng.integers(0, 90, B)
    starts[300:430] = lengths[300:430] = 0                     # a whole stretch of nothing
    lengths[699] = 700
    c = _case(81, B, Hq, heads, dqk, dv, latent, 30, starts, lengths)
    st = status()
    out, lse = _run(L, c, st=st)
    assert st.item() == 0
    _check(c, out, lse)


@pytest.mark.parametrize("heads,dqk,dv,latent", [(8, 128, 128, False), (1, 576, 512, True)])
def test_pools_past_32_bits(L, heads, dqk, dv, latent):
    """Slots behind the first 4 GiB of a pool, and rows 2^31 elements apart, give what a small pool gives, bit for bit."""
    n_big = 2 ** 32 // (heads * 36 * dqk) + 40
    rng = np.random.default_rng(5)
    T = 150
    # rows more than 2^31 elements apart: three tokens of one buffer
    wide = torch.zeros(2 ** 31 + 2 ** 21, dtype=torch.bfloat16, device="cuda")
    rows = wide.as_strided((3, heads, dqk), (2 ** 30, dqk, 1))
    rows.copy_(torch.from_numpy(rng.standard_normal((3, heads, dqk))))
    k = torch.from_numpy(rng.standard_normal((T, heads, dqk))).to("cuda", torch.bfloat16)
    k[:3] = rows
    v = None if latent else torch.from_numpy(rng.standard_normal((T, heads, dv))).to("cuda", torch.bfloat16)
    q = torch.from_numpy(rng.standard_normal((1, 16, dqk))).to("cuda", torch.bfloat16)
    got = []
    for n_slots, first in ((5, 1), (n_big, n_big - 4)):
        kp = L.q4_pool(n_slots, heads, dqk)
        vp = None if latent else L.q4_pool(n_slots, heads, dv)
        table = torch.arange(first, first + 4, dtype=torch.int32, device="cuda")[None]
        slots = first * CH + torch.arange(T, device="cuda")
        st = status()
        L.write_q4(k, kp, slots, v=v, v_pool=vp, status=st)
        L.write_q4(rows, kp, slots[:3].clone(), status=st)     # the same values again, from far apart
        start, length = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (0, T))
        L.append_token_q4(k[7:8].contiguous(), None if latent else v[7:8].contiguous(), None, kp, vp, None, table, start,
                          length, status=st)
        topk = torch.tensor([[3, 70, 149]], dtype=torch.int32, device="cuda")
        out, lse = L.sparse_decode_q4(q, kp, vp, table, topk, torch.tensor([3], dtype=torch.int32, device="cuda"), start,
                                      length, T + 1, dv, 0.05, status=st)
        back = L.read_q4(kp, torch.cat([slots, slots[-1:] + 1]), status=st)
        assert st.item() == 0 and length.item() == T + 1
        got.append((out, lse, back))
        del kp, vp
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(got[0][2][7], got[0][2][T])
