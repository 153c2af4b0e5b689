"""GPU parity of the chunk tables and of the norm with rotation with a 64-bit reference.

Tables are whole numbers and must be equal.  The norm and rotation are fp32 with one rounding at
the end: with u = 2^-24, the sum of squares of n terms, its root and the products leave a relative error of
at most (n / 2 + 6) u on a normalised value x, sine and cosine an absolute error of 4 u each
(the angle is reduced in 64 bits), so a turned pair (x, y) is off by at most
  (n / 2 + 12) u (|x| + |y|), plus half a step of the rows' type.
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


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ tables --

def _tables(L, table, cached, new, n_slots, max_new):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = L.build_tables(cu(table), cu(np.array(cached, np.int32)), cu(np.array(new, np.int32)), n_slots, max_new, status=st)
    ref = R.tables(table, np.array(cached, np.int64), np.array(new, np.int64), n_slots, max_new)
    for name, g, r in zip(("table", "slot_map", "position", "offset", "n_free"), got, ref):
        np.testing.assert_array_equal(g.cpu().numpy(), r, err_msg=name)
    return st.item(), got


def _table(rng, cached, stride, n_slots):
    """Distinct slots for the cached chunks; left-over entries behind them."""
    B = len(cached)
    table = rng.integers(-1, n_slots, (B, stride)).astype(np.int32)
    perm, at = rng.permutation(n_slots).astype(np.int32), 0
    for b, c in enumerate(cached):
        n = -(-c // CH)
        table[b, :n] = perm[at:at + n]
        at += n
    return table


@pytest.mark.parametrize("B,stride,hi_cached,hi_new,n_slots", [
    (1, 1, 1, 63, 1), (1, 5, 300, 20, 7), (3, 9, 250, 200, 40), (32, 65, 4000, 1, 2100), (300, 17, 900, 100, 5200),
    (1500, 4, 120, 60, 4600), (7, 2000, 120000, 500, 15001), (2, 40, 1, 2400, 100001),
    (5000, 3, 60, 60, 11000), (300, 7100, 2000, 40, 9900)])      # the last two: more than one cluster takes
def test_tables_exact(L, B, stride, hi_cached, hi_new, n_slots):
    rng = np.random.default_rng(B + stride)
    cached = rng.integers(0, hi_cached + 1, B)
    new = rng.integers(0, hi_new + 1, B)
    cached[rng.random(B) < 0.2] = 0
    new[rng.random(B) < 0.2] = 0
    table = _table(rng, cached, stride, n_slots)
    st, _ = _tables(L, table, cached, new, n_slots, int(new.sum()) + 5)
    assert st == 0


def test_tables_lengths_at_the_borders(L):
    cached = [0, 0, 1, 63, 64, 65, 127, 128, 0, 64, 320]
    new = [0, 1, 63, 1, 0, 64, 1, 1, 128, 64, 0]
    rng = np.random.default_rng(0)
    st, _ = _tables(L, _table(rng, cached, 5, 40), cached, new, 40, sum(new))
    assert st == 0
    st, _ = _tables(L, _table(rng, [0, 0], 5, 8), [0, 0], [0, 0], 8, 0)
    assert st == 0


def test_tables_shared_prefix_and_step_by_step(L):
    """A full chunk may be shared; decode steps fed with the previous step's table keep every slot."""
    table = np.full((3, 4), -1, np.int32)
    table[0, :2], table[1, :2] = [5, 2], [5, 3]
    cached, new = np.array([100, 128, 0]), np.array([1, 1, 1])
    for _ in range(70):
        st, got = _tables(L, table, cached, new, 8, 3)
        assert st == 0
        before, table = table, got[0].cpu().numpy()
        kept = np.arange(4)[None] < (-(-cached // CH))[:, None]
        np.testing.assert_array_equal(table[kept], before[kept])
        cached = cached + new
    assert (table[0, 0], table[1, 0]) == (5, 5)


def test_tables_report_what_does_not_fit(L):
    none = np.full((2, 3), -1, np.int32)
    st, got = _tables(L, none, [0, 0], [100, 100], 3, 200)       # 4 chunks, 3 slots
    assert st == L.DEV_CAPACITY and int((got[1] < 0).sum()) == 36
    st, _ = _tables(L, none, [0, 0], [10, 10], 3, 15)            # more tokens than entries
    assert st == L.DEV_CAPACITY
    st, _ = _tables(L, none, [0, 0], [193, 1], 9, 200)           # a request longer than its row
    assert st == L.DEV_CAPACITY
    st, _ = _tables(L, none, [0, -5], [10, -1], 9, 20)
    assert st == L.DEV_INDEX
    bad = none.copy()
    bad[0, 0], bad[1, 0] = 9, -1                                 # kept chunks without a valid slot
    st, _ = _tables(L, bad, [10, 10], [60, 1], 9, 61)
    assert st == L.DEV_TABLE
    st, _ = _tables(L, none, [2 ** 31 - 1, 5], [2 ** 31 - 1, 3], 9, 4)
    assert st & L.DEV_CAPACITY


def test_tables_in_a_graph(L):
    """A captured call replayed with other lengths in the same buffers."""
    rng = np.random.default_rng(2)
    cached = rng.integers(0, 500, 6)
    table = cu(_table(rng, cached, 12, 90))
    c, n = cu(cached.astype(np.int32)), cu(np.full(6, 1, np.int32))
    L.build_tables(table, c, n, 90, 40)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = L.build_tables(table, c, n, 90, 40)
    for step in range(3):
        new = rng.integers(0, 6, 6)
        cached = rng.integers(0, 500, 6)
        t = _table(rng, cached, 12, 90)
        table.copy_(cu(t)); c.copy_(cu(cached.astype(np.int32))); n.copy_(cu(new.astype(np.int32)))
        g.replay()
        for a, b in zip(got, R.tables(t, cached, new, 90, 40)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)


# --------------------------------------------------------- norm + rotation --

def _check_rows(out, x, weight, width, pos, inv, ro, inter, eps, before, dtype):
    rd = 2 * len(inv)
    xs = x.double().cpu().numpy()
    w = None if weight is None else weight.double().cpu().numpy()
    ref = R.norm_rope(xs, w, width, pos, inv, ro, inter, eps)
    flat = R.norm_rope(xs, w, width, np.zeros_like(pos), inv, ro, inter, eps)     # the norm alone
    size = np.abs(flat).copy()
    half = rd // 2
    i = np.arange(half)
    iu, iv = (ro + 2 * i, ro + 2 * i + 1) if inter else (ro + i, ro + half + i)
    both = np.abs(flat[..., iu]) + np.abs(flat[..., iv])
    size[..., iu] = both
    size[..., iv] = both
    tol = (x.shape[-1] / 2 + 12) * 2.0 ** -24 * size + EPS[dtype] * np.abs(ref) + 2.0 ** -24 * (dtype == torch.float16)
    got = out.double().cpu().numpy()
    live = pos >= 0
    bad = np.abs(got - ref)[live] > tol[live]
    assert not bad.any(), (int(bad.sum()), np.abs(got - ref)[live].max())
    np.testing.assert_array_equal(got[~live], before[~live])


CASES = [  # T, Hq, Hk, D, q_norm, k_norm, rot_offset, rot
    (1, 1, 1, 128, 128, 128, 0, 128), (5, 32, 8, 128, 128, 128, 0, 128), (3, 128, 1, 576, 0, 512, 512, 64),
    (130, 3, 1, 80, 80, 80, 0, 32), (7, 5, 2, 48, 0, 48, 24, 24), (600, 4, 4, 64, 64, 64, 0, 64),
    (9, 2, 3, 192, 0, 0, 128, 64), (4, 1, 1, 1024, 1024, 1024, 0, 1024), (4, 1, 1, 1022, 1000, 1022, 2, 1018),
    (6, 2, 1, 256, 256, 256, 0, 0), (2, 1, 1, 2, 2, 2, 0, 2), (11, 7, 0, 96, 50, 0, 0, 96), (3, 3, 1, 512, 512, 300, 100, 20)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hk,D,qn,kn,ro,rd", CASES)
def test_norm_rope(L, T, Hq, Hk, D, qn, kn, ro, rd, dtype, inter):
    rng = np.random.default_rng(D + T)
    fused = torch.from_numpy(rng.standard_normal((T, Hq + Hk, D))).to("cuda", dtype)
    q, k = fused[:, :Hq], fused[:, Hq:] if Hk else None           # views of one buffer
    wq = torch.from_numpy(1 + 0.2 * rng.standard_normal(qn)).to("cuda", dtype) if qn else None
    pos = rng.integers(0, 524288, T).astype(np.int32)
    pos[-1] = 0
    if T > 3:
        pos[1] = -1
    inv = (10000.0 ** (-np.arange(rd // 2) / max(rd // 2, 1))).astype(np.float32)
    qo, ko = (torch.full((T, h, D), 7.0, dtype=dtype, device="cuda") for h in (Hq, Hk))
    L.qk_norm_rope(q, k, cu(pos), cu(inv), q_weight=wq, k_weight=None, q_norm_width=qn, k_norm_width=kn, eps=1e-5,
                   rot_offset=ro, interleaved=inter, q_out=qo, k_out=ko if Hk else None)
    before = np.full((T, 1, D), 7.0)
    _check_rows(qo, q, wq, qn, pos, inv, ro, inter, 1e-5, np.broadcast_to(before, (T, Hq, D)), dtype)
    if Hk:
        _check_rows(ko, k, None, kn, pos, inv, ro, inter, 1e-5, np.broadcast_to(before, (T, Hk, D)), dtype)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_norm_rope_unaligned_rows_and_in_place(L, inter, offset):
    """Rows at any element offset and odd strides, head-major layouts, and outputs that are the inputs."""
    T, H, D = 33, 3, 64
    rng = np.random.default_rng(offset)
    buf = torch.from_numpy(rng.standard_normal(H * T * (D + 3) + offset)).to("cuda", torch.bfloat16)
    q = buf[offset:].view(H, T, D + 3)[:, :, :D].transpose(0, 1)       # [T, H, D], odd token stride
    x = q.clone()
    rest = buf[offset:].view(H, T, D + 3)[:, :, D:].clone()
    pos = rng.integers(0, 5000, T).astype(np.int32)
    inv = (1000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).to("cuda", torch.bfloat16)
    L.qk_norm_rope(q, None, cu(pos), cu(inv), q_weight=w, eps=1e-6, interleaved=inter, q_out=q)
    _check_rows(q, x, w, D, pos, inv, 0, inter, 1e-6, x.double().cpu().numpy(), torch.bfloat16)
    assert torch.equal(buf[offset:].view(H, T, D + 3)[:, :, D:], rest)


def test_norm_rope_special_rows(L):
    """A zero row (eps 0 gives NaN as the formula does), a huge row, nothing at all."""
    q = torch.zeros(3, 1, 64, device="cuda")
    q[1] = 1e18
    q[2, 0, 3] = float("inf")
    pos, inv = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    out, _ = L.qk_norm_rope(q, None, pos, inv, q_norm_width=64, eps=1e-6)
    assert torch.equal(out[0], torch.zeros_like(out[0]))
    torch.testing.assert_close(out[1], torch.ones_like(out[1]), rtol=1e-5, atol=0)
    assert bool(out[2].isnan().any())
    out, none = L.qk_norm_rope(q[:0], None, pos[:0], inv, q_norm_width=64)
    assert out.shape == (0, 1, 64) and none is None
