"""Attention over 4-bit pools at the ends of its ranges: scores of any size, queries with an entry far above the others,
weights that a caller of fp32 output can rely on."""
import numpy as np
import pytest
import torch

from tests import q4_reference as R
from tests.test_gpu_q4 import _case, _check, _run, status

pytestmark = pytest.mark.gpu
CH = 64
SHAPES = [(8, 1, 128, 128, False), (16, 1, 128, 128, False), (12, 1, 64, 64, False), (128, 1, 576, 512, True)]


@pytest.fixture(scope="module")
def L():
    from learned_sparse_kv_b200 import lsa
    return lsa


def _one_column(c, column, top, q):
    """Key column `column` holds 6 at position `top` and 0.5 .. 4 elsewhere, in scales of one; queries are 0 but there."""
    codes, scales = (a.copy() for a in R.unpack(c["kp"]))
    group = slice(column // 16 * 16, column // 16 * 16 + 16)
    codes[..., group] = 0
    codes[..., column] = np.random.default_rng(1).integers(1, 7, codes.shape[:-1])
    scales[..., column // 16] = 0x38
    codes[c["table"][0, top // CH], :, top % CH, column] = 7
    c["kp"][...] = R.pack(codes, scales)
    c["q"] = torch.zeros_like(c["q"])
    c["q"][0, :, column] = q


@pytest.mark.parametrize("Hq,heads,dqk,dv,latent", SHAPES)
@pytest.mark.parametrize("n,top", [(300, 130), (3000, 2999), (64, 0)])
def test_scores_of_any_size(L, Hq, heads, dqk, dv, latent, n, top):
    """Scores of 2^9 to 2^100: one row has the largest by a third, so the output is its value row, exactly (a weight of a
    power of two over itself), and the lse is its score, whatever the roundings of the other scores are."""
    rng = np.random.default_rng(n)
    for lo, hi in ((9, 21), (21, 27), (27, 31), (31, 36), (36, 100)):
        c = _case(3, 1, Hq, heads, dqk, dv, latent, 0, [0], [n])
        mult = rng.integers(128, 256, Hq) / 128.0 * 2.0 ** rng.integers(lo, hi, Hq)
        _one_column(c, 3 if not latent else 560, top, torch.from_numpy(mult).bfloat16())
        c["scale"] = 1.0 / 6.0
        st = status()
        out, lse = _run(L, c, torch.float32, st=st)
        assert st.item() == 0
        vv = R.pool_values(c["kp"] if latent else c["vp"])[..., :dv]
        want = vv[c["table"][0, top // CH], 0, top % CH]
        got = out[0].double().cpu().numpy()
        wrong = [(h, got[h, 0], want[0]) for h in np.flatnonzero((got != want).any(-1))]
        assert not wrong, (lo, hi, len(wrong), wrong[:4])
        score = c["q"][0].double().numpy().max(-1)
        assert np.all(np.abs(lse[0].double().cpu().numpy() - score) <= 2.0 ** -21 * score)


@pytest.mark.parametrize("Hq,heads,dqk,dv,latent", SHAPES)
@pytest.mark.parametrize("dtype,power", [(torch.bfloat16, 20), (torch.bfloat16, 30), (torch.float16, 15)])
def test_queries_with_one_large_entry(L, Hq, heads, dqk, dv, latent, dtype, power):
    """One query entry of 2^power beside ordinary ones of 1/4 and more, over a key column of zeros: what is left of the
    scores is the ordinary entries', whose f16 images are exact (2^-32 of the largest or more).  So the bounds are
    those of test_gpu_q4 without its term for query entries below f16's range."""
    c = _case(17, 2, Hq, heads, dqk, dv, latent, 70, [128, 100], [300, 65], dtype=torch.float32)
    column = 5
    codes, scales = (a.copy() for a in R.unpack(c["kp"]))
    codes[..., column] &= 8
    c["kp"][...] = R.pack(codes, scales)
    q = c["q"]
    q = torch.sign(q) * q.abs().clamp(min=0.25)
    q[..., column] = 2.0 ** power
    c["q"] = q.to(dtype)
    out, lse = _run(L, c, torch.float32)
    kv = R.pool_values(c["kp"])
    vv = None if latent else R.pool_values(c["vp"])
    o, s = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(2):
        rows = R.row_set(b, c["table"], c["topk"], c["count"], c["start"], c["length"], len(c["kp"]))
        ro, rl, spread, mag, flat = R.attend(c["q"][b].double().numpy(), kv, vv, dv, rows, c["scale"])
        D = (dqk + 32) * 2.0 ** -23 * mag
        tol = (2.0 ** -11 + 2 * D[:, None] + 2.0 ** -20 + len(rows) * 2.0 ** -24) * spread + 2.0 ** -24 * np.abs(ro) + 2.0 ** -31 * flat
        assert np.all(np.abs(o[b] - ro) <= tol), (b, float((np.abs(o[b] - ro) / tol).max()))
        assert np.all(np.abs(s[b] - rl) <= D + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl)), b


@pytest.mark.parametrize("Hq,heads,dqk,dv,latent", SHAPES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("n", [2, 17, 67, 200])
def test_weights_of_f16_and_fp32_outputs(L, Hq, heads, dqk, dv, latent, out_dtype, n):
    """Scores that are exact products (one key column, one query entry) leave the weights' own error: 2^-22 for the two
    parts, 2^-20 for the exponential and its argument, n 2^-24 for the sums, of sum_j p_j |v_j|; 2^-31 of the largest
    weight where a weight is below f16's normal range (see test_gpu_q4); and the rounding of the result."""
    rng = np.random.default_rng(n)
    c = _case(23, 1, Hq, heads, dqk, dv, latent, 0, [0], [n])
    _one_column(c, 3 if not latent else 560, n // 2, torch.from_numpy(rng.uniform(0.1, 1.5, Hq)).bfloat16())
    c["scale"] = 0.25
    out, lse = _run(L, c, out_dtype)
    kv = R.pool_values(c["kp"])
    vv = None if latent else R.pool_values(c["vp"])
    rows = R.row_set(0, c["table"], c["topk"], c["count"], c["start"], c["length"], len(c["kp"]))
    ro, rl, spread, _, flat = R.attend(c["q"][0].double().numpy(), kv, vv, dv, rows, c["scale"])
    tol = (2.0 ** -22 + 2.0 ** -20 + n * 2.0 ** -24) * spread + torch.finfo(out_dtype).eps / 2 * np.abs(ro) + 2.0 ** -31 * flat
    tol += 2.0 ** -25 * (out_dtype == torch.float16)            # half a step of f16's subnormals
    off = np.abs(out[0].double().cpu().numpy() - ro) / tol.clip(1e-300)
    assert off.max() <= 1, (float(off.max()), int((off > 1).sum()))
    assert np.all(np.abs(lse[0].double().cpu().numpy() - rl) <= 2.0 ** -20 + 2.0 ** -22 * np.abs(rl))


def test_a_launch_longer_than_any_wait(L):
    """Latent rows of one sequence for some two seconds, on one pair of CTAs beside 37 short ones: a launch may last longer
    than the bound of a single wait, and no wait runs out.  The table names one chunk over and over: every row counts
    2^21 times, so the output is that of the chunk alone and its lse is larger by 21 log 2 (fp32 sums of 2^20 terms, each
    off by at most 2^-24 of the sum: 2^-4)."""
    n_ch, B = 2 ** 21, 38
    rng = np.random.default_rng(4)
    rows = torch.from_numpy(rng.standard_normal((CH, 1, 576))).to("cuda", torch.bfloat16)
    pool = L.q4_pool(1, 1, 576)
    L.write_q4(rows, pool, torch.arange(CH, device="cuda"))
    q = torch.from_numpy(rng.standard_normal((1, 16, 576))).to("cuda", torch.bfloat16).repeat(B, 1, 1)
    table = torch.zeros(B, n_ch, dtype=torch.int32, device="cuda")
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    length = torch.full((B,), CH, dtype=torch.int32, device="cuda")
    length[0] = n_ch * CH
    st = status()
    out, lse = L.sparse_decode_q4(q, pool, None, table, None, None, start, length, n_ch * CH, 512, 0.04, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert torch.equal(out[1:], out[1:2].expand(B - 1, -1, -1))
    assert float((lse[0] - lse[1] - 21 * np.log(2)).abs().max()) <= 2.0 ** -4
    assert bool(torch.isfinite(out[0]).all())


@pytest.mark.parametrize("Hq,heads,dqk,dv,latent", SHAPES)
def test_every_negative_index_is_flagged(L, Hq, heads, dqk, dv, latent):
    """The smallest 32-bit integer among the top-k indices is skipped and flagged like any other negative one."""
    c = _case(29, 2, Hq, heads, dqk, dv, latent, 70, [128, 100], [300, 65])
    for bad in (-1, -2 ** 31):
        c["topk"][1, 3] = bad
        st = status()
        out, lse = _run(L, c, st=st)
        assert st.item() == L.DEV_INDEX, bad
        _check(c, out, lse)


def test_latent_two_part_tails_with_cold_caches(L):
    """fp32 results (weights in two parts): one to five tiles a split, gathered rows first or last, nothing in the caches; no
    wait runs out and every run gives the same bits."""
    flush = torch.empty(2 ** 26, dtype=torch.int32, device="cuda")
    for n, (k, n_seq) in enumerate([(0, 74), (64, 74), (200, 74), (0, 37)]):
        rng = np.random.default_rng(n)
        starts = rng.integers(0, 400, n_seq) * (k > 0)
        lengths = rng.integers(0, 640, n_seq)
        c = _case(50 + n, n_seq, 128 if n % 2 else 64, 1, 576, 512, True, k, starts, lengths)
        st, first = status(), None
        for _ in range(4):
            flush.zero_()
            out, lse = _run(L, c, torch.float32, st=st)
            first = first or (out, lse)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        assert st.item() == 0
        _check(c, *first)


@pytest.mark.parametrize("Hq,heads,dqk,dv,latent", [(5, 1, 128, 128, False), (70, 1, 576, 512, True)])
def test_two_parts_under_a_growing_maximum(L, Hq, heads, dqk, dv, latent):
    """Scores that grow along the sequence: both parts of the weights follow the same reference."""
    c = _case(13, 1, Hq, heads, dqk, dv, latent, 0, [0], [2048])
    kp = np.zeros((len(c["kp"]), 1, CH, dqk))
    for i, s in enumerate(c["table"][0]):
        if s >= 0:
            kp[s, 0] = (np.arange(CH)[:, None] + CH * i) / 2048.0 * 6.0
    c["kp"] = R.pack(*R.quantise(kp))
    c["q"] = torch.full_like(c["q"], 1.0)
    for dtype in (torch.float32, torch.float16):
        _check(c, *_run(L, c, dtype))


def test_two_part_wait_that_runs_out(L):
    """The failure path with fp32 results: LSA_DEV_TIMEOUT, and the next call gives the bits of the one before."""
    c = _case(31, 2, 128, 1, 576, 512, True, 64, [640, 128], [700, 900])
    good = _run(L, c, torch.float32)
    st = status()
    L.test_stall_next_wait(L.TEST_STALL_ATTENTION_Q4)
    _run(L, c, torch.float32, st=st)
    torch.cuda.synchronize()
    assert st.item() & L.DEV_TIMEOUT
    st.zero_()
    again = _run(L, c, torch.float32, st=st)
    assert st.item() == 0
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
