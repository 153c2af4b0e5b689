"""The serving operators run together as a server runs them: chunk tables from the requests' lengths, norm and rotation of
the new tokens' rows, 4-bit rows written through the slot map, attention over the whole contexts; and lookahead
windows over 4-bit pools.  Every stage is compared with its 64-bit reference on the inputs that the
stage before it really produced; bounds are those of the stages' own tests."""
import numpy as np
import pytest
import torch

from tests import q4_reference as R
from tests.test_gpu_q4 import _check as check_attention
from tests.test_gpu_q4 import _rows, cu
from tests.test_gpu_tables_rope import _check_rows as check_rotation

pytestmark = pytest.mark.gpu
CH = 64
INV = {64: (10000.0 ** (-np.arange(32) / 32)).astype(np.float32), 128: (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)}


@pytest.fixture(scope="module")
def L():
    from learned_sparse_kv_b200 import lsa
    return lsa


class Server:
    """Device state of B requests; step() makes the calls of one model layer."""

    def __init__(self, L, latent, B=4, n_slots=24, stride=7, max_new=210, seed=0):
        self.L, self.latent, self.B, self.n_slots, self.max_new = L, latent, B, n_slots, max_new
        self.Hq, self.heads, self.dqk, self.dv = (16, 1, 576, 512) if latent else (8, 2, 128, 128)
        rng = np.random.default_rng(seed)
        self.k_width = 512 if latent else 128
        self.wk = torch.from_numpy(1 + 0.2 * rng.standard_normal(self.k_width)).to("cuda", torch.bfloat16)
        self.wq = None if latent else torch.from_numpy(1 + 0.2 * rng.standard_normal(128)).to("cuda", torch.bfloat16)
        self.rot_offset, self.inv = (512, INV[64]) if latent else (0, INV[128])
        self.inv_dev = cu(self.inv)
        self.table = torch.full((B, stride), -1, dtype=torch.int32, device="cuda")
        self.cached = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.start = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.kp = L.q4_pool(n_slots, self.heads, self.dqk)
        self.vp = None if latent else L.q4_pool(n_slots, self.heads, self.dv)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def inputs(self, rng, new):
        """Rows of the new tokens in order; NaN behind them, which nothing may read into a result."""
        def make(h, w):
            x = torch.full((self.max_new, h, w), float("nan"))
            x[:sum(new)] = torch.from_numpy(rng.standard_normal((sum(new), h, w)))
            return x.to("cuda", torch.bfloat16)
        return dict(q=make(self.Hq, self.dqk), k=make(self.heads, self.dqk),
                    v=None if self.latent else make(self.heads, self.dv), new=cu(np.array(new, np.int32)))

    def step(self, x, max_len):
        L, o = self.L, {}
        o["table"], o["slots"], o["position"], o["offset"], o["n_free"] = L.build_tables(
            self.table, self.cached, x["new"], self.n_slots, self.max_new, status=self.status)
        o["q"], o["k"] = L.qk_norm_rope(x["q"], x["k"], o["position"], self.inv_dev, q_weight=self.wq, k_weight=self.wk,
                                        rot_offset=self.rot_offset, interleaved=self.latent)
        L.write_q4(o["k"], self.kp, o["slots"], v=x["v"], v_pool=self.vp, k_scale=0.5, v_scale=0.25, status=self.status)
        self.table.copy_(o["table"])
        self.cached.add_(x["new"])
        last = (o["offset"][1:] - 1).clamp(min=0).long()       # each request's last token
        o["last"] = o["q"][last]
        o["out"], o["lse"] = L.sparse_decode_q4(o["last"], self.kp, self.vp, self.table, None, None, self.start,
                                                self.cached, max_len, self.dv, 0.07, k_scale=0.5, v_scale=0.25,
                                                status=self.status)
        return o


STEPS = [[130, 1, 0, 64], [1, 1, 1, 1], [1, 62, 1, 0], [5, 1, 200, 1], [0, 0, 0, 0], [1, 1, 1, 1]]


@pytest.mark.parametrize("latent", [False, True])
def test_requests_that_grow(L, latent):
    """A ragged prefill, single tokens that end and begin chunks, a late long request, a step with nothing new."""
    s, rng = Server(L, latent), np.random.default_rng(1)
    table, cached = s.table.cpu().numpy(), np.zeros(s.B, np.int64)
    pool_bytes = s.kp.cpu().numpy()
    for new in STEPS:
        x = s.inputs(rng, new)
        o = s.step(x, 400)
        T = sum(new)
        for name, ref in zip(("table", "slots", "position", "offset", "n_free"),
                             R.tables(table, cached, np.array(new), s.n_slots, s.max_new)):
            np.testing.assert_array_equal(o[name].cpu().numpy(), ref, err_msg=name)
        table, cached = o["table"].cpu().numpy(), cached + new
        pos, slots = o["position"].cpu().numpy()[:T], o["slots"].cpu().numpy()[:T]
        if T:
            args = (pos, s.inv, s.rot_offset, latent, 1e-6)
            check_rotation(o["q"][:T], x["q"][:T], s.wq, 0 if latent else 128, *args, np.zeros((T, s.Hq, s.dqk)), torch.bfloat16)
            check_rotation(o["k"][:T], x["k"][:T], s.wk, s.k_width, *args, np.zeros((T, s.heads, s.dqk)), torch.bfloat16)
        codes, scales = (a.copy() for a in R.unpack(pool_bytes))
        qc, qs = R.quantise(o["k"][:T].double().cpu().numpy(), 0.5)
        codes[slots // CH, :, slots % CH], scales[slots // CH, :, slots % CH] = qc, qs
        pool_bytes = s.kp.cpu().numpy()
        np.testing.assert_array_equal(pool_bytes, R.pack(codes, scales))
        assert s.status.item() == 0
        c = dict(q=o["last"].cpu(), kp=pool_bytes, vp=None if latent else s.vp.cpu().numpy(), table=table, topk=None,
                 count=np.zeros(s.B, np.int32), start=np.zeros(s.B, np.int32), length=cached.astype(np.int32), dv=s.dv,
                 scale=0.07)
        if np.isfinite(c["q"].float().numpy()).all():
            check_attention(c, o["out"], o["lse"], 0.5, 0.5 if latent else 0.25)
        else:
            assert not any(new)        # nothing new: the gathered query row is padding


@pytest.mark.parametrize("latent", [False, True])
def test_captured_steps_of_two_servers(L, latent):
    """The whole step captured once for each of two servers and replayed on two streams at once, with lengths and rows
    that change between replays, gives what eager calls give, bit for bit."""
    eager, live = ([Server(L, latent, seed=i) for i in range(2)] for _ in range(2))
    rng = np.random.default_rng(2)
    first = [s.inputs(rng, STEPS[0]) for s in eager]
    for s, x in zip(eager, first):
        s.step(x, 400)
    graphs = []
    for s, x in zip(live, first):
        s.step(x, 400)
        buf = {k: None if v is None else v.clone() for k, v in x.items()}
        keep = [t.clone() for t in (s.table, s.cached, s.kp)] + ([] if latent else [s.vp.clone()])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = s.step(buf, 400)
        for t, k in zip((s.table, s.cached, s.kp, s.vp), keep):
            assert torch.equal(t, k)                  # capturing runs nothing
        graphs.append((g, buf, o, torch.cuda.Stream()))
    for new in STEPS[1:]:
        xs = [s.inputs(rng, new) for s in eager]
        refs = [s.step(x, 400) for s, x in zip(eager, xs)]
        for (g, buf, o, st), x in zip(graphs, xs):
            for name, t in x.items():
                if t is not None:
                    buf[name].copy_(t)
            st.wait_stream(torch.cuda.current_stream())
        for g, buf, o, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (g, buf, o, st), ref in zip(graphs, refs):
            for name in ("table", "slots", "position", "offset", "n_free"):
                assert torch.equal(o[name], ref[name]), name
            T = sum(new)
            assert torch.equal(o["q"][:T], ref["q"][:T]) and torch.equal(o["k"][:T], ref["k"][:T])
            if T:
                assert torch.equal(o["out"], ref["out"]) and torch.equal(o["lse"], ref["lse"])
        for a, b in zip(eager, live):
            assert torch.equal(a.kp, b.kp) and torch.equal(a.table, b.table)
    assert all(s.status.item() == 0 for s in eager + live)


def test_calls_on_a_side_stream(L):
    """Each call with stream=: the work is ordered on that stream, and results are the same."""
    a, b = Server(L, False), Server(L, False)
    rng = np.random.default_rng(3)
    x = a.inputs(rng, STEPS[0])
    o = a.step(x, 400)
    back = L.read_q4(a.kp, o["slots"], scale=0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    table, slots, position, offset, n_free = L.build_tables(b.table, b.cached, x["new"], b.n_slots, b.max_new, stream=side)
    q, k = L.qk_norm_rope(x["q"], x["k"], position, b.inv_dev, q_weight=b.wq, k_weight=b.wk, stream=side)
    L.write_q4(k, b.kp, slots, v=x["v"], v_pool=b.vp, k_scale=0.5, v_scale=0.25, stream=side)
    got = L.read_q4(b.kp, slots, scale=0.5, stream=side)
    new_k, new_v = (torch.ones(4, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wl = x["new"].clone()
    side.wait_stream(torch.cuda.current_stream())
    L.append_token_q4(new_k, new_v, None, b.kp, b.vp, None, table, b.start, wl, stream=side)
    side.synchronize()
    for u, v in ((table, o["table"]), (slots, o["slots"]), (offset, o["offset"]), (q[:195], o["q"][:195]), (got, back)):
        assert torch.equal(u, v)
    # requests 0, 1 and 3 hold chunks; 2 has none, 3's second does not exist: 64 tokens fill its first
    np.testing.assert_array_equal(wl.cpu().numpy(), np.array(STEPS[0]) + [1, 1, 0, 0])


@pytest.mark.parametrize("name,over", [("decode_16k_b1_h16", {}), ("decode_128k_b8_mla", dict(B=2, ctx=(16384, 9600), pass_rate=(0.135, 0.135)))])
def test_windows_over_4bit_pools(L, name, over):
    """Lookahead windows whose pools are 4-bit: every step attends its top-k rows and its window, the appended tokens
    included, as the reference does on the pools' own bytes."""
    import lsa_workloads as W
    from learned_sparse_kv_b200.decode import Shapes, Window
    from lsa_workloads.device import host_build, upload
    wl = W.workload(name, steps=3, **over)
    shapes, t, max_ch, kept_cap, cold = upload(host_build(wl), torch.device("cuda:0"))
    sh = Shapes(**shapes)
    for key in (("kv",) if sh.latent else ("k", "v")):
        rows = t[key]
        n, w = rows.shape[0], rows.shape[-1]
        pool = L.q4_pool(n, 1, w)
        L.write_q4(rows.reshape(n * CH, w), pool, torch.arange(n * CH, device="cuda"), k_scale=0.5)
        t[key] = pool
    t["k_scale"] = t["v_scale"] = 0.5
    win = Window(sh, t, max_ch, kept_cap)
    win.capture()
    win.run()
    torch.cuda.synchronize()
    assert win.device_status() == 0
    table, start = t["chunk_table"].cpu().numpy(), t["window_start"].cpu().numpy()
    kp, vp = win.k_pool.cpu().numpy(), None if sh.latent else win.v_pool.cpu().numpy()
    for s in range(sh.steps):
        c = dict(q=t["q"][s].cpu(), kp=kp, vp=vp, table=table, topk=win.topk_w[0, s].cpu().numpy(),
                 count=win.topk_count_w[0, s].cpu().numpy(), start=start,
                 length=np.full(sh.B, sh.window + s + 1, np.int32), dv=sh.dv, scale=sh.scale)
        check_attention(c, win.out_w[0, s], win.lse_w[0, s], 0.5, 0.5)
        new = t["new_kv" if sh.latent else "new_k"][s].double().cpu().numpy()
        codes, scales = R.unpack(kp)
        for b in range(sh.B):
            pos = int(start[b]) + sh.window + s
            slot, row = table[b, pos // CH], pos % CH
            qc, qs = R.quantise(new[b:b + 1], 0.5)
            np.testing.assert_array_equal(codes[slot, :, row], qc)
            np.testing.assert_array_equal(scales[slot, :, row], qs)
