"""Calls on a side stream while the caller's stream still uses memory that was just freed there: what a call allocates
must not be that memory, and an output dropped while the caller's stream reads it must not be handed out."""
import pytest
import torch

pytestmark = pytest.mark.gpu
CH = 64
CYCLES = 100_000_000          # of the kernel that keeps the caller's stream busy, some 50 ms


@pytest.fixture(scope="module")
def L():
    from learned_sparse_kv_b200 import lsa
    return lsa


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _calls(L):
    """name -> (call, bytes of its workspace)."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, device="cuda", generator=g).to(dtype)
    B, T, n_slots = 2, 150, 8
    table = torch.arange(n_slots, dtype=torch.int32, device="cuda").view(B, 4)
    lens, new, start = ints(200, 130), ints(1, 40), ints(0, 0)
    kp, vp = L.q4_pool(n_slots, 2, 128), L.q4_pool(n_slots, 2, 128)
    slots = torch.arange(T, device="cuda")
    L.write_q4(rand(T, 2, 128), kp, slots, v=rand(T, 2, 128), v_pool=vp)
    q, k, pos = rand(T, 4, 128), rand(T, 2, 128), torch.arange(T, dtype=torch.int32, device="cuda")
    q_dec, inv = rand(B, 16, 128), torch.ones(64, device="cuda")
    kb, vb = rand(n_slots, CH, 128), rand(n_slots, CH, 128)
    topk, count = torch.arange(16, dtype=torch.int32, device="cuda").view(B, 8), ints(8, 8)
    parts, lse = rand(2, B, 4, 64, dtype=torch.float32), rand(2, B, 4, dtype=torch.float32)
    scores, off = rand(3000, dtype=torch.float32), torch.tensor([0, 1000, 3000], device="cuda")
    votes = torch.rand(3, 4, 500, device="cuda", generator=g)
    return {
        "build_tables": (lambda **s: L.build_tables(table, lens, new, 40, 64, **s), L.build_tables_workspace_size(B, 4, 40)),
        "qk_norm_rope": (lambda **s: L.qk_norm_rope(q, k, pos, inv, q_norm_width=128, k_norm_width=128, **s), 0),
        "read_q4": (lambda **s: (L.read_q4(kp, slots, **s),), 0),
        "sparse_decode_q4": (lambda **s: L.sparse_decode_q4(q_dec, kp, vp, table, topk, count, start, lens, 256, 128, 0.1, **s),
                             L.sparse_decode_q4_workspace_size(B, 16, 2, 128, 128, 8, 256)),
        "sparse_decode": (lambda **s: L.sparse_decode(q_dec, kb, vb, table, topk, count, start, lens, 256, 128, 0.1, **s),
                          L.sparse_decode_workspace_size(B, 16, 128, 128, 8, 256)),
        "merge_attention": (lambda **s: L.merge_attention(parts, lse, **s), 0),
        "topk_from_scores": (lambda **s: L.topk_from_scores(scores, off, 2000, 64, **s), 0),
        "label_vote": (lambda **s: L.label_vote(votes, **s), L.label_vote_workspace_size(3, 4, 500)),
    }


NAMES = ["build_tables", "qk_norm_rope", "read_q4", "sparse_decode_q4", "sparse_decode", "merge_attention",
         "topk_from_scores", "label_vote"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_in_use_on_the_callers_stream(L, name):
    call, ws = _calls(L)[name]
    ref = call()
    side = torch.cuda.Stream()
    sizes = sorted({t.nbytes for t in ref} | ({max(ws, 256)} if ws else set()))
    torch.cuda.synchronize()
    # blocks of every size that the call wants, read by kernels that have not started yet, and freed
    xs = [torch.ones(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    ys = [x + 1 for x in xs]
    del xs
    out = call(stream=side)
    torch.cuda.synchronize()
    assert all(bool((y == 2).all()) for y in ys)
    for a, b in zip(out, ref):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_dropped_while_the_callers_stream_reads_them(L, name):
    call, _ = _calls(L)[name]
    ref = call()
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    out = call(stream=side)
    main.wait_stream(side)
    torch.cuda._sleep(CYCLES)
    copies = [t.clone() for t in out]
    del out
    with torch.cuda.stream(side):          # blocks of the same sizes, overwritten at once
        junk = [torch.full((t.nbytes,), 0x55, dtype=torch.uint8, device="cuda") for t in ref for _ in range(8)]
    torch.cuda.synchronize()
    for a, b in zip(copies, ref):
        assert torch.equal(a, b)
    del junk


@pytest.mark.parametrize("name", NAMES)
def test_calls_on_a_side_stream_captured(L, name):
    """A capture that forks to a side stream and joins it again: replays give the eager call's bits."""
    call, _ = _calls(L)[name]
    ref = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        out = call(stream=side)
        main.wait_stream(side)
    for t in out:
        t.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, ref):
        assert torch.equal(a, b)
