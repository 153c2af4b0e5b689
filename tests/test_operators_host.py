"""Refusals of the table, norm + rotation and 4-bit entry points, before anything is launched (no GPU needed)."""
import ctypes as C

import pytest

from learned_sparse_kv_b200 import build as lbuild
from learned_sparse_kv_b200 import lsa

P, U = 4096, 4096 + 2     # never dereferenced: the calls fail validation first


@pytest.fixture(scope="module", autouse=True)
def built():
    lbuild.build()


def refused(rc, code, words):
    assert rc == code, (rc, lsa._lib.lsa_last_error())
    assert words in lsa._lib.lsa_last_error().decode()


def tables(**kw):
    a = dict(table=P, stride=4, cached=P, new=P, B=2, n_slots=8, max_new=4, nxt=P + 64, sm=P, pos=P, off=P, free=P,
             st=None, ws=P, nws=1 << 20)
    a.update(kw)
    return lsa._lib.lsa_build_tables(*a.values(), None)


@pytest.mark.parametrize("kw,code,words", [
    (dict(B=0), 1, "bad sizes"), (dict(B=65536), 1, "bad sizes"), (dict(stride=0), 1, "bad sizes"),
    (dict(n_slots=0), 1, "bad sizes"), (dict(n_slots=1 << 31), 1, "bad sizes"), (dict(max_new=-1), 1, "bad sizes"),
    (dict(table=None), 1, "null"), (dict(sm=None), 1, "null"), (dict(nxt=P), 1, "must not be table"),
    (dict(nws=16), 7, "workspace")])
def test_tables_refusals(kw, code, words):
    refused(tables(**kw), code, words)


def rope(**kw):
    a = dict(dtype=0, T=4, D=64, q=P, qts=64, qhs=64, Hq=1, qw=None, qn=64, qo=P, qots=64, qohs=64, k=None, kts=0, khs=0,
             Hk=0, kw=None, kn=0, ko=None, kots=0, kohs=0, eps=1e-6, pos=P, inv=P, ro=0, rd=64, inter=0)
    a.update(kw)
    return lsa._lib.lsa_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code,words", [
    (dict(dtype=3), 1, "dtype"), (dict(T=-1), 1, "bad sizes"), (dict(Hq=0), 1, "bad sizes"), (dict(Hk=1025), 1, "bad sizes"),
    (dict(D=63), 2, "unsupported"), (dict(D=1026), 2, "unsupported"), (dict(rd=66), 2, "unsupported"),
    (dict(ro=1, rd=2), 2, "unsupported"), (dict(rd=-2), 2, "unsupported"), (dict(ro=32), 2, "unsupported"),
    (dict(qn=65), 1, "norm widths"), (dict(kn=-1), 1, "norm widths"), (dict(eps=-1.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"), (dict(q=None), 1, "null"), (dict(pos=None), 1, "null"), (dict(inv=None), 1, "null"),
    (dict(Hk=1), 1, "null"), (dict(q=P + 1), 1, "aligned"), (dict(dtype=2, qo=U), 1, "aligned")])
def test_norm_rope_refusals(kw, code, words):
    refused(rope(**kw), code, words)


def write(**kw):
    a = dict(dtype=0, T=4, heads=2, k=P, kts=256, khs=128, kw=128, kp=P, kg=1.0, v=None, vts=0, vhs=0, vw=0, vp=None,
             vg=1.0, n_slots=8, sm=P, st=None)
    a.update(kw)
    return lsa._lib.lsa_write_q4(*a.values(), None)


@pytest.mark.parametrize("kw,code,words", [
    (dict(dtype=-1), 1, "dtype"), (dict(heads=0), 1, "bad sizes"), (dict(n_slots=0), 1, "bad sizes"), (dict(T=-1), 1, "bad sizes"),
    (dict(kw=120), 2, "width"), (dict(kw=4112), 2, "width"), (dict(k=None), 1, "null"), (dict(sm=None), 1, "null"),
    (dict(k=U), 1, "aligned"), (dict(khs=129), 1, "aligned"), (dict(kg=0.0), 1, "scale"), (dict(kg=float("inf")), 1, "scale"),
    (dict(kg=float("nan")), 1, "scale"), (dict(v=P), 1, "without a v_pool"), (dict(vp=P, vw=64), 1, "null"),
    (dict(vp=P, v=P, vw=8), 2, "width")])
def test_write_refusals(kw, code, words):
    refused(write(**kw), code, words)


def append(**kw):
    a = dict(dtype=0, heads=2, k=P, kw=128, kp=P, kg=1.0, v=None, vw=0, vp=None, vg=1.0, li=None, lip=None, dl=0,
             n_slots=8, table=P, stride=4, start=P, length=P, B=2, st=None)
    a.update(kw)
    return lsa._lib.lsa_append_token_q4(*a.values(), None)


@pytest.mark.parametrize("kw,code,words", [
    (dict(dtype=9), 1, "dtype"), (dict(B=0), 1, "bad sizes"), (dict(stride=0), 1, "bad sizes"), (dict(table=None), 1, "null"),
    (dict(kw=72), 2, "width"), (dict(li=P), 1, "together"), (dict(li=P, lip=P, dl=12), 1, "multiple of 8"),
    (dict(v=P), 1, "without a v_pool")])
def test_append_refusals(kw, code, words):
    refused(append(**kw), code, words)


def read(**kw):
    a = dict(pool=P, n_slots=8, heads=2, width=128, g=1.0, sm=P, T=4, dtype=0, out=P, st=None)
    a.update(kw)
    return lsa._lib.lsa_read_q4(*a.values(), None)


@pytest.mark.parametrize("kw,code,words", [
    (dict(dtype=5), 1, "dtype"), (dict(heads=0), 1, "bad sizes"), (dict(width=24), 2, "width"), (dict(out=None), 1, "null"),
    (dict(out=U), 1, "aligned"), (dict(g=-1.0), 1, "scale")])
def test_read_refusals(kw, code, words):
    refused(read(**kw), code, words)


def decode(**kw):
    a = dict(qd=0, q=P, kp=P, kg=1.0, vp=P, vg=1.0, n_slots=8, heads=2, table=P, stride=4, ti=P, tc=P, k=4, ws_=P, wl=P,
             mw=100, B=2, Hq=8, dqk=128, dv=128, scale=0.1, od=0, out=P, lse=None, st=None, ws=P, nws=1 << 40)
    a.update(kw)
    return lsa._lib.lsa_sparse_decode_q4(*a.values(), None)


@pytest.mark.parametrize("kw,code,words", [
    (dict(B=0), 1, "bad sizes"), (dict(B=70000), 1, "bad sizes"), (dict(k=-1), 1, "bad sizes"), (dict(mw=-1), 1, "bad sizes"),
    (dict(qd=2), 1, "bf16 or f16"), (dict(od=3), 1, "output dtype"), (dict(q=None), 1, "null"), (dict(ti=None), 1, "null"),
    (dict(Hq=7), 2, "unsupported"), (dict(dqk=96, dv=96), 2, "unsupported"), (dict(dqk=128, dv=64), 2, "unsupported"),
    (dict(vp=None), 2, "unsupported"), (dict(vp=None, dqk=576, dv=512), 2, "unsupported"),
    (dict(vp=None, dqk=576, dv=512, heads=1, Hq=129), 2, "unsupported"), (dict(dqk=576, dv=512, heads=1), 2, "unsupported"),
    (dict(out=U), 1, "aligned"), (dict(q=U), 1, "aligned"), (dict(scale=0.0), 1, "scales"),
    (dict(scale=float("nan")), 1, "scales"), (dict(vg=float("inf")), 1, "scales"), (dict(nws=64), 7, "workspace")])
def test_decode_refusals(kw, code, words):
    refused(decode(**kw), code, words)


def test_sizes_are_host_only():
    assert lsa.q4_chunk_bytes(576) == 20736 and lsa.q4_chunk_bytes(128) == 4608
    with pytest.raises(lsa.LSAError):
        lsa.q4_chunk_bytes(100)
    assert lsa.sparse_decode_q4_workspace_size(2, 8, 2, 96, 96, 0, 64) == 0
    one = lsa.sparse_decode_q4_workspace_size(1, 128, 1, 576, 512, 2048, 8000)
    assert one >= 128 * 514 * 4
    assert lsa.build_tables_workspace_size(0, 4, 8) == 0
    assert lsa.build_tables_workspace_size(4, 16, 1000) >= 32 * 4 + 6 * 4 + 64 * 4


def test_the_binding_refuses_cpu_tensors():
    import torch
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(lsa.LSAError, match="CUDA"):
        lsa.build_tables(t, t[:, 0], t[:, 0], 8, 4)
    with pytest.raises(lsa.LSAError, match="CUDA"):
        lsa.qk_norm_rope(torch.zeros(1, 1, 64), None, t[0, :1], torch.ones(32))
    with pytest.raises(lsa.LSAError, match="CUDA"):
        lsa.write_q4(torch.zeros(1, 1, 64), t, t)
    with pytest.raises(lsa.LSAError, match="CUDA"):
        lsa.sparse_decode_q4(torch.zeros(1, 1, 64), t, t, t, None, None, t, t, 1, 64, 1.0)


def test_what_must_not_overlap():
    refused(tables(nxt=P + 28), 1, "overlap")              # the table's last entry
    refused(tables(nxt=P - 28), 1, "overlap")
    refused(tables(B=65535, stride=40000, nxt=1 << 60, nws=1 << 40), 1, "2^31")
    refused(write(v=P, vts=256, vhs=128, vw=128, vp=P), 1, "the same")
    refused(append(v=P, vw=128, vp=P), 1, "the same")
