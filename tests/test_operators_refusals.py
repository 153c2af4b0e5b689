"""More refusals of the serving operators, before anything is launched (no GPU needed)."""
import pytest

from learned_sparse_kv_b200 import build as lbuild
from learned_sparse_kv_b200 import lsa
from tests.test_operators_host import P, decode, refused, rope, tables


@pytest.fixture(scope="module", autouse=True)
def built():
    lbuild.build()


@pytest.mark.parametrize("kw", [
    dict(qots=0), dict(qots=63), dict(qots=-32), dict(Hq=2, qots=128, qohs=0), dict(Hq=2, qots=128, qohs=62),
    dict(k=P, ko=P, Hk=1, kots=0), dict(k=P, ko=P, Hk=3, kots=192, kohs=32)])
def test_norm_rope_refuses_output_rows_that_overlap(kw):
    """Strides of an expanded output: several rows written to one place."""
    refused(rope(**kw), 1, "overlap")


def test_norm_rope_strides_of_single_rows_do_not_matter():
    refused(rope(T=1, qots=0, qohs=0, eps=-1.0), 1, "eps")
    assert rope(T=0, qots=0) == 0


def test_tables_take_every_slot_count():
    """The bitmap's size at the largest pool, where 32-bit arithmetic would wrap."""
    for n in (2 ** 31 - 32, 2 ** 31 - 31, 2 ** 31 - 1):
        need = lsa.build_tables_workspace_size(4, 16, n)
        assert 2 ** 28 <= need + 4 and need < 2 ** 28 + 4096, (n, need)


def test_workspaces_at_any_other_address_are_refused():
    """Partials and maps are read and written as vectors: a slice of a larger buffer may begin anywhere."""
    for off in (1, 4, 8):
        refused(decode(ws=P + off), 7, "aligned")
        refused(tables(ws=P + off), 7, "aligned")
