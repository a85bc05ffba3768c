"""kv_compact writes the new lengths while other warps read its inputs, so an
array of new lengths that overlaps one of them is refused, without a GPU."""
import pytest

from fp8_paged_kv_append_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    from fp8_paged_kv_append_gb300 import k16v8
    return k16v8.load_library()


# addresses that are never followed: 3 sequences of up to 8 nodes and 8 pages
BATCH, NODES, PAGES = 3, 8, 8
INPUTS = dict(table=0x10000, lens=0x20000, indptr=0x30000, path=0x40000, path_len=0x50000)
WORDS = dict(table=BATCH * PAGES, lens=BATCH, indptr=BATCH + 1, path=BATCH * NODES, path_len=BATCH)


@pytest.mark.parametrize("name", sorted(INPUTS))
def test_overlap_is_refused(lib, name):
    at, words = INPUTS[name], WORDS[name]
    for new in (at, at + 4, at + 4 * (words - 1), at - 4 * (BATCH - 1)):
        assert lib.k16v8_kv_compact(0x60000, 0x70000, 1, INPUTS["table"], PAGES, INPUTS["lens"],
                                    INPUTS["indptr"], INPUTS["path"], NODES, INPUTS["path_len"],
                                    BATCH, 2, 128, 8, new, None, None) == 1
