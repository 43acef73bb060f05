"""Host-side refusals of the page planner, the 8-bit attention and the logits
adjustment at the ends of their arguments' ranges, without a GPU (the pointers
are never dereferenced, and every call below is refused)."""

import ctypes

import pytest

from self_speculative_verification_gb300 import binding as bn

OK, INVALID, UNSUPPORTED, CAPACITY, CUDA = 0, 1, 2, 4, 5
REF = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    return bn.load_library()


# arrays of a plan of 100 requests and 10000 slots, 1 MB apart
B, SLOTS = 100, 10000
ARRAYS = {n: 0x100000 * (i + 1) for i, n in enumerate(("seq_len", "n_new", "table", "free_pages", "free_head",
                                                       "cu", "slots", "new_len"))}
BYTES = dict(seq_len=4 * B, n_new=4 * B, table=4 * B * 8, free_pages=4 * 50, free_head=4, cu=4 * (B + 1),
             slots=8 * SLOTS, new_len=4 * B)


def plan(lib, **ptrs):
    p = dict(ARRAYS, **ptrs)
    return lib.spec_page_plan(B, 16, 64, 8, p["seq_len"], p["n_new"], p["table"], p["free_pages"], 50,
                              p["free_head"], p["cu"], SLOTS, p["slots"], p["new_len"], None)


@pytest.mark.parametrize("out,other", [(o, x) for o in ("cu", "slots", "new_len") for x in ARRAYS if x != o])
def test_a_plan_whose_outputs_overlap_another_array(lib, out, other):
    """Other threads still read the inputs when outputs are written."""
    at = ARRAYS[other]
    assert plan(lib, **{out: at}) == INVALID
    assert plan(lib, **{out: at + BYTES[other] - 4}) == INVALID          # its last element
    assert plan(lib, **{out: at - BYTES[out] + 4}) == INVALID            # its first one


@pytest.mark.parametrize("V", [65535 * 4096 + 1, (1 << 31) - 2048, (1 << 31) - 1])
@pytest.mark.parametrize("Rj,batch", [(1, 1), (1, 4000), (1 << 30, 1)])
def test_vocabularies_past_the_grid(lib, V, Rj, batch):
    d = bn.logits_desc(batch, Rj, V, bn.SPEC_BF16)
    assert lib.spec_logits_adjust(REF(d), 0x1000, 0x1000, *[None] * 14) == UNSUPPORTED


@pytest.mark.parametrize("split", [1 << 30, (1 << 31) - 64])
@pytest.mark.parametrize("pages", [4, 1 << 22])
def test_splits_longer_than_the_cache(lib, split, pages):
    """A split that holds every prefix is one split, whatever its length."""
    c = bn.Kv8Desc(2, 128, 0x1000, 0x1000, 2, 1 << 23, 256, pages, 0x1000)

    def size(tokens):
        a = bn.attn_desc(2, 4, 4, 2, 128, bn.SPEC_F32, 0, split_tokens=tokens)
        n = ctypes.c_size_t(0)
        return lib.spec_verify_attn_kv8_workspace_size(REF(a), REF(c), REF(n)), n.value

    assert size(split) == size(pages * 256)
    assert size(split)[0] == OK and size(split)[1] > 0
