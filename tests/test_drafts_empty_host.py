"""Calls of drafted tokens without a new token in any sequence, without a
GPU: the checks fire, and what has nothing to do returns, before any CUDA call."""
from test_drafts_host import FAKE, INVALID, _pages, lib  # noqa: F401


def test_tree_attn_of_no_new_tokens(lib):  # noqa: F811
    """Tokens that no sequence may hold are refused: their outputs would be
    returned unwritten with nothing flagged."""
    def run(T, max_new, kernel=None):
        args = (_pages(), FAKE, 256, T, 4, FAKE, 2, max_new, FAKE, 4, FAKE, None, 0.125, FAKE, None, FAKE, 1 << 30, None)
        return lib.nt_paged_tree_attn(*args) if kernel is None else lib.nt_selftest_paged_tree_attn(kernel, 0, *args)
    for kernel in (None, 0, 1, 2, 3):
        assert run(6, 0, kernel) == INVALID and run(0, 0, kernel) == 0


def test_tree_of_no_tokens(lib):  # noqa: F811
    """A step without new tokens has a max_new of 0."""
    def run(T, max_new, parents=FAKE, bits=FAKE):
        return lib.nt_draft_tree(parents, FAKE, 2, T, max_new, FAKE, bits, FAKE, None)
    assert run(0, 0) == 0 and run(0, 0, None, None) == 0 and run(0, 5) == 0
    assert run(1, 0) == INVALID and run(0, -1) == INVALID
