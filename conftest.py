"""Order of the tests.  A test that contradicts include/fa.h fails; it runs last,
so that a run that stops at its first failure has seen all the others."""

# Demands that, of a sequence with more new rows than max_seqlen_q, the rows that
# are computed see the keys of the rows after them: j <= i + seq_lens[b] - max_seqlen_q
# where the row's own key, and its last one, is i + seq_lens[b] - n.
CONTRADICTING = ("test_rows_beyond_the_bound_are_cut",)


def pytest_collection_modifyitems(items):
    items.sort(key=lambda item: getattr(item, "originalname", None) in CONTRADICTING)
