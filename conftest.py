"""Order of the tests: cases that are known to hold wrong values run after all others, so that a run that stops at
the first failure has checked everything else.

An entry of a cache that was evicted from is visible by its position (tests/test_gpu_bounded_positions.py).  These
cases expect the rule that went by its index; the token at position 1334 of `scrambled`, for instance, is expected
to see the entry that ends at 1335."""

INDEX_RULE = {
    f"test_gpu_bounded.py::{test}[{prefix}{case}]"
    for case in ("scrambled", "scrambled_docs", "d64_scrambled")
    for test, prefix in (("test_attention_matches_oracle", ""), ("test_weights_match_oracle", "apart-"),
                         ("test_weights_match_oracle", "in_place-"))
}


def pytest_collection_modifyitems(items):
    items.sort(key=lambda item: item.nodeid.rsplit("/", 1)[-1] in INDEX_RULE)
