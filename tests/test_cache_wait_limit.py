"""The limit of the kernels' waits: host logic alone, no call is made."""

from exact_top_selection_gb300 import cache as binding


def test_limits_and_refusals():
    lib = binding._lib()
    try:
        for polls in (0, 1, 1 << 20, -1):
            assert lib.exact_topk_set_wait_limit(polls) == 0
        for polls in ((1 << 20) + 1, 1 << 40):
            assert lib.exact_topk_set_wait_limit(polls) == -2
    finally:
        assert lib.exact_topk_set_wait_limit(-1) == 0
