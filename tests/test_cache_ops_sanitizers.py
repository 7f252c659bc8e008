"""The host-side checks of the calls around the cache under AddressSanitizer and
UndefinedBehaviorSanitizer, as tests/test_sanitizers.py runs the others."""
from tests.test_sanitizers import _run_under_sanitizers


def test_refusals_under_asan_and_ubsan():
    assert " passed" in _run_under_sanitizers("test_cache_ops_refusals.py")
