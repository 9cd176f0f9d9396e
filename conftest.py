"""Order of the tests.

tests/test_gpu_serving.py::test_prefill_reports_bad_starts_and_gates expects a
gate of zero to be refused and to keep the state; by the layer's rule it
forgets the state (tests/test_gpu_zero_gates.py).  It runs after all others, so
that a run that stops at the first failure has been through them.
"""


def pytest_collection_modifyitems(items):
    items.sort(key=lambda item: "test_prefill_reports_bad_starts_and_gates" in item.nodeid)
