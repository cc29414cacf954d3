"""The host code of routing, the weighted sum of routes and the products with
packed 4-bit weights under AddressSanitizer and UndefinedBehaviorSanitizer:
their host-only tests run against an instrumented build in a child process.
Nothing launches a kernel."""
import subprocess
import sys

from tests.test_host_sanitizers import ROOT, sanitized  # noqa: F401


def test_route_validation_under_sanitizers(sanitized):  # noqa: F811
    _, env = sanitized
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "not gpu", "-p", "no:cacheprovider",
                          "tests/test_route_abi.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    text = res.stdout[-3000:] + res.stderr[-3000:]
    assert res.returncode == 0, text
    assert "ERROR: AddressSanitizer" not in res.stderr and "runtime error:" not in res.stderr, text
    assert " passed" in res.stdout, text
