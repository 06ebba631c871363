"""The argument checks of the gated block, the adapters and the token log
probabilities under AddressSanitizer and UndefinedBehaviorSanitizer, on the
CPU: the build and the child process of tests/test_host_sanitizers.py, with the
C-ABI tests of these calls."""

from __future__ import annotations

import os

import pytest


def test_dense_abi_checks_clean_under_host_sanitizers(tmp_path, monkeypatch):
    base = pytest.importorskip("tests.test_host_sanitizers")
    if not os.path.exists(base.HIPCC) or base._asan_runtime() is None:
        pytest.skip("hipcc or the sanitizer runtime is not installed")
    run, ran = base.subprocess.run, []
    old = repr(os.path.join(base.ROOT, "tests", "test_abi.py"))
    new = repr(os.path.join(base.ROOT, "tests", "test_abi_dense.py"))

    def with_these_tests(cmd, **kw):
        if "-c" in cmd[1:2]:
            assert cmd[2].count(old) == 1
            cmd = [*cmd[:2], cmd[2].replace(old, new), *cmd[3:]]
            ran.append(cmd)
        return run(cmd, **kw)

    monkeypatch.setattr(base.subprocess, "run", with_these_tests)
    base.test_abi_checks_clean_under_host_sanitizers(tmp_path)
    assert len(ran) == 1
