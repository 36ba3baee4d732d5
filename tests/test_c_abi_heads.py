"""The rotary and output-layer entry points from C: tests/c_abi_heads_client.c is compiled with gcc as
C99 against include/tb.h alone and linked with libtb.so, as test_c_abi.py does for the others."""
import os
import subprocess

import pytest

import test_c_abi as base


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture
def client(built, tmp_path, monkeypatch):
    monkeypatch.setattr(base, "SRC", os.path.join(base.ROOT, "tests", "c_abi_heads_client.c"))
    return lambda with_cuda: base._compile(tmp_path, with_cuda)


def test_structs_and_argument_checks(client):
    p = subprocess.run([client(False)], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, p.stdout + p.stderr
    assert "argument checks through the C ABI: ok" in p.stdout


@pytest.mark.gpu
def test_kernels_against_closed_forms(client):
    p = subprocess.run([client(True), "gpu"], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout + p.stderr
    assert "rotation" in p.stdout and "output layer's loss" in p.stdout
