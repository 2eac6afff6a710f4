"""soma_ops_check without a GPU: the library's host side against fakes of the CUDA runtime and of the kernels.  It waits for
the device before it reads how often a kernel's bounded wait ran out, reports every new one once, and loses none."""
import ctypes
import os
import shutil
import subprocess

import pytest

from tensor_grad_clip_gb300 import _abi, build

HERE = os.path.dirname(os.path.abspath(__file__))

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture()
def fake(tmp_path):
    lib = tmp_path / "fake.so"  # one per test: the library remembers what it has reported
    cuda = os.path.join(os.path.dirname(os.path.dirname(shutil.which(build.nvcc()) or build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-Wall", "-I", build.INCLUDE, "-I", build.CSRC, "-I", cuda,
                    os.path.join(HERE, "c_abi", "fake_ops.cpp"), os.path.join(build.CSRC, "ops.cpp"), "-o", str(lib)],
                   check=True)
    dll = ctypes.CDLL(str(lib))
    dll.soma_ops_last_error.restype = ctypes.c_char_p
    return dll


def calls(fake):
    seen = (ctypes.c_char * 256).in_dll(fake, "fake_calls")
    text = seen.value.decode().split()
    seen.value = b""
    return text


def test_the_device_is_waited_for_first(fake):
    assert fake.soma_ops_check(0) == 0
    assert calls(fake) == ["sync", "read", "read", "read"]


def test_every_expired_wait_is_reported_once(fake):
    counts = (ctypes.c_uint * 3).in_dll(fake, "fake_counts")
    assert fake.soma_ops_check(0) == 0
    for which, name in enumerate(("layer norm", "linear", "distillation")):
        counts[which] += 5
        assert fake.soma_ops_check(0) == _abi.SOMA_ERR_STATE
        assert name in fake.soma_ops_last_error().decode()
        assert fake.soma_ops_check(0) == 0
    counts[1] = 2 ** 32 - 1
    assert fake.soma_ops_check(0) == _abi.SOMA_ERR_STATE
    counts[1] = 0  # the count wrapped
    assert fake.soma_ops_check(0) == _abi.SOMA_ERR_STATE
    assert fake.soma_ops_check(0) == 0


def test_devices_are_told_apart(fake):
    counts = (ctypes.c_uint * 3).in_dll(fake, "fake_counts")
    counts[0] = 1
    assert fake.soma_ops_check(0) == _abi.SOMA_ERR_STATE
    assert fake.soma_ops_check(1) == _abi.SOMA_ERR_STATE
    assert fake.soma_ops_check(0) == 0 and fake.soma_ops_check(1) == 0


def test_errors_of_the_runtime_are_reported_and_lose_nothing(fake):
    counts = (ctypes.c_uint * 3).in_dll(fake, "fake_counts")
    counts[2] = 1
    for name in ("fake_sync_error", "fake_read_error"):
        ctypes.c_int.in_dll(fake, name).value = 700
        assert fake.soma_ops_check(0) == _abi.SOMA_ERR_CUDA
        ctypes.c_int.in_dll(fake, name).value = 0
    assert fake.soma_ops_check(0) == _abi.SOMA_ERR_STATE
