"""The two launches of an eviction, without a GPU: the rows move behind a selection that has been launched, never behind one
that was refused (the numbers of the rows would be whatever their buffer holds)."""
import ctypes
import os
import subprocess

import pytest

from quantized_decoder_decode_gb300 import build as fqbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    out = os.path.join(str(tmp_path_factory.mktemp("evict_host")), "evict_host.so")
    subprocess.check_call([fqbuild.NVCC, *fqbuild.ARCH, *fqbuild.FLAGS, "-shared", "-cudart", "shared", "-Xlinker", "-Bsymbolic",
                           os.path.join(fqbuild.CSRC, "evict.cu"), os.path.join(HERE, "evict_host.cpp"), "-o", out])
    return ctypes.CDLL(out)


def test_both_are_launched(host):
    assert host.evict_host_launches(-1) == 2


def test_nothing_moves_behind_a_refused_selection(host):
    assert host.evict_host_launches(0) == 1


def test_a_refused_move(host):
    assert host.evict_host_launches(1) == 2
