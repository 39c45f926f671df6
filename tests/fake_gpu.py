"""The library's host code on stand-in GPUs: its objects linked with
fake_cudart.cpp instead of the CUDA runtime."""

from __future__ import annotations

import glob
import os
import shutil
import subprocess

import pytest

from flow_matching_action_dm0_b200 import _lib as L
from flow_matching_action_dm0_b200 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def link(folder) -> str:
    """Path of the library on stand-in GPUs, linked into folder."""
    objects = sorted(glob.glob(os.path.join(B.BUILD, "*.o")))
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    if not shutil.which("g++") or not os.path.isdir(include) or len(objects) != len(B.sources()):
        pytest.skip("the library's objects, CUDA's headers and g++ are needed")
    out = os.path.join(str(folder), "librtv_host.so")
    # (the library's own functions before any of the same name elsewhere in the process)
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-std=c++17", "-Wl,-Bsymbolic", "-I" + include, "-o", out,
                    os.path.join(HERE, "fake_cudart.cpp"), *objects], check=True)
    return out


@pytest.fixture(scope="session")
def host_library_path(tmp_path_factory):
    return link(tmp_path_factory.mktemp("host"))


@pytest.fixture
def gpus(host_library_path, monkeypatch):
    """The package calls the library on two stand-in GPUs; returns it (fake_* are the stand-in's)."""
    monkeypatch.setattr(L, "_lib", None)
    lib = L.load_library(host_library_path)
    lib.fake_gpus(2)
    lib.cudaSetDevice(0)
    return lib
