"""Argument checks of the step plan and of scored attention against a pool
description made on the host: refused before the GPU is touched (no GPU)."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_host_refusals(tmp_path):
    from paged_kv_cache_68_gb300 import pagedkv
    pagedkv.load()
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe, lib = str(tmp_path / "host_refusals"), os.path.dirname(pagedkv.library_path())
    r = subprocess.run([nvcc, "-std=c++20", "-O1", "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(ROOT, "paged_kv_cache_68_gb300", "csrc"),
                        os.path.join(HERE, "host_refusals.cu"), "-o", exe, "-L", lib, "-lpagedkv",
                        "-Xlinker", f"-rpath={lib}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.split() == ["ok"], r.stdout + r.stderr
