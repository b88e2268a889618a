"""Argument checks of the training operators and the build, without a device (CPU)."""
import time
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from masked_grouped_query_b200 import _lib, build
from tests.test_training_boundary import A, _rot


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_rotary_ignores_the_pointers_of_no_heads(lib):
    # Whatever they are: misaligned, or over another tensor.
    for bad in (A[1] + 8, A[0] + 4, 3):
        assert _rot(lib, {1: bad, 3: bad}, hkv=0, length=0) == 0
        assert _rot(lib, {0: bad, 2: bad}, hq=0, length=0) == 0
    assert _rot(lib, {0: A[0] + 8}, hkv=0) == -2
    assert _rot(lib, {3: A[3] + 8}, hq=0) == -2
    if not torch.cuda.is_available():  # past the checks, to the device's
        assert _rot(lib, {1: A[1] + 8, 3: A[0]}, hkv=0) == -7
        assert _rot(lib, {0: A[0] + 8, 2: A[1]}, hq=0) == -7


def test_windows_past_32_bits_stay_windows():
    from masked_grouped_query_b200.attention import _args
    assert [_args(w, None, False)[1] for w in (None, 0, -1, 5, 2 ** 31, 2 ** 32, 2 ** 32 + 7, -2 ** 32 + 5)] \
        == [0, 0, -1, 5, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, -2 ** 31]


def _fake_nvcc(tmp_path, monkeypatch, script):
    """build.build() compiling into tmp_path with a shell script in place of nvcc."""
    fake = tmp_path / "nvcc"
    fake.write_text("#!/bin/sh\n" + script)
    fake.chmod(0o755)
    monkeypatch.setattr(build, "nvcc", lambda: str(fake))
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "LIBRARY", str(tmp_path / "lib.so"))


# Writes a line into the file named after -o.
_WRITE = 'while [ "$1" != -o ]; do shift; done; echo made > "$2"\n'


@pytest.mark.parametrize("unit", build.UNITS)
def test_a_failed_compile_shows_the_compilers_message(tmp_path, monkeypatch, unit):
    _fake_nvcc(tmp_path, monkeypatch,
               f'case "$*" in *{unit}.cu*) echo "error: no such thing in {unit}"; exit 2;; esac\n'
               "sleep 0.3\n" + _WRITE)
    with pytest.raises(RuntimeError, match=f"no such thing in {unit}"):
        build.build(force=True)
    assert [p.name for p in tmp_path.iterdir()] == ["nvcc"]  # no objects left behind


def test_two_builds_at_once_each_publish_a_whole_library(tmp_path, monkeypatch):
    _fake_nvcc(tmp_path, monkeypatch, 'while [ "$1" != -o ]; do shift; done\n'
               'echo first > "$2"; sleep 0.4; echo last >> "$2"\n')
    with ThreadPoolExecutor(2) as pool:
        first = pool.submit(build.build, force=True)
        time.sleep(0.2)
        second = pool.submit(build.build, force=True)
        assert first.result() == second.result() == build.LIBRARY
    assert (tmp_path / "lib.so").read_text() == "first\nlast\n"
    assert sorted(p.name for p in tmp_path.iterdir()) == ["lib.so", "nvcc"]
