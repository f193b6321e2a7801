"""How attention's work is cut (csrc/kv_split.h), built for the host and checked against unbounded integers up to the
largest arguments that a call may have."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "block_scaled_precision_gemm_amd", "csrc")


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    lib = str(tmp_path_factory.mktemp("split") / "split.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fwrapv", "-shared", "-fPIC", f"-I{CSRC}",
                    os.path.join(HERE, "kv_split_c.cpp"), "-o", lib], check=True, timeout=120)
    return ctypes.CDLL(lib)


@pytest.mark.parametrize("tiles", [1, 2, 9, 512, 4_202_521, 1 << 23, (1 << 24) - 1, 1 << 24])
@pytest.mark.parametrize("pieces", [1, 2, 3, 255, 511, 512])
def test_pieces_cover_the_tiles_once(split, pieces, tiles):
    begins = [split.piece_begin(i, pieces, tiles) for i in range(pieces + 1)]
    assert begins == [i * tiles // pieces for i in range(pieces + 1)]
