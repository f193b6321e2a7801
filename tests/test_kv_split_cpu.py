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
    lib, i64 = ctypes.CDLL(lib), ctypes.c_int64
    lib.context_positions.restype = i64
    lib.line_fits.argtypes = [i64, ctypes.c_int, i64, ctypes.c_int, i64]
    return lib


@pytest.mark.parametrize("tiles", [1, 2, 9, 512, 4_202_521, 1 << 23, (1 << 24) - 1, 1 << 24])
@pytest.mark.parametrize("pieces", [1, 2, 3, 255, 511, 512])
def test_pieces_cover_the_tiles_once(split, pieces, tiles):
    begins = [split.piece_begin(i, pieces, tiles) for i in range(pieces + 1)]
    assert begins == [i * tiles // pieces for i in range(pieces + 1)]


def test_the_line_of_all_units_stays_below_32_bits(split):
    # (new tokens and context of a sequence), sequences, query heads per key/value head, key/value heads
    cost, limit = split.unit_cost(), 1 << 31
    seen = set()
    for q, kv in ((1, 1), (1, 64), (3, 4096), (8, 1 << 17), (1, 1 << 30)):
        for seqs in (1, 7, 1 << 10, 1 << 20, 1 << 24):
            for group in (1, 5, 32):
                for heads in (1, 16, 1024):
                    rows = 16 if q * group <= 16 else 32
                    items = -(-q * group // rows) * seqs * heads * (-(-kv // 64) + cost)
                    fits = bool(split.line_fits(q * seqs, group, seqs, heads, kv))
                    assert not fits or items + 512 < limit
                    seen.add(fits)
    assert seen == {True, False}
    assert not split.line_fits(1 << 24, 1, 1 << 24, 16, 1)      # 2^28 units of one tile: the fixed cost alone is too much
    assert split.line_fits(4096, 8, 4096, 8, 1 << 17)            # what programs ask for: 4096 sequences of 131072 positions


@pytest.mark.parametrize("window", [0, 1, 1000, 1 << 30])
def test_positions_that_are_seen(split, window):
    for max_q in (1, 40, 1 << 24):
        for max_kv in (1, 900, 1 << 30):
            want = min(max_kv, window + max_q + 16) if window else max_kv
            assert split.context_positions(window, max_q, max_kv) == want
