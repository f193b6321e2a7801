"""How attention's work is cut (csrc/kv_split.h), built for the host and checked against unbounded integers up to the
largest arguments that a call may have."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
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
    lib.rows_grid.argtypes = [ctypes.c_int, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, i64 * 3]
    lib.attend_fits.argtypes = [i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, i64]
    return lib


def rows_grid(split, rows, new, group, heads):
    out = (ctypes.c_int64 * 3)()
    split.rows_grid(rows, sum(new), len(new), max(new), group, heads, out)
    return bool(out[0]), out[1], out[2]


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


def test_a_long_prompt_beside_many_single_tokens_fits_a_launch(split):
    # 1024 row blocks for each of 1024 sequences and 8 heads would be 2^23 workgroups of 512 threads, one more than a
    # launch may have; 33791 tokens of 64 heads fill about 1056 blocks of 256 rows per head
    new = [32768] + [1] * 1023
    listed, groups, width = rows_grid(split, 256, new, 8, 8)
    assert listed and groups == 8 and 1056 <= width <= 1056 + 1024
    assert split.attend_fits(sum(new), len(new), max(new), 8, 8, 1 << 17)
    assert split.attend_fits(32768, 1, 32768, 8, 8, 1 << 20)         # that prompt alone over a million positions
    assert not split.attend_fits(1 << 22, 1 << 22, 1, 512, 2, 4096)  # 2^23 blocks: refused, not launched


@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 40, 256])
def test_listed_blocks_have_slots_of_their_own(split, rows, group):
    rng = np.random.default_rng(rows + group)
    for new in ([1], [0, 0, 5], [600] + [1] * 70, list(rng.integers(0, 90, 200)), [0] * 65 + [900] + [33] * 64):
        new = [int(n) for n in new]
        starts = np.concatenate([[0], np.cumsum(new)])
        slots = [split.row_slot(int(s), b, group, rows) for b, s in enumerate(starts)]
        assert slots[0] == 0
        for b, n in enumerate(new):
            assert slots[b + 1] > slots[b] and slots[b + 1] - slots[b] >= -(-n * group // rows)
        listed, groups, width = rows_grid(split, rows, new, group, 3)
        blocks = -(-max(new) * group // rows)
        assert (groups, width) == ((3, slots[-1]) if listed else (3 * len(new), blocks))
        assert groups * width <= 3 * 2 * slots[-1]  # never more than twice the blocks that can exist
    assert split.row_slot(1 << 24, 1 << 24, 64, 128) == (1 << 23) + (1 << 24)


def test_even_batches_keep_a_group_for_each_sequence_and_head(split):
    assert rows_grid(split, 256, [2048, 2048], 4, 8) == (False, 16, 32)
    assert rows_grid(split, 128, [20], 4, 1) == (False, 1, 1)


def test_windows_that_no_context_reaches_are_none(split):
    for window in (0, 1, 900, (1 << 30) - 1):
        assert split.kept_window(window) == window
    for window in (1 << 30, (1 << 31) - 1):
        assert split.kept_window(window) == 0
    # what kernels form from a window that is kept: position, new tokens and window at their largest
    assert -(1 << 31) < -(1 << 24) - ((1 << 30) - 1) and (1 << 30) - 1 + (1 << 30) < 1 << 31


def test_short_sequences_of_mixed_batches_are_counted_whatever_the_starts_say(split):
    # two blocks of 16 rows for every sequence, also where the batch has fewer tokens than that
    cost, limit, seen = split.unit_cost(), 1 << 31, set()
    for seqs in (2, 8, 1 << 10, 1 << 17, 1 << 20, 1 << 23):
        for group in (1, 4, 16):
            for kv in (64, 4096, 10240, 1 << 20):
                for heads in (1, 8, 12):
                    fits = bool(split.attend_fits(33 + seqs, seqs, 33, group, heads, kv))
                    assert not fits or 2 * seqs * heads * (-(-kv // 64) + cost) + 512 < limit
                    seen.add(fits)
    assert seen == {True, False}
