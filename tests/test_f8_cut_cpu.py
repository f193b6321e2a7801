"""Which kernel takes an E4M3 product and in how many parts (csrc/f8_cut.h), built for the host."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

import f8_cases

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "block_scaled_precision_gemm_amd", "csrc")
PER_CU = {"T64x32": 3, "T64x64": 3, "T128x64": 2, "T64x32Wide": 3, "T64x64Wide": 3}  # workgroups that run on one CU; others: 1
SHAPE = {w: tuple(int(n) for n in w[1:].removesuffix("Wide").split("x")) for w in f8_cases.WAYS}


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    lib, i64 = str(tmp_path_factory.mktemp("cut") / "cut.so"), ctypes.c_int64
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", f"-I{CSRC}", os.path.join(HERE, "f8_cut_c.cpp"), "-o", lib],
                   check=True, timeout=120)
    lib = ctypes.CDLL(lib)
    lib.cut.argtypes = [ctypes.c_int, i64, i64, i64, ctypes.c_int, i64 * 3, ctypes.POINTER(ctypes.c_double)]

    def choose(gated, tokens, n, k, cus=f8_cases.CUS):
        out, cost = (i64 * 3)(), ctypes.c_double()
        lib.cut(gated, tokens, n, k, cus, out, ctypes.byref(cost))
        return f8_cases.WAYS[out[0]], out[1], out[2], cost.value

    def parts(gated, max_tokens, n, k, cus=f8_cases.CUS):
        out = (i64 * 2)()
        lib.parts(gated, max_tokens, n, k, cus, out)
        return tuple(out)
    lib.parts.argtypes = [ctypes.c_int, i64, i64, i64, ctypes.c_int, i64 * 2]
    lib.tokens_at_once.argtypes, lib.tokens_at_once.restype = [ctypes.c_int, i64, ctypes.c_int], i64
    choose.parts, choose.tokens_at_once = parts, lib.tokens_at_once
    return choose


def test_the_cases_reach_what_they_are_for(cut):
    for gated, cases in ((0, f8_cases.PRODUCTS), (1, f8_cases.GATED), (2, f8_cases.EXACT_PRODUCTS), (3, f8_cases.EXACT_GATED)):
        for t, n, k, way, parts in cases:
            assert cut(gated, t, n, k)[::2] == (way, parts), (t, n, k)
    everything = f8_cases.PRODUCTS + f8_cases.GATED + f8_cases.EXACT_PRODUCTS + f8_cases.EXACT_GATED
    assert {c[3] for c in everything} == set(f8_cases.WAYS)
    for way in f8_cases.WAYS:  # each with parts, where it has them, and with weights' scales that are loaded again
        mine = [c for c in everything if c[3] == way]
        assert any(-(-c[2] // 128) > 64 * c[4] for c in mine), way
        assert way.endswith("256x256") or any(c[4] > 1 for c in mine), way
    for way in ("T256x256", "G256x256"):
        mine = [c for c in f8_cases.PRODUCTS + f8_cases.GATED if c[3] == way]
        assert any(-(-c[0] // 256) * -(-c[1] // (256 if way[0] == "T" else 128)) > f8_cases.CUS for c in mine)
        assert {-(-c[2] // 128) % 2 for c in mine} == {0, 1}
    for t, inter, hidden in f8_cases.FEW_GATED:
        assert t <= 16 and t * -(-max(inter, hidden) // 128) > 512


def test_a_cut_fits_the_device_and_the_call(cut):
    rng = random.Random(0)
    for _ in range(5000):
        gated, exact, t = rng.randint(0, 1), rng.randint(0, 1), rng.choice([17, 32, 33, 64, 65, rng.randint(17, 300), rng.randint(17, 20000)])
        n, k, cus = 16 * rng.randint(1, 1000), 16 * rng.choice([1, rng.randint(1, 100), rng.randint(1, 16384)]), rng.choice([256, 64, 304])
        way, tiles, parts, cost = cut(gated + 2 * exact, t, n, k, cus)
        rows, cols = SHAPE[way]
        assert way[0] == "TG"[gated] and cost > 0
        assert tiles == -(-t // cols) * -(-n // (rows // 2 if gated else rows))
        # the workspace holds the parts of as many workgroups as run at once, and a part is worth a workgroup's start
        assert parts == 1 or (not way.endswith("256x256") and tiles * parts <= cus * PER_CU.get(way, 1) and parts * 4 <= -(-k // 128))
        # exact products are of widened codes, others in gate and up of up to 64 tokens
        assert way.endswith("Wide") == bool(exact or (gated and t <= 64))
        assert cols >= min(t, 32)


def test_equal_costs_and_the_smallest_calls(cut):
    assert cut(0, 17, 16, 16)[0] == "T64x32" and cut(0, 33, 16, 16)[0] == "T64x64"
    assert cut(0, 1 << 24, 1 << 18, 1 << 18)[0] == "T256x256" and cut(1, 1 << 24, 1 << 18, 1 << 18)[0] == "G256x256"
    assert cut(1, 17, 16, 16)[:3] == ("G256x32Wide", 1, 1)


def test_a_workspace_holds_the_parts_of_every_call_and_little_more(cut):
    rng = random.Random(1)
    for _ in range(300):
        gated, cus, most = rng.randint(0, 3), rng.choice([256, 64]), rng.choice([17, 33, 64, 65, 200, 5000])
        n, k = 16 * rng.choice([rng.randint(1, 40), rng.randint(1, 1000)]), 16 * rng.choice([rng.randint(1, 63), rng.randint(64, 16384)])
        floats, counters = cut.parts(gated, most, n, k, cus)
        # never more than the workgroups that run at once have, and nothing where K cannot be split
        assert floats <= cus * 256 * 128 and counters <= cus * 3 // 2
        assert k > 7 * 128 or floats == counters == 0
        for t in {17, most, *(rng.randint(17, most) for _ in range(40))}:
            way, tiles, parts, _ = cut(gated, t, n, k, cus)
            rows, cols = SHAPE[way]
            # (gated: 1, and 2 for exact products)
            assert parts == 1 or (tiles * parts * rows * cols <= floats and tiles <= counters), (gated, t, n, k, cus)


def test_workspaces_of_some_plans(cut):
    assert cut.parts(0, 16, 8192, 8192) == cut.parts(1, 16, 8192, 8192) == (0, 0)
    assert cut.parts(0, 8192, 4096, 896) == (0, 0)                # seven blocks
    assert cut.parts(0, 8192, 1 << 18, 8192) == (0, 0)            # more tiles than run at once
    assert cut.parts(0, 64, 16, 1024) == (2 * 128 * 128, 1)       # one tile of 128 x 128 in two parts


def test_grids_of_many_tiles_stay_below_32_bits_of_threads(cut):
    for way in f8_cases.WAYS[:-2]:
        rows, cols = SHAPE[way]
        for n in (16, 8192, 1 << 18):
            tiles_n = -(-n // (rows // 2 if way[0] == "G" else rows))
            most = cut.tokens_at_once(f8_cases.WAYS.index(way), n, 512)
            assert most > 0 and most % cols == 0 and most // cols * tiles_n * 512 <= 1 << 31 < (most // cols + 1) * tiles_n * 512
    # calls that a device of 288 GB can hold and a grid cannot: inner codes of 69 GB, outputs of 137 GB
    for gated, t, n, k in ((3, 1 << 20, 65536, 16), (2, (1 << 19) + 128, 1 << 17, 16)):
        way, tiles, parts, _ = cut(gated, t, n, k)
        assert parts == 1 and tiles * 512 > 1 << 31 and cut.tokens_at_once(f8_cases.WAYS.index(way), n, 512) < t
