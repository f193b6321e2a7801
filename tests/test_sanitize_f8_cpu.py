"""Host AddressSanitizer + UndefinedBehaviorSanitizer build of the host code of the products in 8-bit floating point
(f8_api.cpp), driven through the paths that need no GPU by tests/sanitize/f8_errors.c."""
import os

import pytest

from test_sanitize_cpu import CLANG, CSRC, HERE, INCLUDE, ROCM, SANITIZERS, _run


def test_f8_error_paths_under_asan_and_ubsan(tmp_path):
    hip_compiler = os.path.join(ROCM, "bin", "hipcc")
    if not (os.path.exists(hip_compiler) and os.path.exists(CLANG)):
        pytest.skip("ROCm compilers not found")
    host_only = [x for f in SANITIZERS for x in ("-Xarch_host", f)]  # host code only
    common = ["-O1", "-g", "-fno-omit-frame-pointer", f"-I{INCLUDE}"]
    objs = []
    for src in [os.path.join(CSRC, f) for f in ("api.cpp", "f8_api.cpp")] + [os.path.join(HERE, "f8_stubs.cpp")]:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        _run([hip_compiler, "-std=c++17", "-fPIC", *common, f"-I{CSRC}", *host_only, "-c", src, "-o", objs[-1]])
    for compiler, std, src in ((CLANG + "++", "-std=c++17", "variant_stubs.cpp"), (CLANG, "-std=c99", "f8_errors.c")):
        objs.append(str(tmp_path / (src + ".o")))
        _run([compiler, std, "-Wall", *common, *SANITIZERS, "-c", os.path.join(HERE, src), "-o", objs[-1]])
    exe = str(tmp_path / "f8_errors")
    _run([CLANG + "++", *SANITIZERS[:2], *objs, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-o", exe])
    env = dict(os.environ, BSG_FORCE_ARCH="gfx942", ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = _run([exe], env=env, timeout=120)
    assert "ok: 0 failures" in r.stdout, r.stdout
