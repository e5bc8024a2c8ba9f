"""The host code of the linear layer, the gated block and gradient clipping built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer: validation, workspace sizes and offsets, the choice of kernel, tiles and splits, driven through
random calls with exact, short and absent workspaces.  The kernel launchers are stand-ins (tests/sanitizer/linear_stub.cpp)
that check every byte range a kernel would touch; no GPU is used.  The same build says which kernels a call launches."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

from sharded_gemm_amd import _abi

from linear_kernel_cases import CASES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sharded_gemm_amd", "csrc")
SAN = os.path.join(ROOT, "tests", "sanitizer")
ROCM = "/opt/rocm"
FLAGS = ["-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
         "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include"]
SOURCES = [os.path.join(CSRC, f) for f in ("plan.cpp", "checker.cpp", "api.cpp", "timing.cpp", "linear_api.cpp",
                                           "linear_launch.cpp")] + \
          [os.path.join(SAN, f) for f in ("stub_kernels.cpp", "linear_stub.cpp", "linear_driver.cpp")]


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(f"{ROCM}/lib/libamdhip64.so"):
        pytest.skip("needs g++ and the HIP runtime library")
    tmp = tmp_path_factory.mktemp("linear_host")
    objs = [str(tmp / (os.path.basename(s) + ".o")) for s in SOURCES]
    procs = [subprocess.Popen([gxx, *FLAGS, "-c", s, "-o", o], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for s, o in zip(SOURCES, objs)]
    for s, p in zip(SOURCES, procs):
        out = p.communicate(timeout=600)[0]
        assert p.returncode == 0, f"compile of {s} failed:\n{out}"
    exe = str(tmp / "driver")
    r = subprocess.run([gxx, "-fsanitize=address,undefined", *objs, f"-L{ROCM}/lib", "-lamdhip64",
                        f"-Wl,-rpath,{ROCM}/lib", "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr

    def run(*args, text=""):
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
        r = subprocess.run([exe, *args], input=text, capture_output=True, text=True, timeout=600, env=env)
        assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
        return r.stdout, r.stderr
    return run


def test_random_calls(driver):
    out, kernels = driver()
    counts = dict(zip(out.split()[0::2], map(int, out.split()[1::2])))
    assert counts["calls"] >= 100_000 and counts["split"] > 10_000
    assert set(kernels.strip().split("\n")) == every_kernel()


def test_no_exception_leaves_a_c_entry(driver):
    """Each host allocation of each call failing in turn: a status and a message come back."""
    out, _ = driver("nomem")
    assert int(out.split()[1]) >= 10


def every_kernel():
    """What the library is compiled for, by name: kernel, what its two weight operands mean, and their layouts."""
    forward = ["one a w", "one a w^T", "dual a w", "dual a w^T"]
    grads = ["cat a w", "cat a w^T", "one a^T w", "pair a^T w"]
    names = set()
    for t in ("bf16", "f32"):
        for edge in (64, 128):
            names |= {f"{t} general{edge} {m}" for m in forward + grads}
        names |= {f"{t} general64 {m} split" for m in forward + grads}
        names |= {f"{t} rows16 {m}" for m in forward} | {f"{t} rows16 {m} split" for m in forward}
        for rows in (32, 64):       # a k-contiguous weight only
            names |= {f"{t} rows{rows} {m}{s}" for m in forward if m.endswith("w^T") for s in ("", " split")}
        names |= {f"{t} activation gradient", f"{t} gated gradient, flat", f"{t} gated gradient, rows"}
    for tile in ("tile256", "tile192", "tile128w", "tile128", "tile64", "tile64short", "tile64k32"):
        for m in forward + grads:
            if (tile == "tile256" and "a^T" in m) or (tile == "tile192" and m.startswith("dual")):
                continue            # no such instance
            names.add(f"{tile} {m}")
            if tile.startswith("tile64"):
                names.add(f"{tile} {m} split")
    return names


def test_the_gpu_tests_reach_every_kernel(driver):
    out, _ = driver("choose", text="\n".join(" ".join(map(str, c)) for c in CASES))
    chosen = [line.split("; ") for line in out.strip().split("\n")]
    assert len(chosen) == len(CASES)
    assert set(k for line in chosen for k in line) == every_kernel()
    # Large tiles turn over their stages, and are not only run at one.
    deep = set()
    for (op, _, _, M, K, N, _), names in zip(CASES, chosen):
        for k in names:
            terms = M if "a^T" in k else N if op.endswith("bwd") else K
            if terms >= 160:
                deep.add(k)
    assert all(k in deep for k in every_kernel() if "128" in k or "256" in k or "192" in k)


def test_few_rows_against_wide_weights(driver):
    """The few-row kernel where it was measured to be the faster one: with a workspace, and (op ending in -) without."""
    rows = [("linear", 4096, 2048), ("linear", 4096, 4096), ("gated", 4096, 2048), ("linear-", 4096, 6144), ("gated-", 4096, 4096),
            ("linear-", 6144, 6144)]
    tiles = [("linear", 4096, 6144), ("linear", 8192, 4096), ("linear", 6144, 8192), ("gated", 6144, 4096),
             ("linear-", 8192, 8192), ("gated-", 4096, 8192)]
    text = "\n".join(f"{op} bf16 linear {M} {K} {N} 0" for M in (17, 32) for op, K, N in rows + tiles)
    out, _ = driver("choose", text=text)
    assert ["rows" in line for line in out.strip().split("\n")] == ([True] * len(rows) + [False] * len(tiles)) * 2


@pytest.mark.parametrize("rows", [17, 24, 32, 33, 47, 64])
def test_a_workspace_suffices_whatever_the_alignment(rows):
    """A workspace is asked for before addresses are known, for the kernels that need aligned rows: one K fewer has the same
    steps and always runs on the unaligned ones."""
    lib = _abi.load()
    n = C.c_int64()

    def size(fn, args):
        assert getattr(lib, fn)(C.byref(args), C.byref(n)) == 0, lib.tp_last_error()
        return n.value
    for N in list(range(1, 200, 7)) + list(range(200, 9000, 611)):
        for K in list(range(32, 2080, 96)) + list(range(2080, 16000, 992)):
            for fn, make in (("tp_linear_ws", lambda k: _abi.tp_linear_args(weight_layout=1, dtype=1, M=rows, N=N, K=k)),
                             ("tp_gated_linear_ws", lambda k: _abi.tp_gated_args(weight_layout=1, dtype=1, M=rows, F=N, K=k))):
                assert size(fn, make(K)) >= size(fn, make(K - 1)), (fn, rows, N, K)
