"""The host code of the vocabulary cross entropy and the AdamW step built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer: validation, workspace sizes and offsets, pieces, the choice of kernel, tiles and splits, driven
through random calls with exact and short workspaces.  The kernel launchers are stand-ins (tests/sanitizer/loss_stub.cpp)
that check every byte range a kernel would touch; no GPU is used.  The same build says which kernels a call launches."""
import os
import shutil
import subprocess

import pytest

from loss_kernel_cases import CASES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sharded_gemm_amd", "csrc")
SAN = os.path.join(ROOT, "tests", "sanitizer")
ROCM = "/opt/rocm"
FLAGS = ["-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
         "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include"]
SOURCES = [os.path.join(CSRC, f) for f in ("plan.cpp", "checker.cpp", "api.cpp", "timing.cpp", "linear_launch.cpp", "ce_api.cpp",
                                           "ce_launch.cpp", "adamw_api.cpp")] + \
          [os.path.join(SAN, f) for f in ("stub_kernels.cpp", "loss_stub.cpp", "loss_driver.cpp")]


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(f"{ROCM}/lib/libamdhip64.so"):
        pytest.skip("needs g++ and the HIP runtime library")
    tmp = tmp_path_factory.mktemp("loss_host")
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
    assert counts["calls"] >= 20_000
    assert own_kernels() <= set(kernels.strip().split("\n"))


def test_no_exception_leaves_a_c_entry(driver):
    """Each host allocation of each call failing in turn: a status and a message come back."""
    out, _ = driver("nomem")
    assert int(out.split()[1]) >= 10


def own_kernels():
    """What the library is compiled for beyond the linear layer's kernels, by name."""
    names = {"logits", "join", "transpose", "sum", "pad"}
    tiles = ("tile256", "tile192", "tile128w", "tile128", "tile64", "tile64short", "tile64k32")
    for mode in ("stats a w", "stats a w^T", "prob a w", "prob a w^T", "scaled a w", "scaled a w^T", "scaled a^T w^T"):
        for tile in tiles:
            if mode == "scaled a^T w^T" and tile == "tile64k32":
                continue            # tokens come in multiples of 64
            names.add(f"{tile} {mode}")
            if tile.startswith("tile64"):
                names.add(f"{tile} {mode} split")
    for t, modes in (("bf16", ("stats a w", "stats a w^T", "prob a w", "prob a w^T", "scaled a w", "scaled a w^T")),
                     ("f32", ("stats a w", "stats a w^T", "prob a w", "prob a w^T", "one a^T w^T"))):
        for mode in modes:
            names |= {f"{t} general64 {mode}", f"{t} general64 {mode} split", f"{t} general128 {mode}"}
    names |= {f"{tile} slices a {w}" for tile in ("tile256", "tile128w") for w in ("w", "w^T")}
    for mode in ("stats a w", "stats a w^T"):
        names |= {f"tile32 {mode}", f"tile32 {mode} split"}
    return names


def test_the_gpu_tests_reach_every_kernel(driver):
    out, _ = driver("choose", text="\n".join(" ".join(map(str, c)) for c in CASES))
    chosen = [line.split("; ") for line in out.strip().split("\n")]
    assert len(chosen) == len(CASES)
    missing = own_kernels() - set(k for line in chosen for k in line)
    assert not missing, sorted(missing)
