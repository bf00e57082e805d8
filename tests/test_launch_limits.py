"""Calls over matrices that are larger than any box's memory, without a GPU:
the library runs in a child process on a recorder in place of the HIP runtime
(launches/recorder.cpp), which refuses a launch of 2^32 work-items as the
runtime does."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(ROOT, "fp32_reductions_amd", "libreduce.so")

CHILD = r"""
import ctypes, sys
fake = ctypes.CDLL({recorder!r}, mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL({library!r})
for name in ("launches", "largest", "allocations", "frees"):
    getattr(fake, "recorded_" + name).restype = ctypes.c_uint64
P, SZ, I, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
A = 0x7F0000000000  # in place of every pointer; nothing reads it
MATRIX = [(P, A), (SZ, "rows"), (SZ, "V"), (SZ, "V")]
GRADIENT = [(P, A), (SZ, "V"), (P, None)]  # in place, on the null stream
CALLS = {{
    "token_logprob": MATRIX + [(P, A), (F, 1.0)] + 3 * [(P, A)] + [(P, None)],
    "token_logprob_grad": MATRIX + [(P, A), (F, 1.0)] + 4 * [(P, A)] + GRADIENT,
    "distill_topk": MATRIX + [(P, A), (P, A), (SZ, 4), (SZ, 4), (P, A), (P, A), (F, 1.0), (P, A),
                              (I, 0), (P, A)] + GRADIENT,
    "policy_loss": MATRIX + 5 * [(P, A)] + [(F, 1.0), (F, 0.2), (F, 0.2), (F, 0.1), (F, 0.1),
                                            (P, A), (I, 0), (P, A), (P, A)] + GRADIENT,
    "preference_loss": MATRIX + [(P, A), (P, A), (SZ, 2), (P, A), (P, A), (I, 0), (F, 0.1),
                                 (F, 0.0), (F, 0.0), (I, 0), (P, A), (I, 0), (P, A)] + GRADIENT,
}}

def call(op, t, rows, V):
    args = CALLS[op]
    fn = getattr(lib, "red_%s_%s" % (op, t))
    fn.restype, fn.argtypes = I, [a for a, _ in args]
    fake.record_from_here()
    status = fn(*[dict(rows=rows, V=V).get(v, v) if isinstance(v, str) else v for _, v in args])
    return status, fake.recorded_launches(), fake.recorded_largest()

"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """run(code): the lines that `code` prints in a child on the recorder."""
    if not os.path.exists(LIBRARY):
        pytest.skip("libreduce.so is not built")
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    recorder = str(tmp_path_factory.mktemp("launches") / "recorder.so")
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC",
                    os.path.join(TESTS, "launches", "recorder.cpp"), "-o", recorder], check=True)

    def child(code):
        code = CHILD.format(recorder=recorder, library=LIBRARY) + code
        p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                           timeout=300)
        assert p.returncode == 0, (p.returncode, p.stdout[-2000:], p.stderr[-2000:])
        return p.stdout.splitlines()

    return child


# (rows, V): a few rows that are cut into segments, up to the longest that the
# calls accept; many rows; more than one launch covers.
SIZES = [(1, 1), (64, 1 << 30), (128, 1 << 29), (128, 1 << 30), (128, (1 << 31) - 8),
         (4096, (1 << 31) - 8), (1 << 19, 262144), ((1 << 21) + 9, 5000), ((1 << 24) + 9, 33)]


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("op", ["token_logprob", "token_logprob_grad", "distill_topk",
                                "policy_loss", "preference_loss"])
def test_no_launch_passes_the_limit(run, op, t):
    sizes = [(r, v) for r, v in SIZES if (op != "distill_topk" or v <= 393216)
             and (op != "preference_loss" or r <= 1 << 19)]
    out = run("for size in %r:\n    print(*size, *call(%r, %r, *size))\n" % (sizes, op, t))
    assert len(out) == len(sizes)
    for line in out:
        rows, V, status, launches, largest = map(int, line.split())
        assert (status, launches > 0) == (0, True), line
        assert 0 < largest < 1 << 32, line


@pytest.mark.parametrize("op", ["policy_loss", "preference_loss", "distill_topk"])
def test_out_of_host_memory_is_a_status(run, op):
    """No exception leaves a C entry point: the call returns the status of a
    failed workspace, holds nothing, and the next one works."""
    out = run("fake.set_out_of_host_memory(1)\n"
              "first = call(%r, 'bf16', 3, 5000)\n"
              "print(*first, fake.recorded_allocations() - fake.recorded_frees())\n"
              "fake.set_out_of_host_memory(0)\n"
              "print(*call(%r, 'bf16', 3, 5000), fake.recorded_allocations())\n" % (op, op))
    status, launches, _, held = map(int, out[0].split())
    assert (status, launches, held) == (3, 0, 0)  # RED_ERR_NOMEM
    status, launches, _, allocated = map(int, out[1].split())
    assert status == 0 and launches > 0 and allocated == 1
