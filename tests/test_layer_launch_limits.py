"""The operators around the output layer over matrices that are larger than any
box's memory, without a GPU: the library runs in a child process on a recorder in
place of the HIP runtime (launches/recorder.cpp), which refuses a launch of 2^32
work-items as the runtime does."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(ROOT, "fp32_reductions_amd", "libreduce.so")

CHILD = r"""
import ctypes
fake = ctypes.CDLL({recorder!r}, mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL({library!r})
for name in ("launches", "largest", "allocations", "frees"):
    getattr(fake, "recorded_" + name).restype = ctypes.c_uint64
P, SZ, I, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
A = 0x7F0000000000  # in place of every pointer; nothing reads it
B, C, D_ = A + (1 << 40), A + (2 << 40), A + (3 << 40)
CALLS = {{
    "add_rmsnorm": [(P, A), (SZ, "rows"), (SZ, "n"), (SZ, "n"), (P, A), (SZ, "n"), (P, A),
                    (F, 1e-6), (P, B), (SZ, "n"), (P, C), (SZ, "n"), (P, D_), (SZ, "n"), (P, A),
                    (P, A), (P, None)],
    "rmsnorm_grad": [(P, A), (SZ, "rows"), (SZ, "n"), (SZ, "n"), (P, A), (P, A), (P, A),
                     (SZ, "n"), (P, A), (SZ, "n"), (P, B), (SZ, "n"), (P, C), (I, 0), (P, None)],
    "router_balance": [(P, A), (SZ, "rows"), (SZ, "n"), (SZ, "n"), (P, A), (SZ, 8), (SZ, 8),
                       (P, A), (F, 0.1), (F, 0.1), (P, B), (I, 0), (P, C), (P, D_), (P, A),
                       (SZ, "n"), (P, None)],
    "linear_ce": [(P, A), (SZ, "rows"), (SZ, "n"), (SZ, "n"), (P, A), (SZ, "V"), (SZ, "n"), (P, A),
                  (P, A), (F, 1.0), (F, 0.1), (P, B), (I, 0), (P, A), (P, A), (P, C), (SZ, "n"),
                  (P, D_), (SZ, "n"), (P, A), (SZ, (1 << 63)), (P, None)],
}}

def call(op, t, **size):
    args = CALLS[op]
    fn = getattr(lib, "red_%s_%s" % (op, t))
    fn.restype, fn.argtypes = I, [a for a, _ in args]
    fake.record_from_here()
    status = fn(*[size.get(v, v) if isinstance(v, str) else v for _, v in args])
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


SIZES = {
    "add_rmsnorm": [(1, 1), (7, 16384), ((1 << 31) + 9, 16384), ((1 << 40) + 1, 64), (1 << 45, 1)],
    "rmsnorm_grad": [(1, 1), (7, 16384), ((1 << 31) + 9, 16384), ((1 << 40) + 1, 64), (1 << 45, 1)],
    "router_balance": [(1, 1), (9, 2048), ((1 << 31) - 1, 2048), ((1 << 31) - 1, 8), (100, 64)],
    "linear_ce": [(1, 8, 1), (1, 65536, 1 << 24), (64, 1024, 1 << 24), (200, 4096, 1 << 24),
                  (1 << 20, 8, 1 << 24), (1 << 20, 65536, 1 << 24), (1 << 20, 65536, 7),
                  (4096, 4096, 131072)],
}


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("op", SIZES)
def test_no_launch_passes_the_limit(run, op, t):
    if (op, t) == ("linear_ce", "f32"):
        pytest.skip("the cross entropy takes 16-bit rows")
    names = ("rows", "n", "V")
    out = run("for size in %r:\n    print(*size, *call(%r, %r, **dict(zip(%r, size))))\n"
              % (SIZES[op], op, t, names))
    assert len(out) == len(SIZES[op])
    for line in out:
        *_, status, launches, largest = map(int, line.split())
        assert (status, launches > 0) == (0, True), line
        assert 0 < largest < 1 << 32, line


@pytest.mark.parametrize("op", ["rmsnorm_grad", "router_balance"])
def test_out_of_host_memory_is_a_status(run, op):
    out = run("fake.set_out_of_host_memory(1)\n"
              "print(*call(%r, 'bf16', rows=3000, n=500), fake.recorded_allocations())\n"
              "fake.set_out_of_host_memory(0)\n"
              "print(*call(%r, 'bf16', rows=3000, n=500), fake.recorded_allocations())\n"
              % (op, op))
    status, launches, _, _ = map(int, out[0].split())
    assert (status, launches) == (3, 0)  # RED_ERR_NOMEM
    status, launches, _, allocated = map(int, out[1].split())
    assert status == 0 and launches > 0 and allocated == 1


def test_workspace_sizes(run):
    """The query on the recorder: what a call needs grows with its rows, and with the
    vocabulary only by the joined sums, 8 bytes a row and tile."""
    out = run("f = lib.red_linear_ce_workspace_bf16\n"
              "f.restype, f.argtypes = I, [SZ, SZ, SZ, I, I, P]\n"
              "def size(*a):\n"
              "    n = ctypes.c_size_t()\n"
              "    assert f(*a, ctypes.byref(n)) == 0\n"
              "    return n.value\n"
              "for V in (32768, 131072, 1048576):\n"
              "    print(size(4096, 4096, V, 0, 0), size(4096, 4096, V, 1, 1))\n")
    forward, both = zip(*(map(int, line.split()) for line in out))
    assert forward[0] < forward[1] < forward[2] < (1 << 28)
    assert both[1] < (1 << 29) + (1 << 28) and both[2] < (1 << 29) + (1 << 28)
    assert both[0] < (1 << 30) + (1 << 28)
