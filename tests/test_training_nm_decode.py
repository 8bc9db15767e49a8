"""The input gradient's decoding of N:M rows, the kernels' own function run on the host: it reads nothing behind the
packed buffers, which end here where readable memory ends, and gives the dense codes of every width."""
import ctypes
import mmap
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# the rows as the kernels walk them: to the dense row's end, K rounded up to 64 (the bf16 values' to 16, which is less)
HARNESS = """
#include "nm_decode.cuh"
extern "C" void expand(const uint8_t* codes, const uint8_t* meta, int64_t ldc, int64_t ldm, int N, int K, int n, int m,
                       uint32_t* out) {
  bl::ExpandArgs e = {};
  e.codes = codes;
  e.meta = meta;
  e.ldc = ldc;
  e.ldm = ldm;
  e.N = N;
  e.K = K;
  e.nm_n = n;
  e.nm_m = m;
  const int words = 4 * ((K + 63) / 64);
  for (int64_t r = 0; r < N; ++r)
    for (int w = 0; w < words; ++w) out[r * words + w] = bl::nm_codes16(e, r, 16 * w);
}
"""
PATTERNS = [(2, 4)] + [(n, 8) for n in range(1, 8)]
# every tail of a row: K around the multiples of 64 and 128 at which rows of codes and of positions grow, and the
# package's own widths
WIDTHS = sorted(set(range(8, 720, 8)) | {2048, 2560, 2568, 4104, 6912, 11000, 11008, 65528, 65536})


def _fenced(data):
    """A copy of `data` (bytes) that ends at the last readable byte of its mapping: its address."""
    libc = ctypes.CDLL(None, use_errno=True)
    libc.mmap.restype = ctypes.c_void_p
    libc.mmap.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_long]
    libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
    page = mmap.PAGESIZE
    size = (len(data) + page - 1) // page * page
    base = libc.mmap(None, size + page, mmap.PROT_READ | mmap.PROT_WRITE, mmap.MAP_PRIVATE | mmap.MAP_ANONYMOUS, -1, 0)
    assert base not in (None, ctypes.c_void_p(-1).value)
    assert libc.mprotect(base + size, page, 0) == 0
    at = base + size - len(data)
    ctypes.memmove(at, data, len(data))
    return at, base, size + page


def _matrix(N, K, n, m, rng):
    """A packed random N:M matrix by the layout's definition: (codes, meta, dense ternary + 1)."""
    blocks = K // m
    keep = np.sort(rng.random((N, blocks, m)).argsort(2)[:, :, :n], 2)
    val = rng.integers(0, 3, (N, blocks, n))
    dense = np.ones((N, blocks, m), np.int64)
    np.put_along_axis(dense, keep, val, 2)
    ldc, ldm = 16 * -(-blocks * n // 64), 16 * -(-K // 128)
    v = np.zeros((N, 4 * ldc), np.uint8)
    v[:, :blocks * n] = val.reshape(N, -1)
    codes = (v.reshape(N, ldc, 4) << np.array([0, 2, 4, 6], np.uint8)).sum(2).astype(np.uint8)
    meta = np.zeros((N, ldm), np.uint8)
    if m == 4:
        nib = np.zeros((N, 2 * ldm), np.uint8)
        nib[:, :blocks] = keep[:, :, 0] | (keep[:, :, 1] << 2)
        meta[:] = nib[:, ::2] | (nib[:, 1::2] << 4)
    else:
        meta[:, :blocks] = (1 << keep).sum(2)
    return codes, meta, dense.reshape(N, K)


def _check(lib, n, m, widths):
    L = ctypes.CDLL(lib)
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.expand.restype, L.expand.argtypes = None, [P, P, i64, i64, i32, i32, i32, i32, P]
    libc = ctypes.CDLL(None)
    libc.munmap.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
    rng = np.random.default_rng(10 * m + n)
    N = 2
    for K in widths:
        codes, meta, dense = _matrix(N, K, n, m, rng)
        (pc, *mc), (pm, *mm) = _fenced(codes.tobytes()), _fenced(meta.tobytes())
        words = 4 * -(-K // 64)
        out = np.zeros((N, words), np.uint32)
        print(K, flush=True)  # the last one printed is the one that read too far
        L.expand(pc, pm, codes.shape[1], meta.shape[1], N, K, n, m, out.ctypes.data)
        got = (out[:, :, None] >> np.arange(0, 32, 2, dtype=np.uint32)) & 3
        want = np.ones((N, 16 * words), np.int64)
        want[:, :K] = dense
        assert np.array_equal(got.reshape(N, -1), want), K
        libc.munmap(*mc)
        libc.munmap(*mm)


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    d = tmp_path_factory.mktemp("nm_decode")
    (d / "harness.cpp").write_text(HARNESS)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
                           "-I" + os.path.join(ROOT, "ternary_weight_linear_fwd_b200", "csrc"),
                           "-o", str(d / "harness.so"), str(d / "harness.cpp")])
    return str(d / "harness.so")


@pytest.mark.parametrize("n,m", PATTERNS)
def test_nm_rows_are_read_inside_their_buffers(harness, n, m):
    """In a process of its own, which a read behind a buffer ends."""
    r = subprocess.run([sys.executable, os.path.abspath(__file__), harness, str(n), str(m)], capture_output=True,
                       text=True)
    assert r.returncode == 0, (r.returncode, r.stdout.split()[-1:], r.stderr[-2000:])
    assert len(r.stdout.split()) == len(WIDTHS)


def test_layout_is_the_library_s():
    """The strides used here are those that callers allocate."""
    from ternary_weight_linear_fwd_b200 import build as b
    b.build()
    import ternary_weight_linear_fwd_b200 as bl
    rng = np.random.default_rng(0)
    for n, m in PATTERNS:
        for K in (8, 72, 264, 720, 11000):
            codes, meta, _ = _matrix(2, K, n, m, rng)
            assert bl.packed_layout(2, K, n, m)[:2] == (codes.shape[1], meta.shape[1])


if __name__ == "__main__":
    _check(sys.argv[1], int(sys.argv[2]), int(sys.argv[3]), WIDTHS)
