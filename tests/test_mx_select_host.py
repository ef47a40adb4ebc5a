"""Which kernel a product of two MXFP4 operands takes (csrc/wq_mx_select.hpp, compiled here for the CPU): the
sizes that the GPU tests run reach every kernel, and the rules' limits lie where the header says."""
import ctypes
import os
import subprocess

import pytest

from mx_cases import DENSE, EXPERTS, KERNELS, rows_of_last_tiles

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_bit_amd", "csrc")
SOURCE = """
#include "wq_mx_select.hpp"
extern "C" int dense(int64_t m, int64_t n, int64_t k) { return wq::mx_dense_kernel(m, n, k); }
extern "C" int experts(int64_t gathered, int64_t pairs, int64_t n, int64_t k, int64_t e) {
  return wq::mx_experts_kernel(gathered, pairs, n, k, e);
}
extern "C" int number(int i) {
  constexpr wq::MxKernel names[] = {NAMES};
  return names[i];
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("select")
    src, so = d / "select.cpp", d / "select.so"
    src.write_text(SOURCE.replace("NAMES", ", ".join("wq::" + k for k in KERNELS)))
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(src), "-o", str(so)],
                   check=True)
    L = ctypes.CDLL(str(so))
    for f, n in ((L.dense, 3), (L.experts, 5)):
        f.argtypes = [ctypes.c_int64] * n
    assert [L.number(i) for i in range(len(KERNELS))] == list(range(len(KERNELS)))
    return L


def _dense(lib, m, n, k):
    return KERNELS[lib.dense(m, n, k)]


def _experts(lib, gathered, pairs, n, k, e):
    return KERNELS[lib.experts(gathered, pairs, n, k, e)]


def test_dense_cases_take_their_kernels(lib):
    for c in DENSE:
        assert _dense(lib, c.m, c.n, c.k) == c.kernel, c
    assert {c.kernel for c in DENSE} == set(KERNELS)
    for kernel, height, classes in (("MX_TILES_256", 256, {0, 1, 2}), ("MX_TILES_128x256", 128, {0, 1}),
                                    ("MX_TILES_128x256_ONE", 128, {0, 1}), ("MX_TILES_128", 128, {0, 1})):
        assert set().union(*(rows_of_last_tiles([c.m], height) for c in DENSE if c.kernel == kernel)) == classes, kernel
    # two-buffer tiles with an odd and an even number of stages, each ending inside one
    for kernel in ("MX_TILES_64", "MX_TILES_128", "MX_TILES_128x256", "MX_TILES_256"):
        assert any(c.k % 256 and c.k > 768 for c in DENSE if c.kernel == kernel), kernel


def test_experts_cases_take_their_kernels(lib):
    for c in EXPERTS:
        assert sum(c.counts) <= c.t * c.topk
        got = _experts(lib, c.t if c.gate_up else 0, c.t * c.topk, c.n, c.k, len(c.counts))
        assert got == c.kernel, (c, got)
    for gate_up in (True, False):
        some = [c for c in EXPERTS if c.gate_up == gate_up]
        assert {c.kernel for c in some} == set(KERNELS) - {"MX_STREAM_32", "MX_TILES_64"}
        for kernel, height, classes in (("MX_TILES_256", 256, {0, 1, 2}), ("MX_TILES_128x256", 128, {0, 1}),
                                        ("MX_TILES_128x256_ONE", 128, {0, 1}), ("MX_TILES_128", 128, {0, 1})):
            assert set().union(*(rows_of_last_tiles(c.counts, height) for c in some if c.kernel == kernel)) == classes


def test_limit_of_gathered_tokens(lib):
    """gate+up's tiles address all tokens' codes with 32 bits: 524287 tokens of hidden 8192 at most.  Down's
    rows are addressed tile by tile and have no such limit."""
    for t, kernel in ((524287, "MX_TILES_256"), (524288, "MX_STREAM_16")):
        assert _experts(lib, t, 8 * t, 3584, 8192, 64) == kernel
        assert _experts(lib, 0, 8 * t, 8192, 3584, 64) == "MX_TILES_256"


def test_limits_of_the_tiles(lib):
    assert _dense(lib, 4096, 8192, 256).startswith("MX_TILES") and _dense(lib, 4096, 8192, 192) == "MX_STREAM_32"
    assert _dense(lib, 33, 1 << 20, 2048).startswith("MX_TILES")
    # one expert's codes: n k / 2 up to 2^31 - 1024
    assert _dense(lib, 64, (1 << 20) - 1, 4096).startswith("MX_TILES") and _dense(lib, 64, 1 << 20, 4096) == "MX_STREAM_32"
    assert _dense(lib, 1 << 16, 256, (1 << 23) - 64).startswith("MX_TILES")
    assert _dense(lib, 1 << 16, 256, 1 << 23).startswith("MX_STREAM")
    assert _dense(lib, 32, 1 << 20, 1024) == "MX_STREAM_32" and _dense(lib, 1, 28672, 4096) == "MX_STREAM_16"
