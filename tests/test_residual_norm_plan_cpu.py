"""How the joint's kernels divide a call: the plan is host code, taken from the source
and compiled by itself.  Every row of up to 7168 columns has a ring (longer ones are
read again for every pass), whatever the type and the number of rows; what the plan
takes fits.  Nothing here touches a device."""
import ctypes
import os
import re
import subprocess

import pytest

from routed_grouped_gemm_routing_gb300 import build

TEXT = open(os.path.join(build.CSRC, "residual_norm.cuh")).read()
MAX_H = 7168


def _cut(start, end):
    at = TEXT.index(start)
    return TEXT[at:TEXT.index(end, at)]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    consts = "".join(m.group(0) + "\n" for m in re.finditer(r"^constexpr int kRn(?!Long)\w+ = [^;]+;", TEXT, re.M))
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(consts + _cut("struct RnShape {", "\n};") + "\n};\n" + _cut("int rn_group_threads", "// Few rows in a backward") + """
extern "C" int plan(long long rows, int H, int elt, int tensors, int threads, int params, int spread, int* out) {
    RnShape s = {};
    s.rows = rows, s.H = H;
    const bool ok = rn_plan(s, elt, tensors, threads, params, out, out + 1, spread);
    out[2] = s.groups, out[3] = s.nt, out[4] = s.stages, out[5] = s.in_smem, out[6] = s.row_bytes;
    return ok;
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", so, src], check=True)
    f = ctypes.CDLL(str(so)).plan
    f.argtypes = [ctypes.c_longlong] + [ctypes.c_int] * 6 + [ctypes.c_void_p]
    out = (ctypes.c_int * 7)()

    def call(*args):
        return (bool(f(*args, out)), *out)

    return call


def _number(name):
    m = re.search(rf"\b{name} = ([^,;]+)[,;]", TEXT)
    return eval(re.sub(r"\b(kRn\w+)\b", lambda n: str(_number(n.group(1))), m.group(1)))


WIDTHS = [1, 31, 32, 33, 128, 255, 256, 257, 512, 513, 768, 1000, 1024, 1025, 1536, 1537, 1700, 1792, 1793, 2048, 2049, 2816, 3328,
          3329, 3500, 3584, 3585, 4096, 5120, 6144, 7000, 7161, MAX_H]
ROWS = [1, 2, 9, 60, 152, 153, 300, 457, 913, 1217, 1825, 3497, 5000, 8192, 100_000, 2 ** 31 - 1]


@pytest.mark.parametrize("elt", [2, 4])
@pytest.mark.parametrize("tensors", [2, 4])
def test_every_width_has_a_ring(plan, elt, tensors):
    smem_most, red, cols = _number("kRnSmem"), _number("kRnRedBytes"), _number("kRnCols")
    for H in WIDTHS:
        for rows in ROWS:
            for threads in (896, 1024):
                for params in (1, 2, 3, 4, 5):
                    for spread in (152, 8):
                        ok, blocks, smem, groups, nt, stages, held, row_bytes = plan(rows, H, elt, tensors, threads, params, spread)
                        at = (H, rows, threads, params, spread)
                        assert ok, at
                        assert 1 <= groups and groups * nt <= threads and nt % 32 == 0 and nt * cols >= H, at
                        assert nt == 32 or groups <= 15, at
                        assert 2 <= stages <= 4 and 0 <= held <= params and 1 <= blocks <= spread, at
                        need = groups * red + held * nt * cols * 4 + stages * groups * tensors * row_bytes
                        assert smem == need <= smem_most and row_bytes >= H * elt + 15, at
                        if tensors == 4:  # the backward's four column sums take the rings' place
                            assert 4 * groups * cols * nt * 4 <= stages * groups * tensors * row_bytes, at


def test_longer_rows_have_none(plan):
    assert not plan(100, MAX_H + 1, 2, 4, 896, 1, 152)[0]
