"""The joint's sums over a group of many warps go through shared memory: parts, a
barrier, results, a barrier, and every warp reads the results.  Nothing holds a fast
warp back between that read and the next call's parts, so those must not lie where
the results of the call before are, whatever number of sums either call has.  The
places are taken from the source and checked here; nothing touches a device."""
import itertools
import os
import re

from routed_grouped_gemm_routing_gb300 import build

TEXT = open(os.path.join(build.CSRC, "residual_norm.cuh")).read()


def _number(name):
    """A constexpr int of the source."""
    m = re.search(rf"\b{name} = ([^,;]+)[,;]", TEXT)
    return eval(re.sub(r"\b(kRn\w+)\b", lambda n: str(_number(n.group(1))), m.group(1)))


def _phases():
    """Subscripts of r in the branch for many warps: before, between and after its barriers."""
    at = TEXT.index("float* r = reinterpret_cast<float*>(red);")
    body = re.sub(r"//[^\n]*", "", TEXT[at:TEXT.index("float sum(float a)", at)])
    parts = body.split("sync();")
    assert len(parts) == 3
    return [re.findall(r"\br\[([^\]]+)\]", p) for p in parts]


def _places(subscripts, N, warps):
    """Every value that the subscripts take."""
    out = set()
    for s in subscripts:
        code = compile(re.sub(r"\b(kRn\w+)\b", lambda n: str(_number(n.group(1))), s), s, "eval")
        for i, warp, lane in itertools.product(range(N), range(warps), range(4)):
            out.add(eval(code, {"N": N, "i": i, "warp": warp, "lane": lane}))
    return out


def test_the_next_calls_parts_leave_the_results_alone():
    before, between, after = _phases()
    assert before and between and after
    for warps in (9, 28, 32):
        for n1, n2 in itertools.product((1, 2, 3), repeat=2):
            read, written = _places(after, n1, warps), _places(before, n2, warps)
            assert not read & written, (warps, n1, n2, sorted(read & written)[:4])


def test_everything_lies_within_the_groups_bytes():
    before, between, after = _phases()
    for N in (1, 2, 3):
        places = _places(before, N, 32) | _places(after, N, 32) | {p for p in _places(between, N, N)}
        assert 0 <= min(places) and 4 * (max(places) + 1) <= _number("kRnRedBytes")
        # what is read at the end is what was written between the barriers
        assert _places(after, N, 32) == _places(between, N, N)
