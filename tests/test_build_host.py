"""Device code compiles without warnings of the compiler about inline assembly."""
import subprocess

import pytest

from mamba_ssd_chunked_amd import build

KERNEL = """
#include "delta_device.hpp"
namespace ssd {
__global__ void k(const float* src, float* dst) {
    __shared__ __align__(16) char sm[2048];
    load_to_lds(src + 4 * threadIdx.x, lds_addr(sm));
    load_to_lds(src + 256 + 4 * threadIdx.x, lds_addr(sm) + 1024);
    wait_barrier<0>();
    mfma_settle();
    dst[threadIdx.x] = reinterpret_cast<float*>(sm)[threadIdx.x];
}
}
"""


def test_loads_into_lds_leave_the_compilers_registers_as_they_were(tmp_path):
    """No reserved register on a clobber list (the compiler calls that undefined), and m0 holds after
    each load what it held before."""
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    src, out = tmp_path / "k.hip", tmp_path / "k.s"
    src.write_text(KERNEL)
    r = subprocess.run([hipcc, *build.FLAGS, "-S", "--offload-device-only", str(src), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0 and "inline asm" not in r.stderr, r.stderr
    ops = [line.split(";")[0].split() for line in out.read_text().splitlines()]
    ops = [(o[0], " ".join(o[1:])) for o in ops if o and "m0" in " ".join(o[1:]) or o and "lds_dwordx4" in o[0]]
    loads = [i for i, (op, _) in enumerate(ops) if "lds_dwordx4" in op]
    assert len(loads) == 2
    for i in loads:
        (_, keep), (_, put), (_, back) = ops[i - 2], ops[i - 1], ops[i + 1]
        reg = keep.split(",")[0]
        assert keep == f"{reg}, m0" and put.startswith("m0, s") and back == f"m0, {reg}" and put != back
