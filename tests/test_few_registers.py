"""CPU check of the form for few rows: its kernels' registers leave room for as
many workgroups a CU as a launch counts on, without spills."""
import os
import re
import subprocess

from group_scaling_fp8_amd import build as B

SOURCE = r"""
#include "mgs_kernels.hpp"
#include "mgs_mm_tile.hpp"
namespace mgs {
template <int PER_CU>
__global__ void counted(int) {}
template <class KIND>
void kernels(const MmArgs& p) {
    hipLaunchKernelGGL((mm_few_kernel<16, 32, 1, true, KIND>), dim3(1), dim3(512), 0, 0, p);
    hipLaunchKernelGGL((counted<kFewPerCu<16, 32, KIND>>), dim3(1), dim3(512), 0, 0, 0);
}
void all(const MmArgs& p) { kernels<KIND>(p); }
}  // namespace mgs
"""
KINDS = ("Rows, Num::Exact, false", "Rows, Num::Int8, false", "Gated, Num::Fast, false, true", "Gated, Num::Exact, false, true",
         "Gated, Num::Int8, false", "Grad, Num::Fast, false, true", "Grad, Num::Exact, false, true", "Grad, Num::Exact, false, false")


def compiled(args):
    d, kind, n = args
    src, out = d / ("few%d.hip" % n), d / ("few%d.s" % n)
    src.write_text(SOURCE.replace("<KIND>", "<Kind<Job::%s>>" % kind))
    flags = [f for f in B.HIPCC_FLAGS if f not in ("-shared", "-Wall")]
    subprocess.run([os.environ.get("HIPCC", "/opt/rocm/bin/hipcc"), *flags, "-w", "--cuda-device-only", "-S", "-I", B.INCLUDE,
                    "-I", B.CSRC, "-o", str(out), str(src)], check=True, capture_output=True)
    return out.read_text()


def test_registers_of_the_smallest_tiles(tmp_path):
    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(4) as pool:
        texts = list(pool.map(compiled, [(tmp_path, k, n) for n, k in enumerate(KINDS)]))
    for kind, text in zip(KINDS, texts):
        per_cu = int(re.search(r"\.amdhsa_kernel _ZN3mgs7countedILi(\d)E", text).group(1))
        meta = text[text.index("amdhsa.kernels:"):]
        few = [k for k in re.split(r"\n  - ", meta) if "mm_few_kernel" in k]
        assert len(few) == 1, kind
        value = lambda name: int(re.search(r"\.%s:\s+(\d+)" % name, few[0]).group(1))  # noqa: E731
        waves = 512 // (-(-value("vgpr_count") // 8) * 8)         # a SIMD's registers, given out by eights
        assert waves * 4 // 8 >= per_cu, (kind, value("vgpr_count"))
        assert value("vgpr_spill_count") == 0 and value("private_segment_fixed_size") == 0, kind
