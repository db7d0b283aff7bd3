"""The check of a projection kernel's registers at its launch: only a form that splits them (setmaxnreg) asks for the
count that the split was sized for.  Compiled with nvcc, no GPU call."""
import os
import shutil
import subprocess

import pytest

from joint_attention_gb300.build import ARCH, CFLAGS

PROGRAM = r"""
#include "qkv_proj.cuh"
using namespace jattn;
template <int D, int kMode>
constexpr int asked = QkvCfg<D, kMode, true>::kLaunchRegs;
// The forms with a split take their count, by eights, and no other.
static_assert(asked<64, kBf16> == QkvRegs::kLaunch && asked<128, kBf16> == QkvRegs::kLaunch, "");
static_assert(asked<64, kE4m3> == QkvRegs::kLaunch && asked<128, kE4m3> == QkvRegs::kLaunch, "");
static_assert(QkvRegs::fits(96, 96) && QkvRegs::fits(89, 96) && !QkvRegs::fits(88, 96) && !QkvRegs::fits(97, 96), "");
// Adapters have none: a build with fewer registers is as good.
static_assert(asked<64, kLora> == 0 && asked<128, kLora> == 0, "");
static_assert(QkvRegs::fits(88, 0) && QkvRegs::fits(96, 0) && QkvRegs::fits(40, 0), "");
int main() { return 0; }
"""


def test_register_check_is_of_the_forms_with_a_split(tmp_path):
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "regs.cu"
    src.write_text(PROGRAM)
    r = subprocess.run([nvcc, *ARCH, *CFLAGS, "-c", str(src), "-o", str(tmp_path / "regs.o")], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
