"""Compile flags of the library, apart from the list of its sources (build.py): the digest of
a kernel's code (profiling.py) takes in this file, and another source leaves it as it is."""
ARCH = "gfx950"
OPTIMIZE = ["-O3", "-std=c++17", "-fPIC"]
DEVICE = ["--offload-arch=" + ARCH, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
# per-source device flags: the WY-factor, scan and KDA kernels keep MFMA
# accumulators in VGPRs; the gradient and forward-output kernels are left to
# the compiler's register-class heuristics
SOURCE_FLAGS = {"gdr_prep.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
                "gdr_scan.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
                "kda_bwd.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}
