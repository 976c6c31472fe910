"""CPU test of what a kernel's digest takes in: the compile flags, not the library's list of sources.  A new source
would otherwise void the traffic summaries of kernels that it does not touch."""
import ast
import os

from chunked_gated_delta_08_amd import build, build_flags, profiling


def test_digests_take_in_the_flags_alone():
    names = {f for files in profiling.KERNEL_SOURCES.values() for f in files}
    assert all(os.path.exists(os.path.join(profiling.ROOT, f)) for f in names)
    assert all("chunked_gated_delta_08_amd/build_flags.py" in files for files in profiling.KERNEL_SOURCES.values())
    assert "chunked_gated_delta_08_amd/build.py" not in names
    assert build.DEVICE is build_flags.DEVICE and build.SOURCE_FLAGS is build_flags.SOURCE_FLAGS
    # every flag that the compiler is given stands in the flags' file; build.py has the include paths
    text = open(os.path.join(profiling.ROOT, "chunked_gated_delta_08_amd", "build.py"), encoding="utf-8").read()
    flags = {n.value for n in ast.walk(ast.parse(text)) if isinstance(n, ast.Constant) and isinstance(n.value, str)
             and n.value.startswith("-") and "\n" not in n.value}
    assert flags <= {"-I", "-c", "-o", "-shared", "-fPIC", "--offload-arch="}, flags
