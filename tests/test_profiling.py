"""CPU tests of the profile bookkeeping: a traffic summary stays valid while
its kernel's code is unchanged (comments and layout do not count) and is
ignored once the code changes."""
import shutil

import pytest

from chunked_gated_delta_08_amd import profiling


def test_code_digest_ignores_comments_and_layout():
    a = "int f(int x) {\n    return x + 1;   // one more\n}\n/* trailing\n   block */\n"
    b = "// header\nint f(int x) { return x + 1; }\n"
    c = "int f(int x) {\n    return x + 2;   // one more\n}\n"
    assert profiling._code_of(a) == profiling._code_of(b)
    assert profiling._code_of(a) != profiling._code_of(c)
    # a line broken inside a call is the same code; a space between two names is not dropped
    assert profiling._code_of("x = f(g(y));") == profiling._code_of("x = f(\n    g(y));")
    assert profiling._code_of("int x;") != profiling._code_of("intx;")


def test_code_digest_follows_the_files(tmp_path, monkeypatch):
    monkeypatch.setattr(profiling, "ROOT", str(tmp_path))
    f = tmp_path / "k.hip"
    f.write_text("__global__ void k() { }  // v1\n")
    d1 = profiling.source_digest(["k.hip"])
    f.write_text("// a note\n__global__ void k()\n{\n}\n")
    assert profiling.source_digest(["k.hip"]) == d1
    f.write_text("__global__ void k() { int x = 0; }\n")
    assert profiling.source_digest(["k.hip"]) != d1


@pytest.mark.skipif(shutil.which("c++filt") is None, reason="names stay as they are without c++filt")
def test_kernel_names_in_clear():
    name = "_ZN5layer12_GLOBAL__N_114glr_fwd_kernelI%sLi2ELi12EEEvNS_7GlrArgsEiib"
    clear = "void layer::(anonymous namespace)::glr_fwd_kernel<%s, 2, 12>(layer::GlrArgs, int, int, bool)"
    for code, t in (("DF16b", "bf16"), ("DF16_", "half"), ("f", "float")):
        assert profiling.readable(name % code) == clear % t
        assert profiling.short_name(name % code) == profiling.short_name(clear % t) == "glr_fwd_kernel"
    both = "_ZN5layer12_GLOBAL__N_119add_norm_fwd_kernelIDF16bfLi4ELi256ELi2ELb1EEEvNS_8NormArgsE"
    assert profiling.readable(both) == "void layer::(anonymous namespace)::add_norm_fwd_kernel<bf16, float, 4, 256, 2, true>(layer::NormArgs)"
    assert profiling.readable(both + ".kd") == profiling.readable(both)
    assert profiling.readable(clear % "float") == clear % "float"


def test_fills_are_the_evicting_write_in_the_bench_only(tmp_path):
    fill = "void at::native::vectorized_elementwise_kernel<4, at::native::FillFunctor<float>, x>(int)"
    csv = tmp_path / "k.csv"
    csv.write_text("Name,Calls,TotalDurationNs,AverageNs,Percentage,MinNs,MaxNs\n" +
                   f'"{fill}",3,5100,1700,50,1400,1900\n"layer::(anonymous namespace)::glr_clear_kernel(x)",3,5000,1700,50,1400,1900\n')
    for cmd, evicts in (("python3 bench.py --steps 5", True), ("python3 -m x.profiling layer --case y", False)):
        out = tmp_path / "out.txt"
        profiling.main(["stats", "--csv", str(csv), "--out", str(out), "--cmd", cmd])
        assert ("bench_evict_fill" in out.read_text()) == evicts
        assert "glr_clear_kernel" in out.read_text()
