"""What the compiler says of the HIP sources (no GPU is needed)."""
import os
import subprocess

import pytest

from selective_state_space_65_amd import build

SOURCES = build.SRCS + [build.PROBE_SRC]


@pytest.mark.parametrize("source", SOURCES, ids=[os.path.basename(s) for s in SOURCES])
def test_no_index_is_past_its_array(source):
    """An index that the compiler sees to be past its array, LDS or registers, is a kernel that reads and writes what it does
    not own."""
    r = subprocess.run([build.hipcc()] + build.HIPCC_FLAGS + ["-Werror=array-bounds", "-I", build.INCLUDE, "--cuda-device-only",
                                                              "-fsyntax-only", source], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_warnings_are_seen(capfd, tmp_path):
    """The build passes on what the compiler says of a file that it compiles, and refuses an index past its array."""
    def compile(text):
        source = tmp_path / "one.hip"
        source.write_text("#include <hip/hip_runtime.h>\n" + text)
        build._run([[build.hipcc()] + build.HIPCC_FLAGS + ["-c", "-o", str(tmp_path / "one.o"), str(source)]], False)

    kernel = "__global__ void one(float* p) { __shared__ float a[1][4]; a[%d][threadIdx.x] = 1; p[0] = a[0][0]; %s}\n"
    compile(kernel % (0, ""))
    assert capfd.readouterr().err == ""
    compile(kernel % (0, "int left; "))
    assert "unused variable 'left'" in capfd.readouterr().err
    with pytest.raises(RuntimeError, match="one.hip"):
        compile(kernel % (1, ""))
    assert "past the end of the array" in capfd.readouterr().err


@pytest.mark.parametrize("io", ["float", "bf16_t"])
def test_loads_to_lds_wait_for_their_base(io, tmp_path):
    """The compiler counts no wait states inside inline assembly.  A scalar register that a vector instruction wrote (a spilled
    one that is read back from a lane, say) may be a vector load's base only five wait states later, so the assembly of a
    load straight to LDS has to hold five of its own in front of the load."""
    source = tmp_path / "one.hip"
    source.write_text('#include "linear_attn_kernel.h"\n'
                      "hipError_t one(const Args& a, hipStream_t st) { return launch_one<%s, 1, 2>(a, 1, false, st); }\n" % io)
    listing = tmp_path / "one.s"
    r = subprocess.run([build.hipcc()] + build.HIPCC_FLAGS + ["-I", build.INCLUDE, "-I", os.path.join(build.HERE, "csrc"),
                                                              "--cuda-device-only", "-S", "-o", str(listing), str(source)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    states, loads = 0, 0
    for line in listing.read_text().splitlines():
        op = line.split()
        if ";;#ASMSTART" in line:
            states = 0
        elif op and op[0].startswith("global_load_lds"):
            loads += 1
            assert states >= 5, "%d wait states before %s" % (states, line.strip())
        elif op and not op[0].startswith((";", ".")):
            states += int(op[1]) + 1 if op[0] == "s_nop" else 1
    assert loads > 0
