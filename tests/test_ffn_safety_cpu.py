"""What the feed-forward operators must not do, shown without a GPU: reads past
their operands, buffers that another stream may take, results cut from a graph."""
import os
import re
import subprocess

import pytest


@pytest.fixture(scope="module")
def iq():
    import int_quantization_amd as m
    if not os.path.exists(m.LIB_PATH):
        from int_quantization_amd import build
        build.build()
    m.load_library()
    return m


def kernels(source, name, tmp_path):
    """{mangled name: [instructions]} of the kernels of csrc/`source` whose name holds `name`, as the compiler writes them."""
    from int_quantization_amd import build
    out = tmp_path / "device.s"
    subprocess.run(["/opt/rocm/bin/hipcc", *build.HIPCC_FLAGS, "-I", os.path.join(build.ROOT, "include"), "--cuda-device-only", "-S",
                    "-o", str(out), os.path.join(build.ROOT, "int_quantization_amd", "csrc", source)], check=True, capture_output=True)
    found, code = {}, None
    for line in out.read_text().splitlines():
        label = re.match(r"(_Z\S*%s\S*):" % name, line)
        if label:
            code = found[label[1]] = []
        elif line.startswith(".Lfunc_end"):
            code = None
        elif code is not None:
            c = line.split(";")[0].strip()
            if c and not c.startswith(".") and not c.endswith(":"):
                code.append(c)
    return found


# ---- reads of packed codes ------------------------------------------------------------
def test_packed_code_loads_carry_their_whole_offset_in_the_range_check(tmp_path):
    """A buffer load compares its vector offset with the buffer's size less its scalar offset, as unsigned numbers, so a
    scalar offset past the buffer's end lets every load through.  Loads of weights past a row's last step are ordinary
    (the batch ahead), and a workgroup may hold a single row shorter than a step: their scalar offset has to be zero."""
    loads = 0
    for name, code in kernels("iq_packed.hip", "k_packed", tmp_path).items():
        for c in code:
            m = re.match(r"buffer_load_dwordx4 \S+ \S+ \S+ (\S+) offen(.*)", c)
            if m and " lds" not in m[2]:
                assert m[1] == "0", f"{name}: {c}"
                loads += 1
    assert loads > 100


@pytest.mark.parametrize("cols", range(32, 289, 32))
def test_packed_code_offsets_stay_in_their_rows(cols):
    """The kernel's offsets in numbers: lane (row, quarter h) of a step reads 16 bytes from row * K / 2 + 16 h + 64 step, steps
    past the matrix standing for its end; what the range check lets through lies in the workgroup's rows."""
    row_bytes, steps = cols // 2, -(-cols // 128)
    for rows in (1, 2, 3, 15, 16, 17, 32):
        size = rows * row_bytes
        for step in range(steps + 4):
            for row in range(rows):
                for h in range(4):
                    at = row * row_bytes + 16 * h + 64 * min(step, steps)
                    if at < size:
                        assert at + 16 <= size
