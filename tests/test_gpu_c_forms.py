"""dspark_adjust, dspark_attend_sinks and dspark_attend_shared from plain C (tests/c_abi/forms_from_c.c):
the header's struct and argument order, as a C compiler lays them out, against the formulas in double."""
import ctypes
import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def compiled(tmp_path, source, *more):
    from speculative_decoding_ragged_gb300 import build
    exe = str(tmp_path / "program")
    r = subprocess.run([build.nvcc(), "-O2", "-I", os.path.join(ROOT, "include"), source, "-o", exe, *more],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_the_binding_lays_the_struct_out_as_c_does(tmp_path):
    from speculative_decoding_ragged_gb300._binding import _Adjustments
    with open(os.path.join(ROOT, "include", "dspark.h")) as f:
        body = re.search(r"typedef struct \{([^}]*)\} dspark_adjustments;", f.read()).group(1)
    names = re.findall(r"(\w+);", body)
    assert names == [n for n, _ in _Adjustments._fields_]
    source = tmp_path / "layout.c"
    source.write_text('#include <stddef.h>\n#include <stdio.h>\n#include <cuda_runtime.h>\n#include "dspark.h"\n'
                      'int main(void) {\n' +
                      "".join(f'printf("%zu ", offsetof(dspark_adjustments, {n}));\n' for n in names) +
                      'printf("%zu", sizeof(dspark_adjustments));\nreturn 0; }\n')
    run = subprocess.run([compiled(tmp_path, str(source))], capture_output=True, text=True, timeout=60)
    want = [getattr(_Adjustments, n).offset for n in names] + [ctypes.sizeof(_Adjustments)]
    assert [int(x) for x in run.stdout.split()] == want


@pytest.mark.gpu
def test_plain_c_caller_matches_the_formulas(tmp_path):
    from speculative_decoding_ragged_gb300 import build
    pkg = os.path.dirname(build.build())
    exe = compiled(tmp_path, os.path.join(HERE, "c_abi", "forms_from_c.c"), "-L", pkg, "-ldspark",
                   "-Xlinker", f"-rpath={pkg}", "-lm")
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr
