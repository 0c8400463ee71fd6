"""The binding's structures are the C header's: sizes and the places of the fields, as the C compiler has them."""

import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT
from ring_all_reduce_02_gb300 import ra

STRUCTS = {"ra_options_t": ra.Options, "ra_adamw_tensor_t": ra.AdamwTensor, "ra_adamw_options_t": ra.AdamwOptions}


def test_structures(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = []
    for name, struct in STRUCTS.items():
        lines.append(f'printf("%zu", sizeof({name}));')
        lines += [f'printf(" %zu %zu", offsetof({name}, {f}), sizeof((({name}*)0)->{f}));' for f, _ in struct._fields_]
        lines.append('printf("\\n");')
    (tmp_path / "structs.c").write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ra.h"\nint main(void) {\n' + "\n".join(lines)
                                        + "\nreturn 0;\n}\n")
    exe = str(tmp_path / "structs")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", f"-I{os.path.join(ROOT, 'include')}", str(tmp_path / "structs.c"), "-o", exe],
                   check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    for line, (name, struct) in zip(got, STRUCTS.items()):
        fields = [getattr(struct, f) for f, _ in struct._fields_]
        want = [ctypes.sizeof(struct)] + [n for f in fields for n in (f.offset, f.size)]
        assert [int(v) for v in line.split()] == want, name
