"""The structs of the serving calls: the ctypes mirrors agree with the header."""
import ctypes
import os
import subprocess

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "mattn.h")


def test_struct_layout_matches_c(tmp_path):
    import masked_attention_gb300 as M
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', 'int main(void){']
    want = {}
    for cls in (M.attn_view, M.attn_rope_params):
        s = cls.__name__
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        want[s] = ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            lines.append(f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));')
            want[f"{s}.{f}"] = getattr(cls, f).offset
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert {k: int(v) for k, v in (line.split() for line in out.splitlines())} == want
