"""CPU test of the inline assembly in the layer's kernels: a statement that
writes m0 has it as an output (it is a reserved register, whose clobber tells
the compiler nothing), and one that touches memory is volatile and clobbers
memory, since the compiler does not look inside."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "fp4_block_scaled_amax_amd", "csrc", "layer", "*.h*")))


def statements():
    for path in SOURCES:
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\b(\s+volatile)?\s*\(", text):
            depth, i, quoted = 1, m.end(), False
            while depth:
                if text[i] == '"':
                    quoted = not quoted
                elif not quoted:
                    depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            body = text[m.end():i - 1]
            parts, quoted, start = [], False, 0
            for at, c in enumerate(body):
                quoted ^= c == '"'
                if c == ":" and not quoted:
                    parts.append(body[start:at])
                    start = at + 1
            parts.append(body[start:])
            code = parts[0].replace("\\n", " ").replace("\\t", " ")
            yield os.path.basename(path), m.group(1) is not None, code, parts[1] if len(parts) > 1 else "", parts[3] if len(parts) > 3 else ""


def test_clobbers():
    loads = 0
    for name, volatile, code, outputs, clobbers in statements():
        assert ("m0" in code) == ('"=&{m0}"' in outputs) and '"m0"' not in clobbers, (name, code)
        if re.search(r"\b(global|buffer|flat|ds)_(load|store|read|write|atomic)\w*", code):
            assert volatile and '"memory"' in clobbers, (name, code)
            if "_lds_" in code:  # the address in LDS, and the state between its write and the load
                assert re.match(r'\s*"s_mov_b32 m0, %\d\s+s_nop 0\s+global_load_lds_', code), (name, code)
                loads += 1
        if "s_waitcnt" in code:
            assert volatile and '"memory"' in clobbers, (name, code)
    assert loads >= 3  # the loads to LDS were found
