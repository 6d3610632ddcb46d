"""CPU tests of the experts' kernels whose loads go straight to LDS: the compiler
knows neither when such a load ends nor what it overwrites, so a wave waits for
its LDS reads before it asks for anything in their place, and the statements say
what they write."""

import glob
import os
import re

import test_layer_asm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp4_block_scaled_amax_amd", "csrc", "experts")


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def body(text, start):
    """The block in braces that begins behind `start`."""
    i = text.index("{", start)
    depth, j = 1, i + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
    return text[i + 1:j - 1]


def governs(text, wait, load):
    """Whether the statement at `wait` runs whenever the one at `load` does: no block that holds it ends between them,
    and no condition stands before it without braces."""
    depth = 0
    for c in text[wait:load]:
        depth += {"{": 1, "}": -1}.get(c, 0)
        if depth < 0:
            return False
    return not re.search(r"(\)|\belse)\s*$", text[:wait])


def test_reads_end_before_their_place_is_loaded_again():
    text = code("gemm_weight_only.hip")
    kernels = list(re.finditer(r"__global__[^;{]*\b(\w+_kernel)\(", text))
    seen = []
    for k in kernels:
        kernel = body(text, k.end())
        if "load_tokens" not in kernel:
            continue
        # the loop over K: the last `for` before the waves' sums are joined that loads tokens
        loops = [body(kernel, m.end()) for m in re.finditer(r"\n    for \(uint32_t \w+ = ", kernel)]
        loops = [b for b in loops if "load_tokens(" in b]
        assert len(loops) == 1, k.group(1)
        loop, at = loops[0], loops[0].index("load_tokens(")
        waits = [m.start() for m in re.finditer(r"lds_reads_done\(\);", loop[:at])]
        assert any(governs(loop, w, at) for w in waits), k.group(1)
        seen.append(k.group(1))
    assert sorted(seen) == ["chunks_kernel", "tokens_kernel"]


def test_loads_to_lds_say_what_they_write(monkeypatch):
    """Every statement that writes m0 has it as an output, what touches memory or waits is volatile and clobbers memory,
    and a load to LDS stands five wait states behind the vector instruction that may have written its scalar base."""
    monkeypatch.setattr(test_layer_asm, "SOURCES", sorted(glob.glob(os.path.join(CSRC, "*.h*"))))
    loads = 0
    for name, volatile, text, outputs, clobbers in test_layer_asm.statements():
        assert ("m0" in text) == ('"=&{m0}"' in outputs) and '"m0"' not in clobbers, (name, text)
        if "s_waitcnt" in text or re.search(r"\b(global|buffer|flat|ds)_(load|store|read|write|atomic)\w*", text):
            assert volatile and '"memory"' in clobbers, (name, text)
        if "_lds_" in text:
            assert re.match(r'\s*"s_mov_b32 m0, %\d\s+s_nop 4\s+global_load_lds_', text), (name, text)
            loads += 1
    assert loads == 3
