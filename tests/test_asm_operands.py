"""Inline asm of several instructions writes outputs before it has read its last input, so these
must not share registers: every such output is an early clobber.  (The compiler gives an input the
register of an output that holds the same value before the statement otherwise.)"""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "stream_compaction_amd", "csrc")


def statements(text):
    """Each asm statement's template, output and input operands."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
        depth, quoted, parts, i = 1, False, [""], m.end()
        while depth:
            c = text[i]
            quoted ^= c == '"' and text[i - 1] != "\\"
            if not quoted:
                depth += (c in "([") - (c in ")]")
                if c == ":" and depth == 1:
                    parts.append("")
                    i += 1
                    continue
            parts[-1] += c if depth else ""
            i += 1
        yield [p.strip() for p in (parts + ["", ""])[:3]]


def test_outputs_of_several_instructions_are_early_clobbers():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        with open(path) as f:
            for template, outputs, inputs in statements(f.read()):
                several = "\\n" in template or re.search(r"[A-Z_]{3,}\(", template)
                if not (several and outputs and inputs):
                    continue
                seen += 1
                for constraint in re.findall(r'"([=+][^"]*)"', outputs):
                    assert "&" in constraint, f"{os.path.basename(path)}: {outputs}"
    assert seen >= 2                      # the paired load and the sums over lanes
