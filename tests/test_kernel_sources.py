"""Rules of the kernels' sources that no run shows: instructions that PTX defines only for a whole warp."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_expert_b200", "csrc")


def functions(text):
    """(name, body) of the file's functions, by their braces."""
    for head in re.finditer(r"__device__[^;{}()]*?(\w+)\([^;{}]*\)\s*\{", text):
        depth, at = 1, head.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield head.group(1), text[head.end():at]


def test_whole_warp_instructions_join_the_warp_first():
    """barrier.cluster, setmaxnreg and the taking and freeing of tensor memory are .aligned: all threads of the warp
    execute them together. Callers come from loops and branches that threads leave at different times, so each such
    function joins the warp itself."""
    with open(os.path.join(CSRC, "tc.cuh")) as f:
        text = f.read()
    # PTX texts hold braces of their own
    text = re.sub(r'"(?:[^"\\]|\\.)*"', lambda m: m.group(0).replace("{", "(").replace("}", ")"), text)
    seen = 0
    for name, body in functions(text):
        at = re.search(r"barrier\.cluster\S*aligned|setmaxnreg|tcgen05\.(alloc|dealloc)", body)
        if at:
            seen += 1
            assert "__syncwarp();" in body[:at.start()], name
    assert seen >= 7
