"""What a warp publishes by one lane's arrival on a barrier, read from the
source: an arrival by lane 0 releases what lane 0 wrote and what was ordered
before it, so the other lanes' writes to shared memory need a __syncwarp
between them and the arrival.  (Votes, shuffles and reductions order no
memory.)  Such a fault shows in no run that can be relied on."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# what every lane of the warp writes to shared memory that an arrival publishes
WRITES = {"ready": [r"ex\.lq\[", r"ex\.x\[", r"s\.own\[", r"buf\[v1 - v0 \+ lane\]", r"patch_ends<"],
          "known": [r"teacher_mass\("],
          "settled": [],
          "taken": []}


def body(source, name):
    """The text of a kernel, from its name to the closing brace of column 0."""
    start = source.index(name + "(const __grid_constant__")
    return source[start:source.index("\n}\n", start)]


def test_arrivals_follow_a_warp_barrier():
    with open(os.path.join(ROOT, "post_processing_gb300", "csrc", "distill.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    branches = re.split(r"\n    \} else (?:if \(warp == kW\) )?\{\n", body(text, "distill_kernel"))
    assert len(branches) == 3, "the streaming warps, the runs' warp, the losses' warp"
    seen = set()
    for text in branches:
        for m in re.finditer(r"mbar_arrive\(&s\.(\w+)\[", text):
            name = m.group(1)
            for write in WRITES.get(name, []):
                at = [w.end() for w in re.finditer(write, text[:m.start()])]
                if not at:
                    continue
                seen.add((name, write))
                assert "__syncwarp()" in text[at[-1]:m.start()], f"no __syncwarp between {write} and the arrival on {name}"
    assert seen == {(n, w) for n, ws in WRITES.items() for w in ws}
