"""How the roles of the many-rows attention kernel keep in step, on the CPU.

A wait that is missing there shows only as a hang, and then only if the timing
is against it.  So the order is checked where it can be: over every
interleaving of a small model of the barriers, and in the source.
"""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a4_mxfp4_post_b200", "csrc", "mx_chunk.cuh")


def softmax_role():
    """Lines of the softmax role's loop over segments, without comments, each with its depth of braces within the loop."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[text.rindex("while (walk.left > 0 && ok) {"):].split("\n")
    depth, lines = 1, []
    for line in body[1:]:
        if line.strip().startswith("}"):
            depth -= line.strip()[:line.strip().find("{")].count("}") if "{" in line else line.count("}")
            if "{" in line:
                lines.append((depth, line.strip()))
                depth += 1
                continue
            if depth <= 0:
                break
            continue
        lines.append((depth, line.strip()))
        depth += line.count("{") - line.count("}")
    return lines


def runs_ahead(tiles, always):
    """Whether some order of events lets a tile announce segment s + 1 before the issuer has taken up segment s.

    tiles: per segment, whether the second tile has rows.  always: both tiles wait for
    `segdone` in every segment (else only one that has no rows does).  The tensor cores'
    commits complete in order, at any time after they are issued.
    """
    S = len(tiles)
    # state: steps of tile 0, tile 1 and the issuer; completed phases of q0, q1, odone0, odone1, segdone; commits in flight
    start = (0, 0, 0, 0, 0, 0, 0, 0, ())
    seen, todo = {start}, [start]
    program = []
    for t in (0, 1):
        steps = []
        for s in range(S):
            has = t == 0 or tiles[s]
            steps.append(("arrive", s))
            if has:
                steps.append(("odone", sum(1 for x in range(s) if t == 0 or tiles[x])))
            if always or not has:
                steps.append(("segdone", s))
        program.append(steps)

    def passes(done, phase):                 # a wait on the parity of `phase`, `done` phases complete
        return done % 2 != phase % 2

    while todo:
        st = todo.pop()
        pc, q, od, sd, flight = list(st[:2]), list(st[3:5]), list(st[5:7]), st[7], st[8]
        issued = st[2]
        nexts = []
        for t in (0, 1):
            if pc[t] == len(program[t]):
                continue
            what, n = program[t][pc[t]]
            if what == "arrive":
                if q[t] > issued:
                    return True              # two arrivals for one wait of the issuer: phases are confused
                ok, q2 = True, [x + (i == t) for i, x in enumerate(q)]
            else:
                ok, q2 = passes(od[t] if what == "odone" else sd, n), q
            if ok:
                pc2 = [x + (i == t) for i, x in enumerate(pc)]
                nexts.append((*pc2, issued, *q2, *od, sd, flight))
        if issued < S and passes(q[0], issued) and passes(q[1], issued):
            commits = ("0", "1", "s") if tiles[issued] else ("0", "s")
            nexts.append((*pc, issued + 1, *q, *od, sd, flight + commits))
        if flight:
            first, rest = flight[0], flight[1:]
            nexts.append((*pc, issued, *q, od[0] + (first == "0"), od[1] + (first == "1"), sd + (first == "s"), rest))
        for n in nexts:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return False


@pytest.mark.parametrize("tiles", [(True, False), (True, False, True, False), (False, True, False, False), (True,) * 4, (False,) * 4])
def test_no_tile_runs_ahead_of_the_segments(tiles):
    assert not runs_ahead(tiles, always=True)


def test_a_wait_left_out_lets_a_tile_run_ahead():
    """What the model is for: a tile that had rows, waits for its own results only and has none in the next segment."""
    assert runs_ahead((True, False, False), always=False)


def test_every_segment_waits_until_it_is_done():
    lines = softmax_role()
    waits = [depth for depth, line in lines if "wait(&segdone" in line]
    assert waits == [1], "one wait for segdone, in no branch of the loop over segments"
    assert lines[-1][1] == "advance();"


def test_each_warpgroup_has_one_setmaxnreg():
    """setmaxnreg is for a whole warpgroup: one for warps 0 to 7, all of one role, and one before the roles for the others, which have two."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = [(m.start(), m.group(1)) for m in re.finditer(r"setmaxnreg\.(inc|dec)\.sync\.aligned", text)]
    assert [kind for _, kind in found] == ["dec", "inc"]
    roles, softmax = text.index("if (warp >= kSoftmaxWarps && warp < kMmaWarp) {"), text.rindex("} else {", 0, found[1][0])
    assert re.search(r"if \(warp >= kSoftmaxWarps\) asm volatile\(\"setmaxnreg\.dec", text[:roles])
    assert text[softmax:found[1][0]].split() == ["}", "else", "{", "asm", 'volatile("']
