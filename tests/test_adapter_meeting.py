"""Host-side model of the meeting in the one-launch adapter kernel (no GPU).

csrc/gsr_adapters.hpp: the workgroup that has written a block's records sets
the block's flag and counts itself in `done`; every tile's workgroup looks at
the flags and then counts itself; the last of them puts flags and count back
to zero, so that the next call on the workspace starts from zeros.  Accesses
of one wave to different addresses may take effect in any order unless the
wave waits for them in between.  The model reads the order of the stores, the
additions and the waits from the source, lets every access take effect at any
time that order allows, in every interleaving of the workgroups, and asks that
flags and count are zero in the end.
"""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HDR = os.path.join(ROOT, "tiled_dense_gemm_scale_amd", "csrc", "gsr_adapters.hpp")

OPS = [("wait", r'asm volatile\("s_waitcnt vmcnt\(0\)"'), ("set", r"__hip_atomic_store\(s\.flags [^,]*, 1u"),
       ("count", r"shrink_done\(")]


def announce_ops(src):
    """The announcing wave's accesses, from the flag's store on, in the order of
    the source."""
    body = src[src.index("void shrink_announce("):]
    body = re.sub(r"//[^\n]*", "", body[: body.index("\n}\n")])
    found = sorted((m.start(), name) for name, pattern in OPS for m in re.finditer(pattern, body))
    names = [name for _, name in found]
    assert names.count("set") == 1 and names.count("count") == 1
    return names[names.index("set"):]


def endings(announce, tiles):
    """Every (flag, done) that the memory may hold once all workgroups have
    ended.  A workgroup is its program, the place in it, and its posted stores;
    an addition takes effect when it is made, because its result is used."""
    programs = [tuple(announce)] + [("look", "count")] * tiles
    arrivals = 1 + tiles
    start = (0, 0, tuple((0, ()) for _ in programs))
    seen, stack, ends = {start}, [start], set()
    while stack:
        flag, done, agents = stack.pop()
        moves = []

        def move(i, agent, flag=flag, done=done):
            moves.append((flag, done, agents[:i] + (agent,) + agents[i + 1:]))

        for i, (at, posted) in enumerate(agents):
            for j, (where, value) in enumerate(posted):  # a posted store takes effect (its address' first)
                if all(w != where for w, _ in posted[:j]):
                    rest = posted[:j] + posted[j + 1:]
                    move(i, (at, rest), **({"flag": value} if where == "flag" else {"done": value}))
            if at == len(programs[i]):
                continue
            op = programs[i][at]
            if op == "wait" and posted:
                continue
            if op == "set":
                move(i, (at + 1, posted + (("flag", 1),)))
            elif op == "count":
                last = (("flag", 0), ("done", 0)) if done == arrivals - 1 else ()
                move(i, (at + 1, posted + last), done=done + 1)
            else:  # a wait that is over, or a look, whose result changes nothing here
                move(i, (at + 1, posted))
        if not moves:
            ends.add((flag, done))
        for m in moves:
            if m not in seen:
                seen.add(m)
                stack.append(m)
    return ends


def test_flags_and_count_end_at_zero():
    with open(HDR) as f:
        ops = announce_ops(f.read())
    for tiles in (1, 2, 3):
        assert endings(ops, tiles) == {(0, 0)}, ops


def test_model_sees_a_missing_wait():
    assert endings(["set", "wait", "count"], 2) == {(0, 0)}
    assert (1, 0) in endings(["set", "count"], 2)
