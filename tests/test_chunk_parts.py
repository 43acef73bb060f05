"""How a warp lets go of a part of the chunk attention's work that it has read from
shared memory: a model of two lanes that run on by themselves between the warp's
collective steps, and that the kernel lets go in the way that holds."""

import os
import re

import pytest

from self_speculative_verification_gb300 import _build

SOURCE = os.path.join(_build.CSRC, "chunk_attn_tc.cu")


def lanes_part(sync_first, reread):
    """Whether the two lanes of a warp can come to different collective steps.  A
    lane's step: "loop" (reads the fills of the part in its place, or has them in a
    register), then "wait" (collective) for each fill, then "release" -- behind a
    barrier of the lanes, or not -- which lane 0 does, then "next" (collective).
    The producer puts a part of one fill more into a place that was let go of."""
    # (fills in the place, let go of, per lane: (step, fills done, fills read))
    start = (1, False, (("loop", 0, None), ("loop", 0, None)))
    seen, todo = {start}, [start]
    while todo:
        fills, free, lanes = todo.pop()
        out = []
        if free:
            out.append((fills + 1, False, lanes))
        for x in (0, 1):
            step, done, known = lanes[x]
            to = None
            if step == "loop":
                n = fills if reread or known is None else known
                to = ("wait" if done < n else "barrier" if sync_first else "release", done, n)
                out.append((fills, free, lanes[:x] + (to,) + lanes[x + 1:]))
            elif step == "release":
                to = ("next", done, known)
                out.append((fills, free or x == 0, lanes[:x] + (to,) + lanes[x + 1:]))
        at = {lane[0] for lane in lanes}
        if at <= {"wait", "barrier", "next"}:
            if len(at) > 1:
                return True
            if at == {"wait"}:
                out.append((fills, free, tuple(("loop", d + 1, n) for _, d, n in lanes)))
            if at == {"barrier"}:
                out.append((fills, free, tuple(("release", d, n) for _, d, n in lanes)))
        for s in out:
            if s not in seen and s[0] < 4:
                seen.add(s)
                todo.append(s)
    return False


@pytest.mark.parametrize("sync_first,reread,parts", [(False, True, True), (True, True, False), (True, False, False)])
def test_lanes_stay_together(sync_first, reread, parts):
    assert lanes_part(sync_first, reread) == parts


def test_the_kernel_syncs_first():
    text = open(SOURCE).read()
    body = re.search(r"template <bool kWarp>\s+__device__ __forceinline__ void release\(Shared &sh\) \{(.*?)\n    \}", text,
                     re.S).group(1)
    assert body.index("if (kWarp) __syncwarp();") < body.index("mbar_arrive(&sh.part_free[i])")
    uses = re.findall(r"^(.*)reader\.release<(true|false)>\(sh\);", text, re.M)
    assert len(uses) == text.count("reader.release") and text.count("part_free[i])") == 1
    # one thread alone: the MMA threads; whole warps, not a lane of them, otherwise
    assert sum(w == "false" for _, w in uses) == 1 and len(uses) == 6
    assert all(not before.strip() for before, _ in uses)
