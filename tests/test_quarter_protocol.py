"""The 8-bit LM head's epilogue: the two warps of a quarter of a tile's rows,
checked on the CPU.

The two meet at a barrier of their own twice a tile, and either's wait for the
tile's accumulator may run out.  A warp that leaves its loop alone would leave
the other standing at the next barrier for good, so they leave by an answer both
read behind the first barrier, whether or not the quarter has rows.  The model
below runs random schedules of two such warps; the source has to be of the form
that it finds sound.
"""
import os
import random
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "invariant_token_log_gb300", "csrc")


def simulate(seed, shared, tiles=12):
    """None if both warps leave their loops after the same tile, else a description.  `shared`: tiles without rows
    go through the exchange too."""
    rnd = random.Random(seed)
    empty = [rnd.random() < 0.5 for _ in range(tiles)]
    fails = (rnd.randrange(2), rnd.randrange(tiles))  # the warp and the tile whose wait runs out
    abort = False
    flags = [True, True]
    left = [None, None]

    def wait(w, tile):
        nonlocal abort
        if (w, tile) == fails:
            abort = True
            return False
        return not (abort and rnd.random() < 0.5)  # a wait that ends in time does not look at the flag

    def warp(w):
        for tile in range(tiles):
            ok = wait(w, tile)
            yield "step"
            if empty[tile] and not shared:
                if not ok:
                    left[w] = tile
                    return
                continue
            flags[w] = ok
            yield "meet"
            if not (flags[0] and flags[1]):
                left[w] = tile
                return
            yield "step"
            yield "meet"
        left[w] = tiles

    warps = [warp(0), warp(1)]
    state = ["step", "step"]
    for _ in range(10000):
        if state[0] == state[1] == "meet":
            state = ["step", "step"]
        live = [w for w in (0, 1) if state[w] == "step"]
        if not live:
            break
        w = rnd.choice(live)
        state[w] = next(warps[w], "done")
    if "meet" in state:
        return "a warp waits for the other for good"
    return None if left[0] == left[1] else f"the warps left after tiles {left}"


def test_the_shared_answer_ends_every_schedule():
    assert [s for s in range(4000) if simulate(s, shared=True) is not None] == []


def test_the_model_finds_a_warp_left_alone():
    assert any(simulate(s, shared=False) == "a warp waits for the other for good" for s in range(4000))


def body_of(text, name):
    """The braces' contents of function `name`, comments blanked."""
    text = re.sub(r"//.*", "", text)
    start = re.search(r"\b" + name + r"\([^;{]*\{", text).end()
    depth, at = 1, start
    while depth:
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        at += 1
    return text[start:at - 1]


def test_the_source_has_the_shared_form():
    text = open(os.path.join(CSRC, "linear.cu")).read()
    body = body_of(text, "epilogue8")
    answers = re.findall(r"if \(!quarter_ok\([^;]*\)\) return false;", body)
    # on the way to every return stands the exchange, and to every `true` the barrier behind it
    assert len(answers) == 2 and body.count("return false") == 2 and body.count("return true") == 2
    paths = body.split("return true;")
    for path in paths[:2]:
        assert path.index("quarter_ok(") < path.index("return false") < path.index("quarter_sync(")
