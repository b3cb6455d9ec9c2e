"""Models of how the warps of the tile kernel meet, with their steps read from its source (no GPU).

Row sums: the two warps that share 32 rows exchange their halves' weight sums through shared memory at the end of every
item.  An item without keys for their row tile has nothing else in it, so the exchange has to be ordered against the next
one by itself.  Every interleaving of the two warps over a few such items is walked; each has to read both halves of the
item it is at.

The end of a wait: when one runs out, warps of the same group look at the abort flag at different times.  If each decides
for itself whether it takes the next item, one can leave while another goes on to a barrier that counts on it, and no limit
holds there.  Every order of publishing, aborting and looking is walked for two warps of a group."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILE_SRC = os.path.join(ROOT, "w4a8_integer_gemm_b200", "csrc", "qoq_attn_tile.cu")


def _source():
    return re.sub(r"//[^\n]*", "", open(TILE_SRC).read())


# ------------------------------------------------------------- row sums ----
def _exchange():
    """The end of an item as a warp sees it: W writes its half, R reads both, B meets the other warp."""
    s = _source()
    s = s[s.index("s_row[t][h][r] = l;"):]
    s = s[:s.index("w.slot < 0")]
    found = re.findall(r"(s_row\[t\]\[h\]\[r\] =)|(s_row\[t\]\[0\]\[r\])|(named_barrier(?:_any)?\(mates)", s)
    return "".join("W" if w else "R" if r else "B" for w, r, b in found)


def _wrong_read(exchange, items=3):
    """Walks every interleaving of two warps doing `exchange` item after item; the first wrong read, or None."""
    steps = [(k, op) for k in range(items) for op in exchange]
    start = (0, 0, (-1, -1))                                  # next step of each warp, the item whose sum each half holds
    seen, todo = {start}, [start]
    while todo:
        a, b, held = todo.pop()
        nxt = []
        at = (a, b)
        ops = [steps[i] if i < len(steps) else None for i in at]
        if ops[0] and ops[1] and ops[0][1] == ops[1][1] == "B":
            nxt.append((a + 1, b + 1, held))
        for w in (0, 1):
            if not ops[w] or ops[w][1] == "B":
                continue
            k, op = ops[w]
            if op == "R" and held != (k, k):
                return f"warp {w} reads the sums of items {held} for item {k}"
            mine = tuple(k if op == "W" and i == w else x for i, x in enumerate(held))
            nxt.append((a + (w == 0), b + (w == 1), mine))
        assert nxt or (a, b) == (len(steps), len(steps)), "a warp waits for good"
        for n in nxt:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return None


def test_the_model_sees_an_unordered_exchange():
    assert _wrong_read("WBR") and _wrong_read("WR") and _wrong_read("WRB")
    assert _wrong_read("WBRB") is None


def test_row_sums_of_items_without_keys():
    exchange = _exchange()
    assert exchange.startswith("WBR")
    assert _wrong_read(exchange) is None


# ------------------------------------------------------ the end of a wait ----
def _roles():
    """How each part of the kernel takes its items: {marker: ["get" or "get_together", ...]}."""
    s = open(TILE_SRC).read()
    marks = ["-- MMA (and the prompts' loader) --", "-- loaders of a cache --", "-- softmax --"]
    at = [s.index(m) for m in marks] + [s.index("Joins a cache's row tiles")]
    return {m: re.findall(r"while \((?:ok && )?(get\w*)\(", s[a:b]) for m, a, b in zip(marks, at, at[1:])}


def _stranded(how):
    """Two warps of a group at the next item; the item is published, and the abort raised, at any time or never.  Each
    warp looks at the barrier first and at the flag next, as often as it likes; with get() by itself, with get_together()
    one looks and tells the other.  Whether a warp can end up waiting for one that left."""
    todo, seen = [("look", "look", False, False)], set()
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        x, y, full, abort = state
        if {x, y} == {"left", "barrier"}:
            return True
        nxt = [(x, y, True, abort), (x, y, full, True)]
        if how == "get_together":
            if x == "look" and (full or abort):               # the one that polls; both do what it found
                nxt.append(("barrier",) * 2 + (full, abort) if full else ("left",) * 2 + (full, abort))
                if abort:                                     # (it may have looked at the barrier just before)
                    nxt.append(("left", "left", full, abort))
        else:
            for w in (0, 1):
                if (x, y)[w] != "look":
                    continue
                for to in ["barrier"] * full + ["left"] * abort:
                    nxt.append((to, y, full, abort) if w == 0 else (x, to, full, abort))
        todo += nxt
    return False


def test_groups_take_an_item_together_or_not_at_all():
    assert _stranded("get") and not _stranded("get_together")
    roles = _roles()
    for marker in ("-- loaders of a cache --", "-- softmax --"):
        assert len(roles[marker]) == 1 and not _stranded(roles[marker][0]), marker
    # the single warps meet nobody in a barrier
    assert roles["-- MMA (and the prompts' loader) --"] == ["get"] * 3


def test_what_was_issued_is_waited_for_however_the_list_ends():
    """The MMA warp's commit and wait, and the prompt loader's, depend on no condition: a list that ends because a wait ran
    out is left by get() like one that ends."""
    s = _source()
    mma = s[s.index("warp == kMmaWarp) {\n            const uint32_t lead"):s.index("if (warp >= kQWarp && warp < kQWarp")]
    tail = mma[mma.index("base += 2 * w.steps;"):]
    assert "mma_commit_lead(lead, done);" in tail and "if (" not in tail
    load = s[s.index("if (BITS == 0 && warp == 16) {"):]
    tail = load[load.index("tma_load_2d("):load.index("else if (BITS && warp >= 16)")]
    assert re.findall(r"if \(([^)]*)\)", tail) == ["lane == 0"] and "mbar_try_wait(full(" in tail
