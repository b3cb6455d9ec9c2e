"""Models of how the warps of the tile kernel meet, with their steps read from its source (no GPU).

Row sums: the two warps that share 32 rows exchange their halves' weight sums through shared memory at the end of every
item.  An item without keys for their row tile has nothing else in it, so the exchange has to be ordered against the next
one by itself.  Every interleaving of the two warps over a few such items is walked; each has to read both halves of the
item it is at."""
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
