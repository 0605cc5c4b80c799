"""The measured cases of perf/operators.py, without a GPU."""
import importlib.util
import os
import random

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("operator_cases", os.path.join(ROOT, "perf", "operators.py"))
    cases = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cases)
    return cases


def test_drawn_tables_hold_every_index_of_the_plain_form():
    """Pages of all positions that a case looks up lie inside its table; block
    tables' free pages reach for the new tokens."""
    cases, rng = load(), random.Random(3)
    seen = set()
    for c in cases.listed() + [cases.draw(rng) for _ in range(200)]:
        ctx, new, kv = cases._lens(c)
        table, blocks, order = cases._tables(c, 5)
        p = c["page"]
        last = kv if c["op"] == "attend" or not c["causal"] else [a + b for a, b in zip(ctx, new)]
        if c["op"] == "tables":
            last = [a + b for a, b in zip(ctx, new)]
            held = sum((a + p - 1) // p for a in ctx)
            assert blocks - held >= sum((a + b + p - 1) // p - (a + p - 1) // p for a, b in zip(ctx, new))
        for r, n in enumerate(last):
            pages = table[r, :(n + p - 1) // p]
            assert len(pages) == (n + p - 1) // p and (pages >= 0).all() and (pages < blocks).all()
        assert len(np.unique(table[table >= 0])) == (table >= 0).sum() and len(order) == blocks
        seen.add((c["op"], c["causal"]))
    assert len(seen) == 6
