"""A kernel initialises each of its shared memory barriers once: what a second
initialisation of a live barrier does is undefined.  Read from the sources: the
calls between a kernel's first mbar_init() and its fence_mbar_init()."""
from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(
    __file__))), "dsa_sparse_attention_fwd_gb300", "csrc")
FILES = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu")))
         if "fence_mbar_init();" in open(p).read()]


def argument(text, at):
    """The first argument of the call whose parenthesis opens at `at`."""
    depth, i = 0, at
    while True:
        c = text[i]
        depth += c in "([" and 1 or c in ")]" and -1 or 0
        if depth == 1 and c == ",":
            return re.sub(r"\s+", "", text[at + 1:i])
        i += 1


def initialised_twice(source):
    """Barriers (or the array that they lie in) that a kernel of `source`
    initialises by more than one call."""
    text = re.sub(r"//[^\n]*", "", source)
    bad = []
    for part in text.split("fence_mbar_init();")[:-1]:
        kernel = part[part.rfind("__global__"):]
        # names of barriers -> the array that they are in
        base = dict(re.findall(r"auto (\w+) = \[&\]\(int[^{]*\{ return (\w+)",
                               kernel))
        base.update(re.findall(r"const uint32_t (\w+) = (\w+)(?: \+ \d+)?;",
                               kernel))
        args = [argument(kernel, m.end() - 1)
                for m in re.finditer(r"\bmbar_init\(", kernel)]
        assert args
        bad += [a for a in set(args) if args.count(a) > 1]
        arrays = {re.match(r"\w+", a).group() for a in args}
        bad += [a for a in arrays if base.get(a) in arrays]
    return bad


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_barriers_are_initialised_once(path):
    with open(path) as fh:
        assert initialised_twice(fh.read()) == []


def test_what_counts_as_twice():
    head = """__global__ void k() {
      const uint32_t bars = base + 64;
      const uint32_t q_full = bars;
      auto p_full = [&](int i) { return bars + 24 + 8 * i; };
      auto e = [&](int w, int s) { return bars + (w * 2 + s) * 16; };
      """
    end = "\nfence_mbar_init(); }"
    twice = lambda body: initialised_twice(head + body + end)
    assert twice("mbar_init(bars + 8 * i, f(i, 1));") == []
    assert twice("mbar_init(bars + i * 16, 1); mbar_init(bars + i * 16 + 8, 1);"
                 ) == []
    assert twice("mbar_init(q_full, 1); mbar_init(p_full(i), 4);") == []
    assert twice("mbar_init(bars + 8 * i, 1); mbar_init(q_full, 4);")
    assert twice("mbar_init(bars + 8 * i, 1); mbar_init(p_full(i), 4);")
    assert twice("mbar_init(bars + 8 * i, 1); mbar_init(e(i, 0), 4);")
    assert twice("mbar_init(q_full, 1); mbar_init(q_full, 4);")
