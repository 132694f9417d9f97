"""Checks of the kernels' source text that need no GPU.

Arrays held in registers are passed by reference with their length in the
parameter's type.  A loop that indexes such a parameter past that length is
undefined, and nothing at run time shows it reliably: the unrolled stores may
be dropped, or land on other locals where the compiler spills them.  So each
loop over the first index of an array parameter is held to run to the length
that the parameter's type gives.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prefix_shared_decode_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def code_of(text: str) -> str:
    """The source without comments and preprocessor lines."""
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    text = re.sub(r"//[^\n]*", " ", text)
    return re.sub(r"^[ \t]*#[^\n]*$", " ", text, flags=re.M)


def closing(text: str, at: int) -> int:
    """The place behind the bracket that closes the one at `at`."""
    pairs = {"(": ")", "{": "}"}
    a, z, depth = text[at], pairs[text[at]], 0
    for i in range(at, len(text)):
        depth += (text[i] == a) - (text[i] == z)
        if depth == 0:
            return i + 1
    raise ValueError("unbalanced")


def statement_end(text: str, at: int) -> int:
    """The end of the statement that begins at `at`."""
    while text[at].isspace():
        at += 1
    if text[at] == "{":
        return closing(text, at)
    m = re.compile(r"(for|if|while)\b(\s+constexpr)?\s*\(").match(text, at)
    if m:
        end = statement_end(text, closing(text, m.end() - 1))
        more = re.compile(r"\s*else\b").match(text, end)
        return statement_end(text, more.end()) if more else end
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] in "({[") - (text[i] in ")}]")
        if text[i] == ";" and depth == 0:
            return i + 1
    raise ValueError("no end")


def loops(body: str):
    """(variable, bound, begin, end) of every counting loop from 0."""
    for m in re.finditer(r"\bfor\s*\(\s*(?:int|uint32_t)\s+(\w+)\s*=\s*0\s*;\s*\1\s*<\s*([^;]+?)\s*;", body):
        head = body.index("(", m.start())
        begin = closing(body, head)
        yield m.group(1), re.sub(r"\s+", "", m.group(2)), begin, statement_end(body, begin)


def within(bound: str, length: str) -> bool:
    if bound.isdigit() and length.isdigit():
        return int(bound) <= int(length)
    return bound == length


def faults(text: str):
    """(function's array, index, loop bound, array length) of each loop that
    runs to something other than the array parameter's length."""
    text = code_of(text)
    found, seen = [], 0
    for m in re.finditer(r"\)\s*(?:->\s*[\w:]+\s*)?\{", text):
        # the parameter list that ends here, and the body that follows
        depth, at = 0, m.start()
        while at >= 0:
            depth += (text[at] == ")") - (text[at] == "(")
            if depth == 0:
                break
            at -= 1
        arrays = dict(re.findall(r"\(&(\w+)\)\[([^\]]+)\]", text[at:m.start()]))
        if not arrays:
            continue
        body = text[m.end() - 1:closing(text, m.end() - 1)]
        same = {a: re.sub(r"\s+", "", b) for a, b in re.findall(r"constexpr int (\w+) = ([^,;]+);", body)}
        nests = [(v, same.get(n, n), a, z) for v, n, a, z in loops(body)]
        for name, length in arrays.items():
            for use in re.finditer(rf"(?<![\w.]){name}\[(\w+)\]", body):
                inner = [x for x in nests if x[0] == use.group(1) and x[2] <= use.start() < x[3]]
                if not inner:
                    continue
                seen += 1
                bound = max(inner, key=lambda x: x[2])[1]
                length_ = re.sub(r"\s+", "", length)
                if not within(bound, same.get(length_, length_)):
                    found.append((name, use.group(1), bound, length))
    return found, seen


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_loops_over_array_parameters_end_at_their_length(path):
    with open(path) as f:
        found, _ = faults(f.read())
    assert not found, f"(array, index, loop runs to, array length): {sorted(set(found))}"


def test_the_check_sees_the_loops():
    """Loops over array parameters are found at all, and a wrong one is told."""
    total = 0
    for path in SOURCES:
        with open(path) as f:
            total += faults(f.read())[1]
    assert total > 40
    text = """template <int N> void f(float (&s)[2 * N][4], const float (&x)[8]) {
    #pragma unroll
        for (int nb = 0; nb < %s; ++nb)
            if (x[0] > 0.f) { s[nb][0] = x[nb]; }
            else
                for (int k = 0; k < 4; ++k) s[nb][k] = 0.f;
    }"""
    assert faults(text % "2 * N")[0] == [("x", "nb", "2*N", "8")]
    assert {f[0] for f in faults(text % "8")[0]} == {"s"}
