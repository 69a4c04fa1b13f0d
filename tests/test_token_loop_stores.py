"""The debug build's checks of the sampling, rotary and page kernels, looked at closely:
every store to memory of the caller's or to the workspace stands in a statement or
block whose own condition checks its place (``dcheck``), or behind one in the same
block that leaves it, and the check says more than the loop or branch around it.
And of their cluster barriers.  CPU only: the sources are read."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_w8a8_rollout_gb300", "csrc")

# stores through pointers into the caller's memory or the workspace, by file, and how many there are at least (a fork's counts
# stand behind a branch on the page that release builds take too)
STORES = {
    "sample.cuh": (r"\ba\.(tokens|lp|lp_kept|kept)\[[^\]]*\] =(?!=)", 4),
    "sample_exact.cu": (r"\batomic\w+\(a\.", 1),
    "rotary.cu": (r"\*reinterpret_cast<uint[24]\*>\((to|code) \+|\b(to|code)\[c[01]\] =(?!=)", 10),
    "pages.cu": (r"\ba\.(list|refs|lens|slots|to|row|out|lens_out|header|info|used)\[[^\]]*\] =(?!=)|\bc\.rows = a\.block|\brow\[[^\]]*\] =(?!=)|"
                 r"\ba\.copies\[\w+\](\.\w+)? =(?!=)|\*at = |\bdst\[place\(|\batomic\w+\(a\.refs \+ old", 25),
}


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def parts(text):
    """The text's pieces between braces, and semicolons outside parentheses: (piece, the character behind it)."""
    piece, depth, outer = "", 0, []
    for c in text:
        depth += (c in "([") - (c in ")]")
        if c in "{}" or (c == ";" and depth == 0):
            yield " ".join(piece.split()), c
            piece = ""
            if c == "{":
                outer.append(depth)
                depth = 0
            elif c == "}":
                depth = outer.pop() if outer else 0
        else:
            piece += c


def stores(name, pattern):
    """(statement, conditions of the blocks around it, checks that leave a block ahead of it) of each store."""
    blocks, found = [], []  # a block: [its head, checks in it that leave it]
    for piece, end in parts(source(name)):
        for m in re.finditer(pattern, piece):
            found.append((piece, [b[0] for b in blocks], [x for b in blocks for x in b[1]]))
        if end == "{":
            blocks.append([piece, []])
        elif end == "}":
            if blocks:
                blocks.pop()
        elif blocks and re.match(r"if \(!dcheck\(.*\)\) (return|continue)$", piece):
            blocks[-1][1].append(piece)
    return found


def checks(text):
    """The clauses of the dchecks in a text, and the text without them."""
    clauses, rest = [], text
    for m in re.finditer(r"dcheck\(", text):
        i, depth = m.end(), 1
        while depth:
            depth += (text[i] == "(") - (text[i] == ")")
            i += 1
        inside = text[m.end():i - 1].rsplit(",", 1)[0]
        clauses += [c.strip() for c in re.split(r"&&|\|\|", inside)]
        rest = rest.replace(text[m.start():i], "")
    return clauses, rest


@pytest.mark.parametrize("name", STORES)
def test_each_store_has_a_check_of_its_own(name):
    pattern, count = STORES[name]
    found = stores(name, pattern)
    assert len(found) >= count, len(found)
    for statement, heads, ahead in found:
        clauses, around = [], []
        for text in [statement, *heads, *ahead]:
            c, rest = checks(text)
            clauses += c
            around.append(rest)
        assert clauses, (name, statement, heads[-2:])
        around = " ".join(around)
        assert any(c not in around for c in clauses), (name, statement, clauses)


@pytest.mark.parametrize("name", ["pages.cu", "sample.cu", "sample.cuh", "sample_exact.cu", "rotary.cu"])
def test_cluster_barriers_ask_for_no_converged_warp(name):
    # the lanes of a warp come to them from branches and loops of their own: an aligned barrier would be undefined there
    text = source(name)
    assert "ptx::cluster_sync" not in text and not re.search(r"barrier\.cluster\.\w+(\.\w+)?\.aligned", text)
