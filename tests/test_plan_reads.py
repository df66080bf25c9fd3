"""What the plan of the prefix attention writes is not read through the read-only path (no GPU): the
kernels behind it may be resident while it writes, and that path is for memory that nobody writes as
long as a kernel lasts."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_231_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, head):
    """The function whose declaration has `head` in it, braces and all."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(head)


def fields(call):
    """Fields of that call's parameters that point into what the plan writes."""
    text = source("prefix.cu")
    kernel = body(text, "prefix_plan_kernel(")
    written = set(re.findall(r"x\.(\w+)\[[^\]]*\] = ", kernel)) | set(
        re.findall(r"\*x\.(\w+) = ", kernel))
    assert {"start", "group_cu", "group_keys", "table_row", "active", "choice", "units"} <= written
    given = re.findall(call + r"->(\w+) = (?:base \? )?x->(\w+)", body(text, "prefix_layout("))
    return {name for name, what in given if what in written}


def test_fields():
    assert fields("shared") == {"cu", "klen", "table_row", "active", "units"}
    assert fields("own") == {"start", "choice"}


def reads(text, names):
    """Loads through the read-only path, in statements that name one of the fields."""
    return [x.strip() for x in re.split(r"[;{}]", text)
            if re.search(r"__ldg|\.nc\.", x) and re.search(r"\bp\.(%s)\b" % "|".join(names), x)]


def test_shared_keys():
    # the tiles, and what they read their sequences with
    assert reads(source("cross_tiles.cu"), fields("shared")) == []
    seq = body(source("cross_dev.cuh"), "read_seq(")
    assert reads(seq, fields("shared")) == []
    # one load there serves all forms: of the shared keys' it is no read-only one
    assert re.search(r"F == kShared \? __ldcg\((\w+)\) : __ldg\(\1\)", seq)
    assert reads(body(source("cross.cu"), "cross_join_kernel("), fields("shared")) == []


def test_own_keys():
    for name in ("cross.cu", "cross_tiles.cu", "cross_dev.cuh"):
        assert reads(source(name), fields("own")) == []
