"""Kernels that start beside the kernel before them do not load what that one writes by the read-only path.

A kernel launched as a programmatic dependent is resident while an earlier kernel still writes its inputs. The read-only
path (__ldg) is for data that stays as it is while the kernel runs, and such a load may be moved ahead of the wait. What
goes wrong with it depends on timing and on the compiler, so the sources are checked instead of a run.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "grok_gqa_attention_gb300", "csrc")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"/\*.*?\*/", " ", re.sub(r"//[^\n]*", " ", text), flags=re.S)


def read_only_loads(name):
    """The addresses loaded by __ldg, as written."""
    text, out = code(name), []
    for m in re.finditer(r"\b__ldg\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        out.append(text[m.end():i - 1])
    return out


def test_the_parser_finds_loads():
    assert any("cos_tab" in x for x in read_only_loads("kv8_append.cu"))


def test_eight_bit_decode():
    assert "griddepcontrol.wait" in code("kv8_decode.cu")
    assert read_only_loads("kv8_decode.cu") == []
    assert read_only_loads("kv8.cuh") == []  # (the block table's lookup, shared with it)


def test_prefill_passes():
    loads = read_only_loads("prefill.cu")
    for written in ("k_scale", "o_scale", "item_count", "item_list", "fb_list", "fb_count", "part_"):
        assert not [x for x in loads if written in x], written
