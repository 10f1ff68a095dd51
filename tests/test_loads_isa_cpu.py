"""Loads into LDS are written out by hand, so the compiler does not count the wait states that a buffer's descriptor needs:
on the library's own gfx950 code, that no vector instruction writes a scalar register that one reads within five states,
along every way that leads there."""
import re

import pytest

from test_ffn_isa_cpu import disassemble

STATES = 5


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    found = disassemble(str(tmp_path_factory.mktemp("isa")))
    found = {k: v for k, v in found.items() if any(is_load(t) for _, t in v)}
    for name in ("ffn_gemm_kernel", "muon_gemm_kernel", "tokens_up_kernel", "tokens_down_kernel"):
        assert any(name in k for k in found), name
    return found


def is_load(text):
    return text.startswith("buffer_load") and text.endswith(" lds")


def scalars(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand) or re.fullmatch(r"s(\d+)()", operand)
    return set(range(int(m[1]), int(m[2] or m[1]) + 1)) if m else set()


def operands(text):
    return [w for part in text.split(None, 1)[1:] for w in re.split(r"[,\s]+", part)]


def written_by_vector(text):
    if not text.startswith("v_"):
        return set()
    ops = operands(text)
    return scalars(ops[0]) | (scalars(ops[1]) if "_co_" in text or "div_scale" in text else set())


def states(text):
    return int(text.split()[1], 0) + 1 if text.startswith("s_nop") else 1


def sources(code):
    """Of each instruction, those that may come before it."""
    at = {a: i for i, (a, _) in enumerate(code)}
    before = [[i - 1] if i else [] for i in range(len(code))]
    for i, (a, text) in enumerate(code):
        m = re.match(r"s_c?branch\S* (\d+)", text)
        if m:
            offset = int(m[1]) - (0x10000 if int(m[1]) >= 0x8000 else 0)
            before[at[a + 4 + 4 * offset]].append(i)
            if text.startswith("s_branch") and i + 1 < len(code):
                before[i + 1].remove(i)
    return before


def too_early(code):
    before, bad = sources(code), []
    for i, (_, text) in enumerate(code):
        if not is_load(text):
            continue
        wanted = set().union(*map(scalars, operands(text)))
        ways = [(j, 0) for j in before[i]]
        while ways:
            j, passed = ways.pop()
            if passed >= STATES:
                continue
            if written_by_vector(code[j][1]) & wanted:
                bad.append((code[j][1], text, passed))
                break
            ways += [(k, passed + states(code[j][1])) for k in before[j]]
    return bad


def test_descriptors_are_not_read_too_early(kernels):
    for name, code in kernels.items():
        bad = too_early(code)
        assert not bad, (name, bad[:3])


def test_the_scan_finds_what_it_looks_for():
    load = "buffer_load_dwordx4 v6, s[8:11], 0 offen lds"
    code = lambda *lines: list(zip(range(0, 4 * len(lines), 4), lines))
    write = "v_readfirstlane_b32 s9, v1"
    assert too_early(code(write, "s_mov_b32 m0, s14", "s_nop 0", load))
    assert not too_early(code(write, "s_nop 4", load))
    assert too_early(code(write, "s_nop 3", load))
    assert not too_early(code("v_readfirstlane_b32 s12, v1", load))
    # around a loop: the branch at 8 goes back to 0
    assert too_early(code(load, write, "s_cbranch_scc1 65533"))
