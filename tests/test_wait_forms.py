"""The kernels' waits give up after a time limit, and then every thread has to reach the block's last barrier.  That
holds if a warp leaves its role as one: a lane that leaves alone waits at that barrier for the others, which wait
for it at their next warp-wide instruction.  Checked on the sources (a wait that runs out cannot be made to happen on
a GPU without breaking a kernel)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_235_gb300", "csrc")
KERNELS = ["mass.cu", "prefill.cu", "decode.cu", "evict.cu", "write_kv.cu", "copy.cu"]
# what opens a block that one thread of the warp runs
ONE = re.compile(r"lane == 0|elect_one\(\)|threadIdx\.x == |\(threadIdx\.x & 31\) == 0")


def strip(text):
    """The source without comments and string literals, line numbers kept."""
    def blank(m):
        return "\n" * m.group(0).count("\n") + " "
    return re.sub(r'//[^\n]*|/\*.*?\*/|"(?:\\.|[^"\\\n])*"', blank, text, flags=re.S)


def statements(text):
    """(line, statement text, headers of the blocks around it): a header is what stands before a block's brace, or an
    unbraced if / for / while before its one statement."""
    stack, start, out = [], 0, []
    depth = 0                                                   # of parentheses: the ; of a for's head ends nothing
    for i, ch in enumerate(text):
        if ch == "(":
            depth += 1
        elif ch == ")":
            depth -= 1
        elif ch in ";{}" and (depth == 0 or ch != ";"):
            part = text[start:i]
            line = text.count("\n", 0, start + len(part) - len(part.lstrip())) + 1
            if part.strip():
                out.append((line, " ".join(part.split()), [h for h, _ in stack]))
            if ch == "{":
                stack.append((" ".join(part.split()), depth))
                depth = 0                                       # a lambda's body within a call's arguments
            elif ch == "}" and stack:
                depth = stack.pop()[1]
            start = i + 1
    return out


def alone(statement, headers):
    """Does one thread run the statement?  (Not: the statement only tests for that thread.)"""
    head = statement if re.match(r"(else )?if\b", statement) else ""
    return any(ONE.search(h) for h in headers) or bool(head and ONE.search(head.split(")")[0] + ")"))


def test_the_reader_finds_what_it_looks_for():
    src = strip("""
    void f() { // if (lane == 0) { goto out; }
      if (lane == 0) {
        for (int i = 0; i < n; ++i) { if (!wait(&b[i])) goto out; }
      }
      g([&](int x) { return x; });
      if (!wait(b)) goto out;
    }""")
    got = [(alone(s, h), s) for _, s, h in statements(src) if "goto" in s]
    assert got == [(True, "if (!wait(&b[i])) goto out"), (False, "if (!wait(b)) goto out")]


@pytest.mark.parametrize("name", KERNELS)
def test_no_thread_leaves_its_role_alone(name):
    with open(os.path.join(CSRC, name)) as f:
        src = strip(f.read())
    bad = [(line, s) for line, s, h in statements(src) if re.search(r"\bgoto\b", s) and alone(s, h)]
    assert not bad, bad


# functions, and functions' local ones, that one thread runs
ONE_THREAD = {"prefill.cu": r"\bproducer\(|auto wait = ", "decode.cu": r"\bload_item\(", "mass.cu": None}
WAIT = re.compile(r"\bmbar_wait\w*\s*(<[^;()]*>)?\(")
LEAVES = re.compile(r"\b(return|break|goto|continue)\b")


def lane_by_lane(text):
    """Does every lane take its own answer and none leaves on it?  Either it is dropped (a bare call: *abort is read
    afterwards), or kept in `live` or `there`, on which nothing leaves but by a vote."""
    text = re.sub(r"^(else )?if \(.*\) (?=mbar_wait)", "", text)
    return bool(re.match(r"(mbar_wait|(bool )?live = |const bool there = )", text))


@pytest.mark.parametrize("name", sorted(ONE_THREAD))
def test_a_warp_waits_as_one(name):
    """mbar_wait and its like give each lane an answer of its own: for one thread, or for lanes that stay together
    whatever it is.  Elsewhere a warp's wait is warp_wait."""
    with open(os.path.join(CSRC, name)) as f:
        src = strip(f.read())
    seen, bad = 0, []
    for line, s, h in statements(src):
        if WAIT.search(s):
            seen += 1
            one = ONE_THREAD[name] and any(re.search(ONE_THREAD[name], x) for x in h)
            if not (one or alone(s, h) or lane_by_lane(s)):
                bad.append((line, s))
        # no lane leaves, and no loop ends, on its own answer
        at = re.sub(r"__(all|any)_sync\([^;]*\)", "", s)
        if re.search(r"\b(live|there)\b", at) and (LEAVES.search(at) or re.match(r"(for|while)\b", at)):
            bad.append((line, s))
        if re.search(r"\b(live|there|gave_up)\b", " ".join(h[-1:])) and LEAVES.search(s) and "_sync" not in h[-1]:
            bad.append((line, s))
    assert seen and not bad, bad


@pytest.mark.parametrize("name,lands", [("decode.cu", r"\*cb\.lost\) let_copies_land\(\)"), ("mass.cu", r"\*b\.abort\) let_copies_land\(\)"),
                                        ("prefill.cu", r"if \(\*b\.abort\) { mbar_wait\(b\.q_full")])
def test_loads_in_flight_land_before_a_block_ends(name, lands):
    """A kernel that loads into its shared memory asynchronously waits for that after a wait gave up: every such kernel
    of the file, or (prefill.cu) the producer that issued the loads."""
    with open(os.path.join(CSRC, name)) as f:
        src = " ".join(strip(f.read()).split())
    kernels = len(re.findall(r"__global__ void __launch_bounds__\([^;{]*?(decode_partial|decode_fp4|key_mass)_kernel\(", src)) or 1
    assert len(re.findall(lands, src)) == kernels
