"""What the kernels' sources must hold to, beside what they compute. No GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_17_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_the_roles_of_the_scan_meet_alike_on_every_way():
    """A role whose wait ran out may go another way than its neighbours, so a barrier without a limit that only one of the ways comes to
    could keep them for ever. There is one: the two warps of 32 rows meet once for each block of A that their rows see, whether the
    chunk has an A of its own for each unit or not, and whether a wait ran out or not."""
    text = source("gdn_ssm_scan_kernel.cuh")
    roles = text[text.index("bool ok = true;"):text.index("if (small.abort)")]
    assert not re.search(r"barrier_all|bar\.sync|barrier\.", text) and roles.count("__syncthreads()") == 1
    meet = re.findall(r"[^\n;{}]*named_barrier[^;]*;", text)
    assert [m.split("named_barrier")[1] for m in meet] == ["(7 + quarter, 64);"] * 2, meet
    own, other = roles[roles.index("if (own_a) {"):].split("} else {", 1)
    assert re.search(r"for \(int i = 0; i < 4; \+\+i\).*if \(i <= quarter\) tc::named_barrier", own, flags=re.S)
    assert re.match(r"\s*if \(SLICES == 1\)\s*#pragma unroll 1\s*for \(int i = 0; i <= quarter; \+\+i\) tc::named_barrier", other)
    operands = roles[roles.index("fewer_registers<kSsmOperandRegs>"):roles.index("fewer_registers<kSsmIssueRegs>")]
    assert not re.search(r"\bbreak\b|\breturn\b|\bcontinue\b", operands)  # every chunk, to the end


def test_every_kernel_source_is_built():
    """CUDA sources lie with the library's, and each is one of its units or included by another."""
    root = os.path.dirname(os.path.dirname(CSRC))
    places = ("gated_delta_rule_17_gb300", "include", "oracle", "gdn_synth", "examples", "perf", "profiles", "tests")
    tracked = [os.path.join(d, f) for p in places for d, _, files in os.walk(os.path.join(root, p)) for f in files if f.endswith((".cu", ".cuh"))]
    tracked += [os.path.join(root, f) for f in os.listdir(root) if f.endswith((".cu", ".cuh"))]
    assert {os.path.dirname(f) for f in tracked} == {CSRC}, sorted(tracked)
    included = set(re.findall(r'#include "([^"]+)"', "".join(open(f).read() for f in tracked)))
    for f in tracked:
        assert f.endswith(".cu") or os.path.basename(f) in included, f
    assert not [i for i in included if os.path.isabs(i)]


def test_every_helper_is_called():
    text = "".join(source(f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))
    names = set(re.findall(r"__device__ __(?:force|no)inline__ [\w:]+ (\w+)\(", text))
    assert len(names) > 100
    assert not [n for n in names if len(re.findall(rf"\b{n}\b", text)) < 2]
