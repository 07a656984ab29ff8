"""The few-token product's counted waits, read off the assembly of its source.

Each K-step's barrier waits until at most N vector memory operations of the wave are
outstanding; they complete in the order of issue. Every path from a kernel's entry to its
epilogue is walked with a queue of the operations it issues, in which only the waits
written in the kernel retire anything (the compiler's own waits may come and go): behind
step u's barrier the direct loads of step u + 1 have to have landed."""
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "hashed_gram_conditional_amd")


def _build_module():
    spec = importlib.util.spec_from_file_location("_engram_build_asm", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    b = _build_module()
    if not os.path.exists(b.hipcc()):
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("asm") / "gemm_mx4.s")
    flags = [f for f in b.HIP_FLAGS if f != "-shared"]
    subprocess.run([b.hipcc(), *flags, "--cuda-device-only", "-S", "-I", os.path.join(ROOT, "include"),
                    "-o", out, os.path.join(PKG, "csrc", "gemm_mx4.hip")], check=True, capture_output=True)
    with open(out) as f:
        return f.read()


# (format of e: 4 for E2M1, 0 for E4M3; 32-column and 32-token tiles of a wave)
INSTANCES = [(ef, ni, mt) for ef in (4, 0) for ni, mt in ((1, 1), (2, 1), (2, 2), (4, 2))]


def blocks_of(text, name):
    """A kernel's basic blocks: {label: (events, successors)}. An event is "direct" (a load
    into LDS), "other" (any other vector memory operation) or the count of a written
    wait that stands before a barrier."""
    m = re.search(r"^_ZN\S*%s\S*:" % name, text, re.M)
    lines = text[m.end():text.index(".Lfunc_end", m.end())].split("\n")
    blocks, label, events, nexts, inside = {}, "entry", [], [], False
    for raw in lines[1:]:
        mark = raw.strip()
        if mark.startswith(";;#ASM"):
            inside = mark == ";;#ASMSTART"
            continue
        line = raw.split(";")[0].strip()
        m = re.match(r"(\.LBB\w+):", line)
        if m:
            blocks[label] = (events, nexts + [m.group(1)])
            label, events, nexts = m.group(1), [], []
            continue
        op = line.split()[0] if line else ""
        if re.match(r"(buffer|global|scratch|flat)_(load|store|atomic)", op):
            events.append("direct" if re.search(r"\blds$", line) else "other")
        elif inside and op == "s_waitcnt":
            events.append(int(re.search(r"vmcnt\((\d+)\)", line).group(1)))
        elif op.startswith("s_cbranch"):
            target = line.split()[1]
            blocks[label] = (events, nexts + [target, label + "'"])
            label, events, nexts = label + "'", [], []
        elif op == "s_branch":
            blocks[label] = (events, nexts + [line.split()[1]])
            label, events, nexts = label + "'", [], []
        elif op == "s_endpgm":
            blocks[label] = (events, [])
            label, events, nexts = label + "'", [], []
    return blocks


def landed_before(step, ef, ni, mt):
    """How many of a wave's direct loads are those of K-steps up to `step` and what is
    issued before them: weight pairs 0 .. and e batches 0, 1, 2, 3 in turn, then a batch
    behind each step's barrier and a weight pair behind each odd one's."""
    e_loads = 64 * mt * (64 if ef == 4 else 128) // 4096
    w_loads = 64 * ni * 128 // 4096
    ring = 4 if ef == 4 and ni < 4 else 3
    order = ["w"] * (ring - 2) + ["e", "e", "w", "e", "e", "w"]
    for u in range(step):
        order += ["e"] + (["w"] if u % 2 else [])
    pairs, batches, loads, need = 0, 0, 0, (step // 2 + 1, step + 1)
    for kind in order:
        if pairs >= need[0] and batches >= need[1]:
            break
        pairs, batches = pairs + (kind == "w"), batches + (kind == "e")
        loads += w_loads if kind == "w" else e_loads
    assert pairs >= need[0] and batches >= need[1]
    return loads


def faults(blocks, ef, ni, mt, loops=3):
    """(K-steps seen, what is wrong) along every path, a loop taken up to `loops` times."""
    wrong, seen = [], set()
    todo = [("entry", [], 0, 0, {})]
    while todo:
        label, queue, landed, step, visits = todo.pop()
        visits = dict(visits)
        visits[label] = visits.get(label, 0) + 1
        if visits[label] > loops:
            continue
        queue = list(queue)
        events, nexts = blocks[label]
        done = False
        for k, ev in enumerate(events):
            if isinstance(ev, str):
                queue.append(ev)
                continue
            retired = queue[:len(queue) - ev] if ev < len(queue) else []
            landed += retired.count("direct")
            queue = queue[len(retired):]
            if ev == 0:                  # the wait before the epilogue
                seen.add(step)
                done = True
                break
            need = landed_before(step, ef, ni, mt)
            if landed < need:
                wrong.append((step, ev, need - landed))
            step += 1
        if not done:
            todo += [(n, queue, landed, step, visits) for n in nexts]
    return seen, sorted(set(wrong))


@pytest.mark.parametrize("ef,ni,mt", INSTANCES)
def test_every_step_waits_for_the_next_one(assembly, ef, ni, mt):
    blocks = blocks_of(assembly, "mx4_skinny_kernelILi%dELi%dELi%dE" % (ef, ni, mt))
    seen, wrong = faults(blocks, ef, ni, mt)
    unroll = 8 if ef == 4 and ni < 4 else 12
    # one barrier before step 0 and one in each step: up to two turns of the loop and a tail
    assert set(range(2, 3 * unroll)) <= seen
    assert not wrong, "(barrier, count, loads that may be in flight): %s" % wrong[:12]
