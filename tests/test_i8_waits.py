"""The 8-bit product's counted waits, read off the assembly of its source.

A barrier waits until at most N vector memory operations of the wave are outstanding; they
complete in the order of issue. In the few-block kernel every step issues the same number
of direct loads behind its barrier, and the step after it has landed when the loads of all
but R - 2 of the R steps in flight have. In the many-token kernel the waits count nothing
outstanding, but for the first step of a tile, which lets the stores of a whole tile
before it pass: there the loads stand before all of them."""
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "hashed_gram_conditional_amd")


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    spec = importlib.util.spec_from_file_location("_engram_build_i8", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    if not os.path.exists(b.hipcc()):
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("asm") / "gemm_i8.s")
    flags = [f for f in b.HIP_FLAGS if f != "-shared"]
    subprocess.run([b.hipcc(), *flags, "--cuda-device-only", "-S", "-I", os.path.join(ROOT, "include"), "-o", out,
                    os.path.join(PKG, "csrc", "gemm_i8.hip")], check=True, capture_output=True)
    with open(out) as f:
        return f.read()


def events(text, name):
    """A kernel's vector memory operations and written waits in the order of the text: "D" a
    direct load, "S" a store, "o" any other, "wN" a wait for N, "|" a label, "b" a branch."""
    m = re.search(r"^_ZN\S*%s\S*:" % name, text, re.M)
    found, inside = [], False
    for raw in text[m.end():text.index(".Lfunc_end", m.end())].split("\n"):
        mark = raw.strip()
        if mark.startswith(";;#ASM"):
            inside = mark == ";;#ASMSTART"
            continue
        line = raw.split(";")[0].strip()
        if re.match(r"(buffer|global|scratch|flat)_(load|store|atomic)", line):
            found.append("D" if re.search(r"\blds$", line) else "S" if "_store" in line else "o")
        elif inside and line.startswith("s_waitcnt"):
            found.append("w" + re.search(r"vmcnt\((\d+)\)", line).group(1))
        elif line.startswith(".LBB"):
            found.append("|")
        elif re.match(r"s_c?branch", line):
            found.append("b")
    return found


@pytest.mark.parametrize("f32", [0, 1])
@pytest.mark.parametrize("once", [0, 1])
@pytest.mark.parametrize("nb,mt,waves,ring", [(1, 1, 4, 6), (2, 1, 4, 6), (2, 2, 8, 4), (2, 4, 8, 3), (4, 2, 8, 3)])
def test_few_block_waits(assembly, f32, once, nb, mt, waves, ring):
    seen = events(assembly, "i8_skinny_kernelILb%dELi%dELi%dELi%dELb%dE" % (f32, nb, mt, waves, once))
    loads = (64 * nb + 64 * mt) // 8 // waves
    flat = " ".join(e for e in seen if e not in "|b")
    step = " w%d" % ((ring - 2) * loads) + " D" * loads
    want = " ".join("D" * (ring * loads)) + " w%d" % ((ring - 1) * loads) + step * ring + " w0"
    # the loop's body stands once, whatever else follows its end
    assert flat.startswith(want), flat[:400]
    assert "D" not in flat[len(want):]
    # nothing but the loop's own edge lies between the first wait and the last
    inner = seen[seen.index("w%d" % ((ring - 1) * loads)):]
    inner = inner[:inner.index("w0")]
    assert inner.count("|") <= 3 and "S" not in inner and "o" not in inner


@pytest.mark.parametrize("f32,stores", [(0, 32), (1, 64)])
def test_many_token_waits(assembly, f32, stores):
    seen = events(assembly, "i8_wide_kernelILb%dE" % f32)
    counted = [e for e in seen if e[0] == "w" and e != "w0"]
    # one wait, in the first step of a tile behind another, that lets the stores pass
    assert counted == ["w%d" % min(stores, 63)]
    # a whole tile issues at least that many stores, all behind the last of the loads
    last = len(seen) - 1 - seen[::-1].index("D")
    assert sum(e == "S" for e in seen[last:]) >= stores
    assert not any(e == "S" for e in seen[:last])
