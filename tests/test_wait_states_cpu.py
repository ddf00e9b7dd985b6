"""Wait states between a matrix-core product and the first use of its result, in the
built library, along every path (no GPU needed).

The hardware does not hold back an instruction that reads a product's result too soon:
the compiler puts wait states between.  Where a branch skips a block, it has been seen
to count them along the path through the block only, so that the shorter path, over the
taken branch, read a stale result.  Sources cannot rule that out, so the instructions
themselves are checked: from each product, over all branches, to the first
instruction that names one of its result registers.

A product of P passes (4 cycles each) needs P + 4 wait states before its result is read
or written over, an fp32 one P + 2.  A product may have it at once as the whole of its
accumulator input, and one that takes no fewer passes may write over it.  An instruction
is one wait state, ``s_nop n`` is n + 1."""
import os
import re
import shutil
import subprocess

import pytest

from gemm_decode_q1_amd import q1 as B

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

pytestmark = pytest.mark.skipif(not (os.path.exists(B.LIB_PATH) and os.path.exists(OBJDUMP)),
                                reason="libq1.so or llvm-objdump is not there")

# passes by shape and type; f8f6f4: with an fp8 operand
PASSES = {"16x16x32_bf16": 4, "16x16x32_f16": 4, "32x32x16_bf16": 8, "32x32x16_f16": 8, "16x16x128_f8f6f4": 8,
          "32x32x64_f8f6f4": 16, "16x16x4_f32": 8}


def wait_states(op):
    shape = re.match(r"v_mfma_(?:scale_)?(?:f32|ld)_(\w+)", op).group(1)
    return PASSES[shape] + (2 if shape.endswith("x4_f32") else 4)


def registers(text):
    found = set()
    for kind, lo, hi in re.findall(r"\b([av])\[(\d+):(\d+)\]", text):
        found |= {(kind, i) for i in range(int(lo), int(hi) + 1)}
    return found | {(kind, int(n)) for kind, n in re.findall(r"\b([av])(\d+)\b", text)}


def operands(args):
    return [x.strip() for x in re.split(r",\s*(?![^\[]*\])", args)]


def parse(listing):
    """{function: [(address, mnemonic, arguments)]} of llvm-objdump -d."""
    functions, body = {}, None
    for line in listing.splitlines():
        head = re.match(r"^[0-9a-f]+ <(.+)>:$", line)
        if head:
            body = functions.setdefault(head.group(1), [])
        elif body is not None and "// " in line:
            text, _, note = line.partition("// ")
            op, _, args = text.strip().partition(" ")
            body.append((int(note.split(":")[0], 16), op, args.strip()))
    return functions


def too_soon(body):
    """(product, reader, wait states between, needed) for every read that comes too early."""
    at = {a: i for i, (a, _, _) in enumerate(body)}
    bad = []
    for i, (_, op, args) in enumerate(body):
        if not op.startswith("v_mfma"):
            continue
        need, out = wait_states(op), registers(operands(args)[0])
        todo, best = [(i + 1, 0)], {}
        while todo:
            j, waited = todo.pop()
            while j < len(body) and waited < need and best.get(j, need) > waited:
                best[j] = waited
                a, o, x = body[j]
                if o == "s_endpgm":
                    break
                if o.startswith("s_cbranch") or o == "s_branch":
                    jump = int(x.split()[0])
                    target = at[a + 4 + 4 * (jump - 65536 if jump >= 32768 else jump)]
                    if o == "s_branch":
                        j, waited = target, waited + 1
                        continue
                    todo.append((target, waited + 1))
                elif o.startswith("v_mfma"):
                    p = operands(x)
                    inputs = registers(" ".join(p[1:3]))
                    if registers(p[3]) != out:
                        inputs |= registers(p[3])
                    if inputs & out or (registers(p[0]) & out and wait_states(o) < need):
                        bad.append((body[i], body[j], waited, need))
                    if registers(p[0]) & out:
                        break
                elif out & registers(x):
                    bad.append((body[i], body[j], waited, need))
                    break
                j, waited = j + 1, waited + (int(x, 0) + 1 if o == "s_nop" else 1)
    return bad


def test_the_check_itself():
    """A short wait is found straight ahead, over a taken branch and around a loop; a long one, and sums into
    the same registers, are not."""
    product = "v_mfma_f32_16x16x32_bf16", "v[0:3], v[4:7], v[8:11], v[0:3]"
    read = "v_add_f32_e32", "v20, v1, v2"

    def code(*ops):
        return [(4 * i, *o) for i, o in enumerate(ops)] + [(4 * len(ops), "s_endpgm", "")]

    nop = lambda n: ("s_nop", str(n))  # noqa: E731
    assert too_soon(code(product, nop(6), read))[0][2:] == (7, 8)
    assert not too_soon(code(product, nop(7), read))
    assert not too_soon(code(product, product, nop(7), read))
    # jump over a block of ten wait states
    assert too_soon(code(product, ("s_cbranch_scc1", "1"), nop(9), read))[0][2:] == (1, 8)
    assert not too_soon(code(product, nop(6), ("s_cbranch_scc1", "1"), nop(9), read))
    # back to the top of a loop
    assert too_soon(code(read, product, ("s_cbranch_scc1", "65533")))[0][2:] == (1, 8)
    # another product takes the result as a factor, or part of it as a sum
    assert too_soon(code(product, ("v_mfma_f32_16x16x32_bf16", "v[12:15], v[0:3], v[8:11], v[12:15]")))
    assert too_soon(code(product, ("v_mfma_f32_16x16x32_bf16", "v[12:15], v[4:7], v[8:11], v[2:5]")))


def test_library(tmp_path):
    lib = shutil.copy(B.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, stdout=subprocess.DEVNULL, cwd=tmp_path)
    products, bad = 0, []
    for f in sorted(tmp_path.glob("*gfx950")):
        text = subprocess.run([OBJDUMP, "-d", str(f)], check=True, stdout=subprocess.PIPE, text=True).stdout
        if "v_mfma" not in text:
            continue
        for name, body in parse(text).items():
            products += sum(op.startswith("v_mfma") for _, op, _ in body)
            bad += [(name, *b) for b in too_soon(body)]
    assert products > 1000
    assert not bad, "\n".join(f"{name}: {p[1]} {p[2]} -> {r[1]} {r[2]} after {w} of {n}" for name, p, r, w, n in bad[:20])
