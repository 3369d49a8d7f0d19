"""The wide tiles of k_head.hip write their matrix-core products as assembly, which the compiler neither spaces nor
keeps in place.  This compiles the file to assembly with the build's own flags and checks what the hardware leaves to
the program: no vector instruction writes a product's operand or a sum within the two instructions before it, EXEC
stays as it is for four, nothing but the next product into the same registers reads a result for 19 wait states, and
nothing is spilled, which would move sums between products."""
import os
import re
import subprocess

import pytest

import sparse_ternary_bit_amd.build as B


def _regs(op):
    m = re.match(r"^([va])\[(\d+):(\d+)\]$", op)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.match(r"^([va])(\d+)$", op)
    return {(m.group(1), int(m.group(2)))} if m else set()


def faults(lines):
    """(products, what is wrong) of a kernel's instructions, in the order they stand in."""
    ins = [line.split(";")[0].strip() for line in lines]
    ins = [i for i in ins if i and not i.startswith(".") and not i.endswith(":")]
    split = [(i.split()[0], [a.strip() for a in i[len(i.split()[0]):].split(",")]) for i in ins]
    products, bad, written = 0, [], {}
    waited, states = [], 0                       # wait states up to each instruction
    for op, args in split:
        waited.append(states)
        states += int(args[0]) + 1 if op == "s_nop" else 1
    for k, (op, args) in enumerate(split):
        if op.startswith("scratch_"):
            bad.append(ins[k])
        if op.startswith("v_mfma"):
            products += 1
            taken = set().union(*(_regs(a) for a in args[1:]))
            for back in range(k - 1, max(-1, k - 6), -1):
                o, a = split[back]
                near = waited[k] - waited[back]
                if o.startswith("v_") and not o.startswith("v_mfma") and near <= 2 and _regs(a[0]) & taken:
                    bad.append(f"{ins[back]} | {ins[k]}")
                if (o.startswith("v_cmpx") or (o.startswith("s_") and a[0] == "exec")) and near <= 4:
                    bad.append(f"{ins[back]} | {ins[k]}")
            for r in _regs(args[0]):
                written[r] = k
            continue
        for r in set().union(*(_regs(a) for a in args)):
            if r in written:
                if waited[k] - waited[written[r]] < 20:
                    bad.append(f"{ins[written[r]]} ... {ins[k]}")
                del written[r]
    return products, bad


def test_what_the_check_finds():
    product = "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]"
    far = ["s_nop 15", "s_nop 15"]
    assert faults([product, product, *far, "v_accvgpr_read_b32 v9, a2"]) == (2, [])
    assert faults([product, "s_nop 7", "v_accvgpr_read_b32 v9, a2"])[1]
    assert faults(["v_and_b32_e32 v5, v8, v9", product])[1]
    assert faults(["v_accvgpr_write_b32 a1, 0", "s_nop 0", product])[1]
    assert not faults(["v_accvgpr_write_b32 a1, 0", "s_nop 3", product])[1]
    assert faults(["s_mov_b64 exec, s[0:1]", "s_nop 0", product])[1]
    assert faults(["scratch_store_dword off, v1, s0", product])[1]


def test_products_of_the_wide_tiles(tmp_path):
    out = tmp_path / "k_head.s"
    r = subprocess.run([B._hipcc(), *B.COMMON, "--offload-device-only", "-S", os.path.join(B.CSRC, "k_head.hip"), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    text = out.read_text()
    names = re.findall(r"^(_ZN\S*nt_wide_kernel\S*):", text, flags=re.M)
    assert len(names) >= 5       # statistics and gradients of bf16 and of 8-bit rows, and sums
    for name in names:
        at = text.index(name + ":")
        products, bad = faults(text[at:text.index(".size", at)].split("\n"))
        assert products >= 128 and not bad, (name, products, bad[:5])
