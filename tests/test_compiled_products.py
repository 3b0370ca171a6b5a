"""The matrix-core kernel of the linear head's cross entropy, as it was compiled.

Its products are inline assembly, whose latency the compiler does not know: what it puts
between them on its own (a spill, a copy of an accumulator) could read a result before it
is there.  The source ends every chain of products with a wait; these tests hold that
nothing else touches the accumulators before it, in the library built here."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_scan_diagonal_amd", "liblrs.so")
LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
OBJDUMP, READELF = (os.path.join(LLVM, n) for n in ("llvm-objdump", "llvm-readelf"))

pytestmark = pytest.mark.skipif(not all(os.path.exists(p) for p in (LIB, OBJDUMP, READELF)),
                                reason="liblrs.so or the LLVM tools are missing")

# Wait states after which any matrix instruction's result may be read (the 16x16x32
# products, of 8 passes, need fewer; the longest, of 16, need 19).
WAIT = 20


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """The device code object that holds the kernel."""
    tmp = tmp_path_factory.mktemp("code")
    lib = tmp / "lib.so"
    lib.write_bytes(open(LIB, "rb").read())
    subprocess.run([OBJDUMP, "--offloading", str(lib)], cwd=tmp, check=True, capture_output=True)
    found = [p for p in tmp.iterdir() if "gfx950" in p.name and b"k_gemm" in p.read_bytes()]
    assert len(found) == 1
    return str(found[0])


def test_no_spills(code):
    notes = subprocess.run([READELF, "--notes", code], check=True, capture_output=True, text=True).stdout
    kernels = [k for k in re.split(r"\n  - (?=\.agpr_count)", notes) if re.search(r"\.name: +\S*k_gemm", k)]
    assert len(kernels) >= 15
    for k in kernels:
        for field in ("private_segment_fixed_size", "vgpr_spill_count", "sgpr_spill_count"):
            assert re.search(rf"\.{field}: +0\n", k), (field, re.search(r"\.name: +(\S+)", k).group(1))


def functions(code):
    """{name: [(offset, mnemonic, operands, branch target or None)]} of the kernel's forms."""
    text = subprocess.run([OBJDUMP, "-d", code], check=True, capture_output=True, text=True).stdout
    out = {}
    for part in re.split(r"\n(?=[0-9a-f]{16} <)", text):
        head = re.match(r"([0-9a-f]{16}) <(\S*k_gemm\S*)>:", part)
        if not head:
            continue
        start, lines = int(head.group(1), 16), []
        for line in part.splitlines()[1:]:
            m = re.match(r"\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):", line)
            if m:
                to = re.search(r"<\S+?\+0x([0-9a-f]+)>", line) if m.group(1).startswith("s_cbranch") \
                    or m.group(1) == "s_branch" else None
                lines.append((int(m.group(3), 16) - start, m.group(1), m.group(2),
                              int(to.group(1), 16) if to else None))
        out[head.group(2)] = lines
    return out


def accumulators(operands):
    """The accumulator registers that an operand list names."""
    regs = set()
    for lo, hi, one in re.findall(r"\ba(?:\[(\d+):(\d+)\]|(\d+)\b)", operands):
        regs |= set(range(int(lo), int(hi) + 1)) if lo else {int(one)}
    return regs


def early(lines):
    """The first instruction, on any path, that is not a product and touches an
    accumulator within WAIT wait states of the product that wrote it; or None."""
    at = {off: i for i, (off, *_rest) in enumerate(lines)}
    # at an instruction: registers whose product has not ended -> wait states since
    pending, todo = {0: {}}, [0]
    while todo:
        i = todo.pop()
        while i is not None:
            state = dict(pending[i])
            _, op, args, to = lines[i]
            if op.startswith("v_mfma"):
                steps, written = 1, accumulators(args.split(",")[0])
            else:
                if accumulators(args) & set(state):
                    return lines[i]
                steps, written = int(args, 0) + 1 if op == "s_nop" else 1, ()
            state = {r: n + steps for r, n in state.items() if n + steps < WAIT}
            state.update(dict.fromkeys(written, 0))
            here, i_next = i, None
            for n in ([] if op in ("s_endpgm", "s_branch") else [here + 1]) + ([] if to is None else [at[to]]):
                old = pending.get(n)
                new = state if old is None else {r: min(state.get(r, WAIT), old.get(r, WAIT))
                                                 for r in set(state) | set(old)}
                if new != old:
                    pending[n] = new
                    if n == here + 1:
                        i_next = n
                    else:
                        todo.append(n)
            i = i_next
    return None


def test_accumulators_are_left_alone_until_their_wait(code):
    found = functions(code)
    assert len(found) >= 15
    for name, lines in found.items():
        assert sum(m.startswith("v_mfma") for _, m, _, _ in lines) >= 32, name
        assert any(m == "v_accvgpr_read_b32" for _, m, _, _ in lines), name
        assert early(lines) is None, (name, early(lines))


def test_the_check_finds_an_early_read():
    """In lists of instructions: in a row, over a branch, round a loop."""
    mfma = (0, "v_mfma_f32_16x16x32_bf16", "a[0:3], v[0:3], v[4:7], a[0:3]", None)
    read = (8, "v_accvgpr_read_b32", "v9, a2", None)
    end = (99, "s_endpgm", "", None)
    nop = (4, "s_nop", "15", None)
    assert early([mfma, read, end]) == read
    assert early([mfma, nop, read, end]) == read
    assert early([mfma, nop, (6, "s_nop", "15", None), read, end]) is None
    assert early([mfma, (4, "s_cbranch_scc1", "3", 8), (5, "s_nop", "15", None), (6, "s_nop", "15", None),
                  read, end]) == read
    first = (0, "v_accvgpr_read_b32", "v9, a2", None)
    assert early([first, (4, *mfma[1:]), (6, "s_cbranch_scc1", "-3", 0), end]) == first
    assert early([mfma, (8, "v_accvgpr_read_b32", "v9, a4", None), end]) is None


def test_m0_serves_the_loads_to_lds_alone(code):
    """The loads to LDS take their address from m0, which the compiler does not know to
    be written: it must not use m0 for anything of its own."""
    for name, lines in functions(code).items():
        for i, (_, op, args, _) in enumerate(lines):
            if re.search(r"\bm0\b", args):
                assert op == "s_mov_b32" and args.startswith("m0,"), (name, lines[i])
                assert lines[i + 1][1] == "s_nop" and lines[i + 2][1] == "global_load_lds_dwordx4", name
            else:
                assert not op.startswith(("s_sendmsg", "v_movrel", "ds_gws", "buffer_load_lds")), name
