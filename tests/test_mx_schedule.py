"""The order of memory operations in the built kernels of the linear layer (CPU: the
library's own gfx950 code is disassembled, nothing runs).

mx_tile_rows waits by count: a step may begin when at most N operations are still on
their way, and they end in the order in which they were issued.  That is a wait for the
step's transfers to LDS only if N others were issued after them: the transfers of the
first three steps come before the loads of their codes, and nothing is moved to the
other side of a branch.  mx_tile_cols waits for all but a block's loads, which have to
follow each step's transfers."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

import sharded_mixed_precision_shard_amd as zs

TOOL = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
COLS = re.compile(r"mx_tile_colsILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb[01]ELb([01])E")
ROWS = re.compile(r"mx_tile_rowsILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb([01])E")


def kernels(pattern):
    """{match of the name: instructions} of the library's kernels."""
    found = {}
    with tempfile.TemporaryDirectory() as d:
        lib = shutil.copy(zs.LIB_PATH, d)
        subprocess.run([TOOL, "--offloading", lib], check=True, capture_output=True, cwd=d)
        for name in sorted(os.listdir(d)):
            if "gfx950" not in name:
                continue
            path = os.path.join(d, name)
            if b"mx_tile_rows" not in open(path, "rb").read():
                continue
            text = subprocess.run([TOOL, "-d", "--no-show-raw-insn", path], check=True,
                                  capture_output=True, text=True).stdout
            here = None
            for line in text.splitlines():
                label = re.match(r"[0-9a-f]+ <(\S+)>:", line)
                if label:
                    here = pattern.search(label.group(1))
                    if here:
                        found[here] = []
                elif here and line.strip():
                    found[here].append(line.split("//")[0].strip())
    return found


def events(lines):
    """D: a transfer to LDS, c: 16 bytes to registers, o: any other operation that vmcnt counts,
    an int: a wait for all but so many, |: a barrier, b: a branch."""
    out = []
    for line in lines:
        op = line.split()[0]
        if op.startswith("buffer_load") and line.endswith(" lds"):
            out.append("D")
        elif re.match(r"(global|flat|buffer)_load_dwordx4", op):
            out.append("c")
        elif re.match(r"(global|flat|buffer)_(load|store|atomic)", op):
            out.append("o")
        elif op == "s_waitcnt" and "vmcnt" in line:
            out.append(int(re.search(r"vmcnt\((\d+)\)", line).group(1)))
        elif op == "s_barrier":
            out.append("|")
        elif op.startswith(("s_cbranch", "s_branch")):
            out.append("b")
    return out


@pytest.mark.skipif(not os.path.exists(TOOL), reason="no llvm-objdump")
def test_the_first_step_waits_for_its_transfers():
    found = kernels(ROWS)
    assert len(found) == 10
    for match, lines in found.items():
        bi, bj, wi, wj, _, f8 = (int(x) for x in match.groups())
        each = bi * 8 // (wi * wj * 64)                  # transfers of a stage
        codes = bj // wj // 32 * (2 if f8 else 1)        # loads of a step's codes
        seq = events(lines)
        seq = seq[seq.index("D"):]
        seq = seq[:seq.index("|")]                       # up to the first step's barrier
        stage = ["D"] * each
        want = stage * 3 + ["c"] * codes * (2 if f8 else 3)
        assert seq[:len(want)] == want, match.group(0)
        waits = [n for n, e in enumerate(seq) if isinstance(e, int)]
        behind = [e for e in seq[each:waits[-1]] if e in ("D", "c", "o")]
        assert seq[waits[-1]] <= len(behind), match.group(0)


@pytest.mark.skipif(not os.path.exists(TOOL), reason="no llvm-objdump")
def test_a_block_s_loads_follow_each_step_s_transfers():
    found = kernels(COLS)
    assert len(found) == 16
    for match, lines in found.items():
        bi, _, wi, wj, _, f8 = (int(x) for x in match.groups())
        each, loads = bi * 8 // (wi * wj * 64), 3 if f8 else 2
        seq = events(lines)
        at = [n for n, e in enumerate(seq) if e == "D"]
        # before the loop, and the two steps of a turn
        assert len(at) == 3 * each, match.group(0)
        for stage in range(3):
            last = at[(stage + 1) * each - 1]
            end = at[(stage + 1) * each] if stage < 2 else \
                next(n for n in range(last, len(seq)) if seq[n] == 0)
            behind = [e for e in seq[last:end] if e in ("c", "o")]
            assert len(behind) >= loads, match.group(0)
        waits = [seq[n] for n in range(at[0], at[-1]) if isinstance(seq[n], int)
                 and "|" in seq[n + 1:n + 2]]
        assert waits == [loads, loads], match.group(0)
