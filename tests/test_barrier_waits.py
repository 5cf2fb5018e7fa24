"""A workgroup's barrier does not wait for the LDS accesses that a wave has under way: where the barrier is written out (the
builtin, not __syncthreads), the wave waits for them first, or another wave may overwrite what it still reads, or read what
it has not yet written.  Checked in the sources, and in the code that the compiler makes of them."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_moe_layer_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FILES = ["gemm_dma.hip", "linear_tiles.hip"]


def statements(path):
    """The source's statements without comments, the functions that wrap the barrier and compiler-only fences left out."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    text = re.sub(r"void block_sync\(\) \{.*?\n\}", "", text, flags=re.S)
    text = re.sub(r'asm volatile\("" ::: "memory"\);|__builtin_amdgcn_sched_barrier\(0\);', "", text)
    return [" ".join(s.split()) for s in re.split(r"[;{}]", text) if s.strip()]


def waits_for_lds(statement):
    m = re.search(r"__builtin_amdgcn_s_waitcnt\((.*)\)$", statement)
    if not m:
        return False
    return "lgkm0" in m.group(1) or (re.fullmatch(r"0x[0-9A-Fa-f]+|\d+", m.group(1)) is not None
                                     and int(m.group(1), 0) & 0xF00 == 0)


@pytest.mark.parametrize("name", FILES)
def test_sources_wait_before_a_barrier(name):
    st = statements(os.path.join(CSRC, name))
    at = [i for i, s in enumerate(st) if s in ("block_sync()", "__builtin_amdgcn_s_barrier()")]
    assert at
    for i in at:
        assert waits_for_lds(st[i - 1]), f"{name}: before {st[i]}: {st[i - 1]}"


def kernels(listing):
    """(name, basic blocks, successors) of each kernel of a listing."""
    for name, body in re.findall(r"^(_Z\w+):[^\n]*\n(.*?)^\.Lfunc_end", listing, re.S | re.M):
        names, blocks = [""], [[]]
        for line in body.splitlines():
            line = line.split(";")[0].strip()
            m = re.match(r"(\.LBB\S+):", line)
            if m:
                names.append(m.group(1))
                blocks.append([])
            elif line and not line.startswith("."):
                blocks[-1].append(line)
        index = {n: i for i, n in enumerate(names)}
        succ = []
        for i, b in enumerate(blocks):
            to = [index[m.group(1)] for m in (re.match(r"s_c?branch\S*\s+(\.LBB\S+)", l) for l in b) if m]
            if not any(l.startswith(("s_branch", "s_endpgm")) for l in b) and i + 1 < len(blocks):
                to.append(i + 1)
            succ.append(to)
        yield name, blocks, succ


def under_way(block, pending, found=None):
    """Whether an access of the LDS's memory may be under way behind the block; the barriers it meets go to found."""
    for line in block:
        if re.match(r"ds_(read|write|add|load|store)", line):
            pending = line
        elif line.startswith("s_waitcnt") and "lgkmcnt(0)" in line:
            pending = None
        elif line.startswith("s_barrier") and found is not None:
            found.append(pending)
    return pending


@pytest.mark.timeout(300)
@pytest.mark.parametrize("name", FILES)
def test_built_code_waits_before_a_barrier(name, tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("ROCm compiler not present")
    from sparse_moe_layer_amd import build
    out = str(tmp_path / "listing")
    r = subprocess.run([HIPCC] + [f for f in build.FLAGS if f != "-fPIC"] + ["-x", "hip", "--cuda-device-only", "-S",
                       os.path.join(CSRC, name), "-o", out], capture_output=True, text=True, timeout=280)
    assert r.returncode == 0, r.stderr
    barriers = 0
    for kernel, blocks, succ in kernels(open(out).read()):
        entry = [None] * len(blocks)
        todo = list(range(len(blocks)))
        while todo:  # one bit a block, set at most once
            i = todo.pop()
            after = under_way(blocks[i], entry[i])
            for s in succ[i]:
                if after and not entry[s]:
                    entry[s] = after
                    todo.append(s)
        for i, b in enumerate(blocks):
            found = []
            under_way(b, entry[i], found)
            barriers += len(found)
            assert not any(found), f"{kernel}: {found}"
    assert barriers
