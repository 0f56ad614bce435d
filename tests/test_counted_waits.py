"""Kernels that copy to LDS ahead of time wait for "all but the last N loads" before a barrier, so N may not exceed the
loads that every wave issues behind the awaited ones, whichever way its branches go.  A load that the compiler puts under a
branch does not count: a wave that skips it would pass the wait with a copy still in flight.  Checked on the instructions
of the built library: for each barrier, the fewest loads on any path to it from a barrier before, against the wait ahead of it."""

import heapq
import os
import re
import shutil
import struct
import subprocess

import pytest

import post_nvfp4_weight_amd as nvq

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
LOADS = ("buffer_load", "global_load", "flat_load", "scratch_load", "buffer_store", "global_store", "flat_store", "scratch_store",
         "buffer_atomic", "global_atomic", "flat_atomic")   # what the counter counts


def _code_objects(path):
    """The device code objects that a library holds, one per source."""
    data, at = open(path, "rb").read(), 0
    while (at := data.find(b"__CLANG_OFFLOAD_BUNDLE__", at)) >= 0:
        entry = at + 32
        for _ in range(struct.unpack_from("<Q", data, at + 24)[0]):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            if size and b"gfx950" in data[entry + 24:entry + 24 + length]:
                yield data[at + offset:at + offset + size]
            entry += 24 + length
        at += 24


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{name: [(operation, operands, index that a branch goes to)]} of every kernel of the library."""
    if not shutil.which(OBJDUMP):
        pytest.skip("no llvm-objdump")
    found = {}
    file = tmp_path_factory.mktemp("code") / "object"
    for code in _code_objects(nvq.LIB_PATH):
        file.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(file)], capture_output=True, text=True, check=True).stdout
        for name, body in re.findall(r"^[0-9a-f]+ <(\S+)>:\n(.*?)(?=^\s*$|\Z)", text, flags=re.M | re.S):
            lines = re.findall(r"^\s+(\S+) ?(.*?)\s*// ([0-9A-F]+):.*?(?:<\S+\+0x([0-9a-f]+)>)?$", body, flags=re.M)
            first = int(lines[0][2], 16) if lines else 0
            index = {int(a, 16) - first: i for i, (_, _, a, _) in enumerate(lines)}
            found[name] = [(op, args, index.get(int(to, 16)) if to else None) for op, args, _, to in lines]
    return found


def _next(code, i):
    op, _, to = code[i]
    if op == "s_endpgm":
        return []
    if op == "s_branch":
        return [to]
    return [i + 1, to] if op.startswith("s_cbranch") else [i + 1]


def _waits(code):
    """(fewest loads from a barrier to the next on any path, how many loads the wait before that one lets stay out)."""
    out = []
    for b, (op, _, _) in enumerate(code):
        if op != "s_barrier":
            continue
        best, queue, ends = {b: 0}, [(0, b)], {}
        while queue:
            n, i = heapq.heappop(queue)
            if n > best[i]:
                continue
            for j in _next(code, i):
                if code[j][0] == "s_barrier":
                    ends[j] = min(ends.get(j, n), n)
                    continue
                c = n + code[j][0].startswith(LOADS)
                if c < best.get(j, c + 1):
                    best[j] = c
                    heapq.heappush(queue, (c, j))
        for j, n in ends.items():
            while not (code[j][0] == "s_waitcnt" and "vmcnt" in code[j][1]):
                j -= 1
            out.append((n, int(re.search(r"vmcnt\((\d+)\)", code[j][1]).group(1))))
    return out


def _some(kernels, part):
    found = {n: c for n, c in kernels.items() if part in n}
    assert found, part
    return found.items()


@pytest.mark.parametrize("part", ["mx_dx_kernel", "grouped_dx_kernel"])
def test_gradient_waits_for_the_next_step(kernels, part):
    """The copies of the next step were issued before the last barrier: no more may stay out than were issued since."""
    for name, code in _some(kernels, part):
        waits = _waits(code)
        assert any(0 < out for _, out in waits), name
        for fewest, out in waits:
            assert out <= fewest, (name, fewest, out)


def test_weight_only_product_waits_for_the_next_step(kernels):
    """The step's activations were issued first of the step before, four copies; behind them in that step and in this one all else."""
    for name, code in _some(kernels, "nvfp4_gemm_big_kernel"):
        steps = [(fewest, out) for fewest, out in _waits(code) if out > 0]
        assert steps, name
        least = min(fewest for fewest, _ in steps)
        for _, out in steps:
            assert out <= 2 * least - 4, (name, least, out)


# mx_tile_kernel's ring of R buffers: the copies of R - 2 steps may stay out.
@pytest.mark.parametrize("tile,ring", [("Li2ELi4ELi4ELi2ELi2E", 2), ("Li2ELi2ELi2ELi2ELi2E", 2), ("Li2ELi2ELi2ELi1ELi4E", 4),
                                       ("Li2ELi2ELi1ELi1ELi6E", 6)])
def test_block_scaled_product_waits_for_its_step(kernels, tile, ring):
    for name, code in _some(kernels, "mx_tile_kernelI" + tile):
        for fewest, out in _waits(code):
            assert out <= (ring - 2) * fewest, (name, fewest, out)
