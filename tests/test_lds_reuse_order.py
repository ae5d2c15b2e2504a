"""Kernels that load into LDS directly and write their results through the same
LDS in the end: read from the code that the library was built to, on the CPU.

A direct load of any wave may land anywhere in a stage until that wave has
waited for it, and the other waves know that it has only behind a barrier that
follows the wait.  So on every path, a wait for all vector memory and then a
workgroup barrier lie between the last direct load and the first write of
results."""

import re
import subprocess

import pytest

from helpers import build_library, lib_is_stale

LLVM = "/opt/rocm/llvm/bin/"


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """{symbol: its instructions as (address, text)}"""
    import quantize_scaled_gemm_amd as q

    if lib_is_stale():
        build_library()
    tmp = tmp_path_factory.mktemp("code")
    fat, obj = tmp / "fat", tmp / "code.o"
    subprocess.run([LLVM + "llvm-objcopy", "--dump-section", f".hip_fatbin={fat}", q.LIB_PATH, "/dev/null"], check=True)
    # one bundle for each source file, each at a multiple of 4096 bytes
    magic, data = b"__CLANG_OFFLOAD_BUNDLE__", fat.read_bytes()
    starts = [m.start() for m in re.finditer(magic, data) if m.start() % 4096 == 0] + [len(data)]
    out = {}
    for lo, hi in zip(starts, starts[1:]):
        if not re.search(b"gemm_wgrad_bf16_dma|gemm_int8_tile", data[lo:hi]):
            continue
        fat.write_bytes(data[lo:hi])
        subprocess.run([LLVM + "clang-offload-bundler", "--unbundle", "--type=o", f"--input={fat}", f"--output={obj}",
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950"], check=True)
        text = subprocess.run([LLVM + "llvm-objdump", "-d", "--no-show-raw-insn", str(obj)], check=True,
                              capture_output=True, text=True).stdout
        name = None
        for line in text.splitlines():
            m = re.match(r"[0-9a-f]+ <(\w+)>:", line)
            if m:
                name = m[1]
                out[name] = []
            elif name and "//" in line:
                ins, _, note = line.partition("//")
                out[name].append((int(note.split(":")[0], 16), ins.strip()))
    return out


def writes_too_early(ins, write):
    """Writes of results that a path reaches without the wait and the barrier
    behind its last direct load."""
    index = {a: i for i, (a, _) in enumerate(ins)}
    # 0: direct loads may be in flight; 1: this wave's have landed; 2: every wave's have
    seen, todo, early = {}, [(0, 2)], set()
    while todo:
        i, state = todo.pop()
        while i < len(ins):
            if seen.get(i, 3) <= state:
                break
            seen[i] = state
            addr, op = ins[i]
            if re.match(r"buffer_load_\w+ .*\blds\b", op):
                state = 0
            elif op.startswith("s_waitcnt") and "vmcnt(0)" in op and state == 0:
                state = 1
            elif op == "s_barrier" and state == 1:
                state = 2
            elif re.match(write, op) and state < 2:
                early.add((hex(addr), op))
            m = re.match(r"s_(c?)branch\w* (\d+)", op)
            if m:
                off = int(m[2])
                todo.append((index[addr + 4 + 4 * (off - 65536 if off >= 32768 else off)], state))
                if not m[1]:
                    break
            elif op.startswith("s_endpgm"):
                break
            assert not op.startswith(("s_setpc", "s_swappc", "s_cbranch_g_fork")), op
            i += 1
    return early


def test_the_walk_finds_a_missing_barrier():
    good = ["buffer_load_dwordx4 v1, s[0:3], 0 offen lds", "s_waitcnt vmcnt(0)", "s_barrier", "ds_write_b32 v0, v1", "s_endpgm"]
    ins = lambda ops: [(4 * i, op) for i, op in enumerate(ops)]
    assert not writes_too_early(ins(good), "ds_write")
    assert writes_too_early(ins(good[:2] + good[3:]), "ds_write")  # no barrier
    assert writes_too_early(ins(good[:1] + good[2:]), "ds_write")  # no wait
    assert writes_too_early(ins([good[0], good[2], good[1], *good[3:]]), "ds_write")  # the wait behind the barrier
    # a path that jumps over the barrier
    assert writes_too_early(ins([*good[:2], "s_cbranch_scc1 1", *good[2:]]), "ds_write")
    # a loop back to the write
    assert writes_too_early(ins([*good[:4], good[0], "s_branch 65533"]), "ds_write")


# the weight gradient's codes are widened into stages of their own by writes of
# 16 bytes; its results are written 4 bytes at a time
@pytest.mark.parametrize("kernel, write, count", [
    ("gemm_wgrad_bf16_dma_kernelILb1E", r"ds_write(2|2st64)?_b32", 1),
    ("gemm_int8_tile_kernel", "ds_write", 8),
])
def test_results_wait_for_every_waves_loads(code, kernel, write, count):
    names = [n for n in code if kernel in n and code[n]]
    assert len(names) == count, names
    for n in names:
        assert any(re.match(write, op) for _, op in code[n])
        assert any(re.match(r"buffer_load_\w+ .*\blds\b", op) for _, op in code[n])
        early = writes_too_early(code[n], write)
        assert not early, (n, len(early), sorted(early)[:3])
