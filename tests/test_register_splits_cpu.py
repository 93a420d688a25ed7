"""Kernels that move registers between their warpgroups: the shares fit what the kernel is launched with.

An increase beyond that would wait for ever, so the launch is refused on the host instead; that the built kernels have the
registers is read off what the assembler prints for them.
"""
import importlib.util
import os
import re
import subprocess

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_05_gb300")
CSRC = os.path.join(PKG, "csrc")


def sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "regs_claim<" in open(os.path.join(CSRC, f)).read()]


def test_every_such_launch_is_checked():
    assert len(sources()) >= 2
    for path in sources():
        text = open(path).read()
        assert re.search(r"numRegs[\s\S]{0,600}kRegsNeeded\)\s*return cudaErrorInvalidConfiguration", text), path


def test_prompt_attention_has_the_registers(tmp_path):
    spec = importlib.util.spec_from_file_location("_build_of_registers", os.path.join(PKG, "_build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    source = os.path.join(CSRC, "prompt_attn.cu")
    flags = [f for f in build.FLAGS if f != "-lineinfo"]
    out = subprocess.run([build.nvcc(), *build.ARCH, *flags, "-Xptxas", "-v", "-c", source, "-o", str(tmp_path / "x.o")],
                         capture_output=True, text=True, check=True).stderr
    found = dict(re.findall(r"prompt_attn_kernelILb([01])E[^\n]*\n(?:(?!Compiling)[\s\S])*?Used (\d+) registers", out))
    text = open(source).read()
    threads = re.search(r"kThreads = FP8 \? (\d+) : (\d+);", text).groups()
    softmax = re.search(r"kSoftmaxRegs = FP8 \? (\d+) : (\d+),", text).groups()
    others = int(re.search(r"kOtherRegs = (\d+);", text).group(1))
    assert set(found) == {"0", "1"}
    for i, fp8 in enumerate("10"):
        n = int(threads[i])
        assert int(found[fp8]) * n >= 256 * int(softmax[i]) + (n - 256) * others
