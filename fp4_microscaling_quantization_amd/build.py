"""Build libmxq.so (the HIP kernels and the C ABI) for gfx950, in-tree.

hipcc compiles every source under csrc/ into one shared library next to this
file.  Flags: -O3, no floating-point contraction (each rounding in the
quantizer is the single IEEE operation written), and packed-fp32
instructions disabled.

Beside it stands libmxq_loop.so, for the tests: the same library with launches
over rows of at most LOOP_GRID workgroups, so that few rows make every
workgroup take several in turn, with pieces of the vocabulary of one tile, and
with a function that says which kernels a size takes.
"""
import glob
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmxq.so")
LOOP_LIB = os.path.join(HERE, "libmxq_loop.so")
LOOP_GRID = 5
LOOP_SOURCES = ("norm.hip", "logprobs.hip", "distill.hip", "linear_ce.hip")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.hip")) +
                  glob.glob(os.path.join(HERE, "csrc", "*.cpp")))


def build(verbose: bool = False, jobs: int = 8) -> str:
    """Compile each source to an object (in parallel), then link."""
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    common = ["-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "-ffp-contract=off",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
              "-Wall", "-Wno-unused-function", "-Werror=inline-asm"]
    procs = []

    def compile_to(src, obj, flags):
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        cmd = [HIPCC] + common + flags + lang + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        if len(procs) >= jobs:
            _wait(procs.pop(0))
        return obj

    def link(objs, lib):
        cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950"] + objs + ["-o", lib + ".tmp"]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        os.replace(lib + ".tmp", lib)

    objs, loop_objs = [], []
    for src in sources():
        name = os.path.basename(src)
        objs.append(compile_to(src, os.path.join(objdir, name + ".o"), []))
        loop_objs.append(compile_to(src, os.path.join(objdir, name + ".loop.o"),
                                    [f"-DMXQ_ROW_GRID={LOOP_GRID}", "-DMXQ_PIECE_LOGITS=1", "-DMXQ_TESTS"]) if name in LOOP_SOURCES else objs[-1])
    for p in procs:
        _wait(p)
    link(objs, LIB)
    link(loop_objs, LOOP_LIB)
    return LIB


def _wait(item):
    src, p = item
    out, _ = p.communicate()
    text = out.decode(errors="replace")
    # the host pass does not know the packed-fp32 target feature; harmless
    lines = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
    if p.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n" + "\n".join(lines))
    if lines:
        print("\n".join(lines))


if __name__ == "__main__":
    print(build(verbose=True))
