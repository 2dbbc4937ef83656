"""Build libscan_amd.so (the HIP kernels and the C ABI) in-tree for gfx950.

    python -m stream_compaction_amd.build

Each source compiles to an object under ``_build/`` in parallel, then hipcc
links the shared library next to this file.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(HERE, "libscan_amd.so")
SOURCES = ["scan_rows.hip", "scan_device.hip", "select.hip", "reduce.hip", "reduce_by_key.hip",
           "radix_sort.hip", "causal_conv.hip", "selective_scan.hip", "selective_scan_grad.hip",
           "embedding.hip", "gated_scan.hip", "gated_scan_grad.hip", "beam.hip", "api.cpp",
           "api_sequence.cpp", "api_gated.cpp", "api_beam.cpp"]
# measurement aid for the benchmark (16-byte copy kernel), kept out of the scan library
COPY_LIB_PATH = os.path.join(HERE, "libscan_copy.so")
COPY_SOURCES = ["copy_ceiling.hip"]
# test-only build of the scan library whose look-back never waits: any
# predecessor descriptor not yet published is recomputed from the input at
# once, so the tests exercise that recovery path on every call; whose gated
# scan asks for a state once and then takes it as lost, and does not write some;
# and whose launches of beam_reorder hold three workgroups, so that rows go out
# in several
FALLBACK_LIB_PATH = os.path.join(HERE, "libscan_amd_lbtest.so")
FALLBACK_DEFINES = ["-DSCA_LOOKBACK_TIMEOUT_TICKS=0ull", "-DSCA_TILE_POLLS=0u", "-DSCA_TILE_MUTE",
                    "-DSCA_REORDER_BLOCKS=3"]
# the sources that these are of; the others' objects are the library's own
FALLBACK_SOURCES = ("scan_device.hip", "select.hip", "reduce_by_key.hip", "gated_scan.hip", "gated_scan_grad.hip",
                    "beam.hip")
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # no packed-FP32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"),
]
# Pairing float operations into vectors gains nothing without packed instructions, and
# keeps broadcasts across lanes from folding into the products that use them.
FILE_FLAGS = {"selective_scan.hip": ["-fno-slp-vectorize"],
              "selective_scan_grad.hip": ["-fno-slp-vectorize"],
              "gated_scan.hip": ["-fno-slp-vectorize"],
              "gated_scan_grad.hip": ["-fno-slp-vectorize"]}


def compile_cmd(src, obj, defines=()):
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    return [HIPCC, *CFLAGS, *FILE_FLAGS.get(src, ()), *defines, *lang, "-c", os.path.join(CSRC, src), "-o", obj]


def build(verbose=False):
    os.makedirs(OBJ_DIR, exist_ok=True)
    procs = []
    libs = {LIB_PATH: [], COPY_LIB_PATH: [], FALLBACK_LIB_PATH: []}
    jobs = [(LIB_PATH, s, ()) for s in SOURCES] + [(COPY_LIB_PATH, s, ()) for s in COPY_SOURCES] + \
        [(FALLBACK_LIB_PATH, s, FALLBACK_DEFINES) for s in FALLBACK_SOURCES]
    for lib, src, defines in jobs:
        tag = "_lbtest" if defines else ""
        obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + tag + ".o")
        libs[lib].append(obj)
        cmd = compile_cmd(src, obj, defines)
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    libs[FALLBACK_LIB_PATH] += [os.path.join(OBJ_DIR, os.path.splitext(s)[0] + ".o") for s in SOURCES
                                if s not in FALLBACK_SOURCES]
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        # hipcc's host pass does not know the device-only feature flag: drop that note
        lines = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln]
        if lines and (verbose or p.returncode != 0):
            print("\n".join(lines), file=sys.stderr)
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    for path, lib_objs in libs.items():
        tmp = path + ".tmp"
        subprocess.check_call([HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", *lib_objs,
                               "-o", tmp])
        os.replace(tmp, path)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
