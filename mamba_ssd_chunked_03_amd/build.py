"""Build libssd.so in-tree with hipcc for gfx950.

Every kernel source and the C ABI are compiled to objects under ``_build/`` in
parallel, then linked into ``mamba_ssd_chunked_03_amd/libssd.so``.  All HIP
code is compiled with packed-fp32 instruction selection disabled.
"""
import concurrent.futures
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(HERE, "libssd.so")
BUILD_DIR = os.path.join(ROOT, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

TABLE_JSON = os.path.join(HERE, "tuning", "table.json")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC, "-I", BUILD_DIR,
]


def _write_inc(name, struct, array, comment, rows):
    lines = ["// generated by build.py from tuning/table.json: " + comment]
    if rows:
        lines.append("static const %s %s[] = {" % (struct, array))
        lines += ["    {%s}," % ", ".join(str(v) for v in r) for r in rows]
        lines.append("};")
    else:
        lines.append("static const %s %s[] = {{%s}};" % (struct, array, ", ".join("0" for _ in comment.split(","))))
    lines.append("static const int %sCount = %d;" % (array, len(rows)))
    text = "\n".join(lines) + "\n"
    path = os.path.join(BUILD_DIR, name)
    if not os.path.exists(path) or open(path).read() != text:
        with open(path, "w") as f:
            f.write(text)
    return path


def write_table_include():
    """The tuned per-shape table (tuning/table.json, written by tuning/sweep.py on
    the GPU) as the C++ arrays the launchers look up: the state passing's rows in
    tuned_scan.inc, the chunk-state kernels' in tuned_cs.inc; empty tables when the
    file or its section is absent.  Returns the two paths."""
    import json
    t = {}
    if os.path.exists(TABLE_JSON):
        with open(TABLE_JSON) as f:
            t = json.load(f)
    scan = [(int(e["chunks_per_seq"]), int(e["lanes"]), int(e["variant"])) for e in t.get("state_passing", [])]
    cs = [(int(e["headdim"]), int(e["dstate"]), int(e["heads_per_group"]), int(e["chunk"]), int(e["variant"]))
          for e in t.get("chunk_state", [])]
    return (_write_inc("tuned_scan.inc", "ScanEntry", "kTunedScan", "(chunks per sequence, lanes, variant)", scan),
            _write_inc("tuned_cs.inc", "CsEntry", "kTunedCs",
                       "(headdim, dstate, heads per group, chunk, variant)", cs))


# The delta rule's kernels keep MFMA accumulators that vector code works on between the
# products: in plain VGPRs those need no accumulator moves (176 of 1900 instructions of
# the forward chain).
DELTA_FLAGS = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]


def _compile(src):
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC, "-x", "hip", "-c", src, "-o", obj] + FLAGS
    if os.path.basename(src).startswith("k_delta"):
        cmd += DELTA_FLAGS
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, r.stderr))
    return obj


def build(verbose=False):
    """Compile every source and link libssd.so; returns its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    write_table_include()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + sorted(glob.glob(os.path.join(CSRC, "api*.cpp")))
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % r.stderr)
    os.replace(tmp, OUT)
    if verbose:
        print("built", OUT)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
