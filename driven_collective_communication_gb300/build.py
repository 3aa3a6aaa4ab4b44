"""Build libdcc.so (the CUDA library behind include/dcc.h) in-tree for sm_103a.

Each translation unit compiles in its own nvcc process (in parallel), then one
nvcc link produces ``driven_collective_communication_gb300/libdcc.so``.  Only
sm_103a code is generated.  No fast-math and no flush-to-zero: the kernels'
fp32 adds must be IEEE round-to-nearest-even with subnormals kept.

``build(checked=True)`` builds ``libdcc_checked.so`` from the same sources with
``-DDCC_CHECK_BOUNDS=1`` (every data access of the kernels checked against the
call's ranges; a violation is recorded and skipped) into ``_build/checked``.

The AUTO algorithm table (``tuning/one_shot_max.json``, written by
``bench.py --write-auto-table`` from a measured sweep) is turned into a C
header (``_build/gen/dcc_tuning.h``) before compiling, so the JSON file is the
table's only source.
"""
import concurrent.futures
import json
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
GEN = os.path.join(BUILD, "gen")
LIB = os.path.join(PKG, "libdcc.so")
LIB_CHECKED = os.path.join(PKG, "libdcc_checked.so")
TUNING = os.path.join(PKG, "tuning", "one_shot_max.json")
DTYPE_ORDER = ("int32", "fp32", "fp16", "bf16")  # dcc_dtype_t values 0..3
MAX_RANKS = 16

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-ftz=false",
              "-prec-div=true", "-prec-sqrt=true", "-fmad=false",
              "-I" + INCLUDE, "-I" + CSRC, "-I" + GEN]

SOURCES = ["dcc_host.cu", "sync_kernels.cu", "coll_allgather.cu",
           "coll_int32.cu", "coll_fp32.cu", "coll_fp16.cu", "coll_bf16.cu", "noalloc.cu",
           "proxy.cu", "coll_fused_bulk.cu", "coll_max.cu", "coll_min.cu", "coll_fused_mma.cu",
           "ops_status.cu", "kv4_cache.cu", "kv4_pages.cu", "kv4_attention.cu",
           "kv4_attention_bf16.cu", "kv4_attention_fp16.cu", "linear.cu"]
# Sources without data accesses that DCC_CHECK_BOUNDS checks (their kernels check
# what they read from tables by themselves): one object serves both builds.
SHARED = [s for s in SOURCES if s.startswith(("kv4_", "linear", "ops_"))]


def nvcc():
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdcc")


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "dcc.h"),
                                                                 os.path.abspath(__file__), TUNING]


def load_auto_table(path=TUNING):
    """{n_ranks: {dtype: bytes}} for n_ranks 1..16 from the tuning JSON (every
    rank count and dtype must be present)."""
    with open(path) as f:
        doc = json.load(f)
    table = {}
    for n in range(1, MAX_RANKS + 1):
        row = doc["one_shot_max_bytes"][str(n)]
        table[n] = {t: int(row[t]) for t in DTYPE_ORDER}
        if any(v < 0 for v in table[n].values()):
            raise ValueError("negative threshold for %d ranks in %s" % (n, path))
    return table


def tuning_header(table):
    """C source of the generated header: kOneShotMaxTable[n][dtype]."""
    lines = ["// Generated by build.py from tuning/one_shot_max.json; do not edit.",
             "// AUTO: largest out-of-place message (bytes per rank) run one-shot,",
             "// [n_ranks][dcc_dtype_t]; row 0 is unused.",
             "#pragma once",
             "static const unsigned long long kOneShotMaxTable[%d][4] = {" % (MAX_RANKS + 1),
             "    {0ull, 0ull, 0ull, 0ull},"]
    for n in range(1, MAX_RANKS + 1):
        lines.append("    {%s},  // %d ranks" % (", ".join("%dull" % table[n][t] for t in DTYPE_ORDER), n))
    lines.append("};")
    return "\n".join(lines) + "\n"


def write_tuning_header():
    os.makedirs(GEN, exist_ok=True)
    text = tuning_header(load_auto_table())
    path = os.path.join(GEN, "dcc_tuning.h")
    if not os.path.exists(path) or open(path).read() != text:
        tmp = path + ".tmp.%d" % os.getpid()
        with open(tmp, "w") as f:
            f.write(text)
        os.replace(tmp, path)
    return path


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force=False, verbose=False, extra_flags=(), checked=False):
    """Compile and link libdcc.so (libdcc_checked.so with checked=True) if any
    source changed; returns its path.  Concurrent callers (e.g. parallel test
    workers) serialise on a lock file."""
    import fcntl
    lib = LIB_CHECKED if checked else LIB
    deps = _deps()
    if not force and not _stale(lib, deps):
        return lib
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, ".lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        if not force and not _stale(lib, deps):  # another process built it meanwhile
            return lib
        flags = list(extra_flags) + (["-DDCC_CHECK_BOUNDS=1"] if checked else [])
        return _build_locked(verbose, flags, lib, os.path.join(BUILD, "checked") if checked else BUILD)


def _build_locked(verbose, extra_flags, lib, objdir):
    cc = nvcc()
    write_tuning_header()
    os.makedirs(objdir, exist_ok=True)

    deps = _deps()

    def compile_one(src):
        shared = src in SHARED and "-DDCC_CHECK_BOUNDS=1" in extra_flags
        obj = os.path.join(BUILD if shared else objdir, os.path.splitext(src)[0] + ".o")
        if shared and not _stale(obj, deps):
            return obj
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib + ".tmp.%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else (),
                checked="--checked" in sys.argv))
