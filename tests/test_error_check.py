"""pa_error_check without a GPU: the transfers it makes, against a stand-in for the runtime
calls that it and the tree calls need (preloaded into a process of its own)."""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

import pytest

from paged_kv_cache_287_gb300 import binding

RUNTIME = """
#include <stddef.h>
#include <string.h>
/* The device's error words, by symbol, and how often they are read and written. */
static const void *sym[16];
static unsigned word[16];
int words, reads, writes, launches;
static unsigned *of(const void *s) {
    for (int i = 0; i < words; ++i) if (sym[i] == s) return &word[i];
    sym[words] = s;
    return &word[words++];
}
int cudaStreamSynchronize(void *stream) { (void)stream; return 0; }
int cudaMemcpyFromSymbol(void *dst, const void *s, size_t n, size_t off, int kind) {
    (void)off; (void)kind; ++reads; memcpy(dst, of(s), n); return 0;
}
int cudaMemcpyToSymbol(const void *s, const void *src, size_t n, size_t off, int kind) {
    (void)off; (void)kind; ++writes; memcpy(of(s), src, n); return 0;
}
void set_word(int i, unsigned bits) { word[i] = bits; reads = writes = 0; }
/* Launches that only count. */
int cudaGetDevice(int *dev) { *dev = 0; return 0; }
int cudaDeviceGetAttribute(int *value, int attr, int dev) {
    (void)attr; (void)dev; *value = 152; return 0;
}
int cudaFuncSetAttribute(const void *f, int attr, int value) {
    (void)f; (void)attr; (void)value; return 0;
}
static int encode(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char *name, void **fn, unsigned version,
                                     unsigned long long flags, int *found) {
    (void)name; (void)version; (void)flags; *fn = (void *)encode; *found = 0; return 0;
}
int cudaLaunchKernelExC(const void *config, const void *f, void **args) {
    (void)config; (void)f; (void)args; ++launches; return 0;
}
"""

PROGRAM = """
import ctypes, sys
runtime, lib = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
count = lambda name: ctypes.c_int.in_dll(runtime, name).value
P, i, i64, f, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                    ctypes.c_size_t)
lib.pa_error_check.argtypes = [P]
lib.pa_tree_attention.argtypes = [P, P, P, P, i, i, i, P, i, i, i, i, i, P, i, P, i, f, P, sz, P]
lib.pa_tree_verify.argtypes = [P, P, P, P, i64, P, i64, P, P, P, i, i, i, i, P, P, P]
lib.pa_tree_accept.argtypes = [P, i, i, i, i, P, P, P, i, i, P, i, P, P, P]
F = 1 << 20  # an address that nothing reads
steps = [lambda: 0,
         lambda: lib.pa_tree_accept(F, 9, 16, 8, 128, F, F, F, 3, 8, F, 4, F, None, None),
         lambda: lib.pa_tree_verify(F, F, F, F, 100, F, 100, F, F, F, 3, 9, 8, 100, F, F, None),
         lambda: lib.pa_tree_attention(F, F, F, F, 3, 9, 8, F, 9, 16, 32, 8, 128, F, 4, F, 64,
                                       0.1, F, 1 << 40, None)]
for step, launched in zip(steps, (0, 1, 1, 1)):
    before = count("launches")
    assert step() == 0
    assert count("launches") >= before + launched
    runtime.set_word(15, 0)
    assert lib.pa_error_check(None) == 0
    print(count("words"), count("reads"), count("writes"))
for w in range(count("words")):
    for bits, status in ((1, 4), (2, 5), (4, 7), (3, 5)):
        runtime.set_word(w, bits)
        assert lib.pa_error_check(None) == status, (w, bits)
        assert lib.pa_error_check(None) == 0, (w, bits)
"""


def test_a_check_costs_the_copies_of_what_was_launched(tmp_path):
    """Six small copies (three words read and cleared) where no tree call was made, one more
    read for each kind that was; whatever a word holds is reported once and cleared."""
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no host compiler")
    if not os.path.exists(binding.LIB_PATH):
        from paged_kv_cache_287_gb300 import build
        build.build()
    src, so = tmp_path / "runtime.c", tmp_path / "runtime.so"
    src.write_text(RUNTIME)
    subprocess.run([cc, "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(so), binding.LIB_PATH],
                       env={**os.environ, "LD_PRELOAD": str(so)}, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    words, reads, writes = zip(*(map(int, line.split()) for line in r.stdout.splitlines()))
    assert words == reads == (3, 4, 5, 6)
    assert writes == (3, 3, 3, 3)
