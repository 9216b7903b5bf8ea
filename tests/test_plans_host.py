"""The plan functions compiled for the host alone, with every undefined
operation (a division by zero, a signed overflow) made a trap, and called over
sizes from no rows at all to past the limits."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "memory_bounded_expert_amd", "csrc")
INCLUDE = os.path.join(ROOT, "include")
HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")

# the runtime's side of a host object: nothing here reaches a launch
STUBS = r"""
#include <stdlib.h>
static void* none;
void** __hipRegisterFatBinary(const void* b) { (void)b; return &none; }
void __hipUnregisterFatBinary(void** m) { (void)m; }
void __hipRegisterFunction(void) {}
void __hipRegisterVar(void) {}
"""
SWEEP = r"""
#include <stdio.h>
#include <stdint.h>
static const int64_t rows[] = {INT64_MIN, -1, 0, 1, 2, 3, 63, 64, 65, 255, 256, 257, 777, 4096, 4097, 8192, 65536, 1 << 20,
    (1 << 23) - 1, (1 << 26) - 1, 1 << 26, (1 << 30) - 1, 1 << 30, INT32_MAX, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX};
#define ROWS(n) for (unsigned i_##n = 0; i_##n < sizeof rows / sizeof *rows; ++i_##n) for (int64_t n = rows[i_##n], once_##n = 1; once_##n; once_##n = 0)
static const int32_t sizes[] = {INT32_MIN, -1, 0, 1, 2, 3, 64, 128, 256, 384, 512, 640, 7168, 20224, 65536, 65537, 1 << 22, 1 << 29, INT32_MAX};
#define SIZES(n) for (unsigned i_##n = 0; i_##n < sizeof sizes / sizeof *sizes; ++i_##n) for (int32_t n = sizes[i_##n], once_##n = 1; once_##n; once_##n = 0)
int main(void) {
    long ok = 0;
    CALLS
    printf("%ld\n", ok);
    return 0;
}
"""
CALLS = {
    "route": ("route_score", "route.h", """
    ROWS(N) SIZES(E) SIZES(k) for (int g = -1; g <= 8; g += 3) for (int s = 0; s < 2; ++s) {
        route_plan_t p; ok += route_plan(N, E, k, s, g, g > 2 ? 2 : 1, 2, s, 1.f, &p) == MOE_OK; }"""),
    "lnorm": ("lnorm", "lnorm.h", """
    ROWS(N) SIZES(H) for (int d = 0; d < 2; ++d) { lnorm_plan_t p; ok += lnorm_plan(N, H, d, 1e-5f, &p) == MOE_OK; }"""),
    "embed": ("embed", "embed.h", """
    ROWS(N) ROWS(V) SIZES(H) for (int d = 0; d < 2; ++d) { embed_plan_t p; ok += embed_plan(N, V, H, d, 1.f, &p) == MOE_OK; }"""),
    "kd": ("distill", "distill.h", """
    ROWS(N) ROWS(V) SIZES(H) SIZES(v) for (int d = 0; d < 2; ++d) {
        kd_plan_t p; ok += kd_plan(N, H, V, v, 7, 2.f, MOE_BF16, d, &p) == MOE_OK; }"""),
}


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")
@pytest.mark.parametrize("name", sorted(CALLS))
def test_plans_do_nothing_undefined(name, tmp_path):
    source, header, calls = CALLS[name]
    obj, main, exe = (str(tmp_path / n) for n in ("plan.o", "main.c", "main"))
    subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}",
                    "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fsanitize-trap=undefined",
                    "-c", os.path.join(CSRC, source + ".hip"), "-o", obj], check=True)
    open(main, "w").write('#include "%s"\n' % header + STUBS + SWEEP.replace("CALLS", calls))
    # what only a launch would call stays unresolved
    subprocess.run(["gcc", "-std=c99", f"-I{INCLUDE}", main, obj, "-o", exe, "-lstdc++", "-lm",
                    "-Wl,--unresolved-symbols=ignore-all"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, f"{name}: a plan's arithmetic trapped ({r.returncode})"
    assert int(r.stdout) > 20
