"""The library allocates no host memory in a call, so no C++ exception for want of it can
leave a C entry point: calls that remember a plan, with every allocation refused."""
import os
import subprocess

import swiglu_gated_mlp_amd as sw

SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <dlfcn.h>
#include <new>

// operator new of the whole process: fails, once told to, where the library itself calls it
static const void *base;
static int refused;
void *operator new(size_t n) {
    Dl_info at;
    if (base && dladdr(__builtin_return_address(0), &at) && at.dli_fbase == base) {
        ++refused;
        throw std::bad_alloc();
    }
    void *p = malloc(n ? n : 1);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void *p) noexcept { free(p); }
void operator delete(void *p, size_t) noexcept { free(p); }

int main(int, char **argv) {
    void *lib = dlopen(argv[1], RTLD_NOW);
    if (!lib) return printf("%s\n", dlerror()), 2;
    auto sizes = (size_t(*)(int64_t, int64_t, int64_t))dlsym(lib, "swiglu_train_workspace_bytes");
    auto forward = (size_t(*)(int64_t, int64_t, int64_t))dlsym(lib, "swiglu_train_forward_workspace_bytes");
    sizes(4, 64, 72);   // whatever the runtime allocates on its first use
    Dl_info at;
    dladdr((void *)sizes, &at);
    size_t without[3][2], with[3][2];
    for (int pass = 0; pass < 2; ++pass) {
        base = pass ? nullptr : at.dli_fbase;
        for (int i = 0; i < 3; ++i) {
            auto &to = pass ? with : without;
            to[i][0] = sizes(64 << (2 * i), 896, 4864);
            to[i][1] = forward(64 << (2 * i), 4864, 896);
        }
    }
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 2; ++j)
            if (with[i][j] != without[i][j]) return printf("differ at %d %d\n", i, j), 1;
    printf("refused %d\n", refused);
    return 0;
}
"""


def test_plans_without_an_allocation(tmp_path):
    src, exe = str(tmp_path / "t.cpp"), str(tmp_path / "t")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-rdynamic", "-o", exe, src, "-ldl"], check=True)
    run = subprocess.run([exe, os.path.abspath(sw.LIB_PATH)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                         text=True, timeout=120)
    assert run.returncode == 0, run.stdout
    assert int(run.stdout.split("refused")[-1]) == 0
