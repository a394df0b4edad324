"""The calls of linear attention and the block norms on a stand-in for the CUDA runtime that launches nothing, counts, and can refuse one
launch (no GPU): a launch that fails ends its call with the error, without a later launch or an error left over for the next call; and
what a call writes may not overlap what it reads."""
import json
import os
import subprocess
import sys

import pytest

import hybrid_linear_attention_rule_gb300.build as B

FAKE = r"""
#include <stddef.h>
static int launches, refused, last;
void fake_refuse(int nth) { launches = 0; refused = nth; last = 0; }
int fake_launches(void) { return launches; }
static int launch(void) { return ++launches == refused ? (last = 1) : 0; }
int __cudaLaunchKernel(void) { return launch(); }
int cudaLaunchKernel(void) { return launch(); }
int cudaLaunchKernelExC(void) { return launch(); }
int cudaLaunchCooperativeKernel(void) { return launch(); }
int cudaGetLastError(void) { const int e = last; last = 0; return e; }
static int encode(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char *name, void **fn, unsigned version, unsigned long long flags, int *found) {
    *fn = (void *)encode;
    *found = 0;
    return 0;
}
int cudaGetDevice(int *device) { *device = 0; return 0; }
int cudaDeviceGetAttribute(int *value, int which, int device) { *value = 152; return 0; }
const char *cudaGetErrorString(int e) { return e ? "refused" : "no error"; }
const char *cudaGetErrorName(int e) { return cudaGetErrorString(e); }
static int module;
void **__cudaRegisterFatBinary(void *binary) { static void *handle = &module; return &handle; }
void __cudaRegisterFatBinaryEnd(void **handle) {}
void __cudaUnregisterFatBinary(void **handle) {}
void __cudaRegisterFunction(void) {}
void __cudaRegisterVar(void) {}
int __cudaGetKernel(void **kernel, const void *function) { *kernel = &module; return 0; }
int __cudaPushCallConfiguration(void) { return 0; }
int __cudaPopCallConfiguration(void) { return 0; }
int cudaFuncGetAttributes(void) { return 1; }
int cudaFuncSetAttribute(void) { return 0; }
int cudaGetSymbolAddress(void) { return 1; }
int cudaMemcpyAsync(void) { return 1; }
int cudaMemcpyFromSymbolAsync(void) { return 1; }
int cudaMemcpyToSymbolAsync(void) { return 1; }
int cudaMemsetAsync(void) { return 1; }
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(void) { return 1; }
int cudaStreamSynchronize(void) { return 1; }
"""

CHILD = r"""
import ctypes, json, sys
fake = ctypes.CDLL("libcudart.so.13")
lib = ctypes.CDLL(sys.argv[1])
P, I, F, L, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_size_t
at = lambda n: P(n << 40)
big = Z(1 << 38)
E = {0: 4, 1: 2}                                                     # bytes of an element
def prefill(bf, N, T, Hk, H):
    return lib.k3lin_prefill(at(1), at(2), at(3), I(bf), at(4), I(0), at(5), None, None, I(0), at(6), None, I(N), I(T), I(Hk), I(H), I(64), I(64), F(1),
                             at(7), I(bf), at(8), at(9), big, None)
def decode():
    return lib.k3lin_decode_step(at(1), at(2), at(3), I(1), at(4), I(0), at(5), None, None, I(4), I(4), I(2), I(2), I(64), I(64), F(1), at(6), I(1), None)
def backward(bf, fixed, N, T, Hk, H, dg):
    return lib.k3lin_backward(at(1), at(2), at(3), I(bf), at(4), I(fixed), at(5), at(6), None, I(N), I(T), I(Hk), I(H), I(64), I(64), F(1), at(7), at(8),
                              at(10), at(11), at(12), at(13) if dg else None, at(14), at(9), big, None)
def norm(back):
    if not back:
        return lib.k3blk_norm(at(1), I(1), at(2), at(3), I(0), at(4), at(5), L(100), I(64), F(1), F(0), at(6), at(7), None)
    return lib.k3blk_norm_backward(at(1), I(1), at(2), at(3), at(4), at(5), I(0), at(6), at(7), L(100), I(64), F(1), F(0), at(10), at(11), at(12), at(13),
                                   at(14), at(9), big, None)
calls = {"prefill bf16": lambda: prefill(1, 2, 5000, 2, 4), "prefill bf16, short": lambda: prefill(1, 1, 40, 2, 2), "prefill f32, cut": lambda: prefill(0, 1, 5000, 2, 2),
         "prefill f32": lambda: prefill(0, 400, 5000, 2, 2), "decode": decode, "norm": lambda: norm(False), "norm backward": lambda: norm(True)}
for bf in (0, 1):
    for fixed in (0, 1):
        for dg in (0, 1):
            for hk in (2, 4):
                calls["backward %d %d %d %d" % (bf, fixed, dg, hk)] = lambda bf=bf, fixed=fixed, dg=dg, hk=hk: backward(bf, fixed, 2, 5000, hk, 4, dg)
# arrays of a call: name, bytes, and whether it is written; calls take them by name
def lin(kind, bf, fixed):
    N, T, Hk, H, dk, dv, slots = 2, 40, 2, 4, 64, 32, 3
    key, rows, g, states = T * Hk * dk * E[bf], T * H * dv, (1 if fixed else T) * H * 4, H * dk * dv * 4
    if kind == "decode":
        key, rows, g = N * Hk * dk * E[bf], N * H * dv, (1 if fixed else N) * H * 4
    a = dict(q=(key, 0), k=(key, 0), v=(rows * E[bf], 0), g=(g, 0), workspace=(1 << 30, 1))
    if kind == "prefill":
        a.update(first=(slots * states, 0), out=(rows * E[1 - bf], 1), last=(slots * states, 1), cu=(4 * N + 4, 0), idx=(4 * N, 0))
        def call(p):
            return lib.k3lin_prefill(p["q"], p["k"], p["v"], I(bf), p["g"], I(fixed), p["first"], p["idx"], None, I(slots), p["cu"], None, I(N), I(T),
                                     I(Hk), I(H), I(dk), I(dv), F(1), p["out"], I(1 - bf), p["last"], p["workspace"], Z(1 << 30), None)
        a["workspace"] = (lib.k3lin_prefill_workspace_size(I(N), I(T), I(Hk), I(H), I(dk), I(dv), I(bf)), 1)
    elif kind == "decode":
        del a["workspace"]
        a.update(state=(slots * states, 1), out=(rows * E[1 - bf], 1), idx=(4 * N, 0))
        def call(p):
            return lib.k3lin_decode_step(p["q"], p["k"], p["v"], I(bf), p["g"], I(fixed), p["state"], p["idx"], None, I(slots), I(N), I(Hk), I(H), I(dk),
                                         I(dv), F(1), p["out"], I(1 - bf), None)
    else:
        a.update(do=(rows * E[bf], 0), first=(N * states, 0), dlast=(N * states, 0), dq=(key, 1), dk=(key, 1), dv=(rows * E[bf], 1), dg=(g, 1),
                 dfirst=(N * states, 1), cu=(4 * N + 4, 0))
        def call(p):
            return lib.k3lin_backward(p["q"], p["k"], p["v"], I(bf), p["g"], I(fixed), p["first"], p["cu"], None, I(N), I(T), I(Hk), I(H), I(dk), I(dv),
                                      F(1), p["do"], p["dlast"], p["dq"], p["dk"], p["dv"], p["dg"], p["dfirst"], p["workspace"], Z(1 << 30), None)
        a["workspace"] = (lib.k3lin_backward_workspace_size(I(N), I(T), I(Hk), I(H), I(dk), I(dv), I(bf)), 1)
    return a, call
def norms(kind, bf, _):
    rows, D = 37, 96
    size, w = rows * D * E[bf], 4 * D
    a = dict(x=(size, 0), gate=(size, 0), post=(w, 0), pre=(w, 0))
    if kind == "norm":
        a.update(residual=(size, 0), s=(size, 1), y=(size, 1))
        def call(p):
            return lib.k3blk_norm(p["x"], I(bf), p["residual"], p["gate"], I(0), p["post"], p["pre"], L(rows), I(D), F(1), F(0), p["s"], p["y"], None)
    else:
        a.update(ds=(size, 0), dy=(size, 0), sum=(size, 0), dx=(size, 1), dresidual=(size, 1), dgate=(size, 1), dpost=(w, 1), dpre=(w, 1),
                 workspace=(lib.k3blk_norm_backward_workspace_size(L(rows), I(D)), 1))
        def call(p):
            return lib.k3blk_norm_backward(p["x"], I(bf), p["ds"], p["dy"], p["sum"], p["gate"], I(0), p["post"], p["pre"], L(rows), I(D), F(1), F(0),
                                           p["dx"], p["dresidual"], p["dgate"], p["dpost"], p["dpre"], p["workspace"], Z(1 << 30), None)
    return a, call
def in_place(kind, x, y, a):
    # whether output x may be y
    if kind == "prefill":
        return (x, y) == ("last", "first")
    return "norm" in kind and a[x][0] == a[y][0] and not a[y][1] and (x, y) not in (("dresidual", "x"), ("dresidual", "gate"))
def overlaps():
    out = []
    for kind in ("prefill", "decode", "backward", "norm", "norm backward"):
        for bf in (0, 1):
            for fixed in (0, 1):
                a, call = (norms if "norm" in kind else lin)(kind, bf, fixed)
                place = {name: (i + 1) << 40 for i, name in enumerate(a)}
                run = lambda at: call({x: P(y) for x, y in at.items()})
                out.append([kind, "apart", "", 0, run(place)])
                for x, (size, written) in a.items():
                    if not written:
                        continue
                    for y, (other, _) in a.items():
                        if x == y:
                            continue
                        # x's last bytes on y's first, its first on y's last, the same place, and next to one another on either side
                        down, up = (size - 1) // 256 * 256, (other - 1) // 256 * 256
                        for to in (place[y] - down, place[y] + up, place[y]):
                            out.append([kind, x, y, 0 if to == place[y] and in_place(kind, x, y, a) else 1, run({**place, x: to})])
                        for to in (place[y] - (size + 255) // 256 * 256, place[y] + (other + 255) // 256 * 256):
                            out.append([kind, x, y, 0, run({**place, x: to})])
    return out
out = {"overlaps": overlaps()}
for name, call in calls.items():
    fake.fake_refuse(0)
    status, n = call(), fake.fake_launches()
    rows = [[status, n, fake.cudaGetLastError()]]
    for k in range(1, n + 1):
        fake.fake_refuse(k)
        rows.append([call(), fake.fake_launches(), fake.cudaGetLastError()])
    out[name] = rows
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def results(tmp_path_factory):
    d = tmp_path_factory.mktemp("cudart")
    (d / "fake.c").write_text(FAKE)
    (d / "fake.map").write_text("libcudart.so.13 { global: *; };\n")
    subprocess.run(["gcc", "-w", "-shared", "-fPIC", "-o", "libcudart.so.13", "fake.c", "-Wl,-soname,libcudart.so.13", "-Wl,--version-script,fake.map"],
                   cwd=d, check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, B.build()], env={**os.environ, "LD_LIBRARY_PATH": str(d)}, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)


def test_every_launch_is_checked(results):
    results = {name: rows for name, rows in results.items() if name != "overlaps"}
    assert len(results) == 23
    for name, (clean, *refused) in results.items():
        assert clean[0] == 0 and clean[1] > 0 and clean[2] == 0, name
        for k, (status, launches, left) in enumerate(refused, 1):
            assert status == -5, f"{name}: launch {k} of {clean[1]} failed and the call returned {status}"
            assert launches == k, f"{name}: launch {k} of {clean[1]} failed and the call went on to {launches}"
            assert left == 0, f"{name}: launch {k} of {clean[1]} left its error behind"


def test_calls_have_the_launches_that_they_should(results):
    n = {name: rows[0][1] for name, rows in results.items() if name != "overlaps"}
    assert n["prefill bf16, short"] == 2 and n["prefill bf16"] == 4 and n["decode"] == n["norm"] == 1 and n["norm backward"] == 2
    assert n["prefill f32, cut"] == 2 and n["prefill f32"] == 1


def test_what_is_written_may_not_overlap_what_is_read(results):
    seen = set()
    for kind, x, y, shared, status in results["overlaps"]:
        assert status == (-1 if shared else 0), (kind, x, y, shared)
        seen.add((kind, x, y))
    for kind, name in (("prefill", "apart"), ("decode", "apart"), ("backward", "apart")):
        assert (kind, name, "") in seen
    assert ("norm", "s", "x") in seen and ("norm backward", "dx", "dresidual") in seen
    assert ("prefill", "out", "first") in seen and ("backward", "dq", "dlast") in seen and ("backward", "dfirst", "g") in seen
