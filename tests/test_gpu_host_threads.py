"""Host threads that call the library at once: calls that share a kernel and differ in the shared memory they need.

Python threads hardly overlap inside the calls, so the loops are C++ (compiled here against include/bsa.h).
"""
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <atomic>
#include <thread>
#include "bsa.h"
template <typename F, typename G>
static int both(int n, F f, G g) {
    std::atomic<int> ready{0}, bad{0};
    auto run = [&](auto call) {
        ++ready;
        while (ready < 2) {}
        for (int i = 0; i < n && !bad; ++i)
            if (int rc = call()) bad = rc;
    };
    std::thread a([&] { run(f); }), b([&] { run(g); });
    a.join();
    b.join();
    return bad;
}
extern "C" int norms(int n, const bsa_plan* p, const bsa_norm_args* wide, const bsa_norm_args* narrow, const void* x,
                     const void* y, void* x1, void* h1, void* h2, void* s1, void* s2) {
    return both(n, [&] { return bsa_residual_norm(p, wide, x, y, x1, h1, s1); },
                [&] { return bsa_norm_modulate(p, narrow, x, h2, s2); });
}
extern "C" int norm_gradients(int n, const bsa_plan* p, const bsa_norm_args* wide, const bsa_norm_args* narrow,
                              const void* x, const void* y, void* x1, void* x2, void* w1, void* w2, size_t bytes, void* s1,
                              void* s2) {
    auto one = [=](const bsa_norm_args* a, void* dx, void* w, void* s) {
        return bsa_norm_modulate_bwd(p, a, y, x, dx, nullptr, nullptr, nullptr, nullptr, w, bytes, s);
    };
    return both(n, [=] { return one(wide, x1, w1, s1); }, [=] { return one(narrow, x2, w2, s2); });
}
struct Route {
    const bsa_plan* p;
    const void *q, *k;
    int32_t *rows, *cols;
    int64_t cap;
    float* load;
    int64_t* nnz;
    void* ws;
    size_t bytes;
    void* stream;
    int operator()() const {
        return bsa_route(p, q, k, BSA_BF16, 0.5f, 2, rows, cols, cap, load, nnz, ws, bytes, stream);
    }
};
extern "C" int routes(int n, const Route* a, const Route* b) { return both(n, *a, *b); }
"""


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_top_b200 import build
    build.build()
    import block_sparse_attention_top_b200 as m
    return m


@pytest.fixture(scope="module")
def race(bsa, tmp_path_factory):
    d = tmp_path_factory.mktemp("race")
    (d / "race.cpp").write_text(SOURCE)
    home = os.path.dirname(bsa.LIB_PATH)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I",
                    os.path.join(os.path.dirname(home), "include"), str(d / "race.cpp"), bsa.LIB_PATH,
                    f"-Wl,-rpath,{home}", "-o", str(d / "race.so")], check=True)
    return ctypes.CDLL(str(d / "race.so"))


def rand(shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def P(t):
    return ctypes.c_void_p(t.data_ptr())


def test_norms(bsa, race):
    B, N, C = 1, 4, 5120
    plan = bsa.Plan(B, 1, 1, 1, N, 64, 64, bsa.BSA_ORDER_IDENTITY)
    x, y = rand((B, N, C), 1, torch.float32), rand((B, N, C), 2)
    (x1, h1), h2 = bsa.residual_norm(plan, x, y), bsa.norm_modulate(plan, x)
    got = [torch.empty_like(t) for t in (x1, h1, h2)]
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    a = bsa.NormArgs(C, 1, bsa.BSA_F32, bsa.BSA_NORM_LAYER, bsa.BSA_NORM_NONE, 1e-6, 1.0)
    rc = race.norms(20000, plan.handle, ctypes.byref(a), ctypes.byref(a), P(x), P(y), *map(P, got),
                    *(ctypes.c_void_p(t.cuda_stream) for t in s))
    torch.cuda.synchronize()
    assert rc == bsa.BSA_OK
    for t, want in zip(got, (x1, h1, h2)):
        assert torch.equal(t, want)


def test_norm_gradients(bsa, race):
    B, N, C, narrow = 1, 4, 4096, 2048
    plan = bsa.Plan(B, 1, 1, 1, N, 64, 64, bsa.BSA_ORDER_IDENTITY)
    x, y = rand((B, N, C), 1, torch.float32), rand((B, N, C), 2)
    lo = [t.view(-1)[:B * N * narrow].view(B, N, narrow) for t in (x, y)]
    want = bsa.norm_modulate_backward(plan, y, x).dx, bsa.norm_modulate_backward(plan, lo[1], lo[0]).dx
    got = [torch.empty_like(t) for t in want]
    ws = [torch.empty(1 << 24, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    a, b = (bsa.NormArgs(c, 1, bsa.BSA_F32, bsa.BSA_NORM_LAYER, bsa.BSA_NORM_NONE, 1e-6, 1.0) for c in (C, narrow))
    rc = race.norm_gradients(20000, plan.handle, ctypes.byref(a), ctypes.byref(b), P(x), P(y), *map(P, got), *map(P, ws),
                             ctypes.c_size_t(1 << 24), *(ctypes.c_void_p(t.cuda_stream) for t in s))
    torch.cuda.synchronize()
    assert rc == bsa.BSA_OK
    for t, w in zip(got, want):
        assert torch.equal(t, w)


class Route(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "q", "k", "rows", "cols")] + [("cap", ctypes.c_int64)] + \
        [(n, ctypes.c_void_p) for n in ("load", "nnz", "ws")] + [("bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)]


@pytest.mark.parametrize("sizes", [(1009, 1024), (1300, 2000)])
def test_routing(bsa, race, sizes):
    calls, checks, keep = [], [], []
    for nb in sizes:
        N, d = nb * 64, 64
        plan = bsa.Plan(1, 1, 1, 1, N, d, 64, bsa.BSA_ORDER_IDENTITY)
        q, k = rand((1, N, 1, d), nb), rand((1, N, 1, d), nb + 1)
        want = bsa.route(plan, q, k, 0.5, 2)
        got, ws, s = [torch.empty_like(t) for t in want], plan.workspace(bsa.BSA_OP_ROUTE), torch.cuda.Stream()
        calls.append(Route(plan.handle, q.data_ptr(), k.data_ptr(), got[0].data_ptr(), got[1].data_ptr(), got[1].numel(),
                           got[2].data_ptr(), got[3].data_ptr(), ws.data_ptr(), ws.numel(), s.cuda_stream))
        checks.append((got, want))
        keep.append((plan, q, k, ws, s))
    torch.cuda.synchronize()
    rc = race.routes(2000, ctypes.byref(calls[0]), ctypes.byref(calls[1]))
    torch.cuda.synchronize()
    assert rc == bsa.BSA_OK
    for got, want in checks:
        n = int(want[3].item())
        for a, b in zip((got[0], got[1][:n], got[2], got[3]), (want[0], want[1][:n], want[2], want[3])):
            assert torch.equal(a, b)
