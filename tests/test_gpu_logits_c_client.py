"""The logits calls from C: a program compiled with gcc against include/ws.h
allocates device memory itself, runs the log probabilities, their gradient and
the distillation on short and long rows on a stream of its own, and writes the
results, which must be within the bounds of the 64-bit definitions
(logits_ref.py)."""
import os
import subprocess

import numpy as np
import pytest

import logits_ref as ref
import synth

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
K, T = 8, 1.25
SHAPES = [(4, 1000), (2, 50000)]

CLIENT = r"""
#include <stdio.h>
#include <stdlib.h>
#include <cuda_runtime.h>
#include "ws.h"

#define CHECK_WS(call) do { ws_status s_ = (call); if (s_ != WS_OK) { \
    fprintf(stderr, "%s: %s (%s)\n", #call, ws_status_string(s_), ws_last_error()); exit(1); } } while (0)
#define CHECK_CUDA(call) do { cudaError_t e_ = (call); if (e_ != cudaSuccess) { \
    fprintf(stderr, "%s: %s\n", #call, cudaGetErrorString(e_)); exit(1); } } while (0)

static const char* dir;

static void* input(const char* name, size_t bytes) {
    char path[4096];
    snprintf(path, sizeof path, "%s/%s", dir, name);
    void *h = malloc(bytes), *d;
    FILE* f = fopen(path, "rb");
    if (!h || !f || fread(h, 1, bytes, f) != bytes) { fprintf(stderr, "cannot read %s\n", path); exit(1); }
    fclose(f);
    CHECK_CUDA(cudaMalloc(&d, bytes));
    CHECK_CUDA(cudaMemcpy(d, h, bytes, cudaMemcpyHostToDevice));
    free(h);
    return d;
}

static void* output(size_t bytes) {
    void* d;
    CHECK_CUDA(cudaMalloc(&d, bytes));
    CHECK_CUDA(cudaMemset(d, 0x55, bytes));
    return d;
}

static void dump(const char* name, int i, const void* d, size_t bytes) {
    char path[4096];
    snprintf(path, sizeof path, "%s/%s%d", dir, name, i);
    void* h = malloc(bytes);
    CHECK_CUDA(cudaMemcpy(h, d, bytes, cudaMemcpyDeviceToHost));
    FILE* f = fopen(path, "wb");
    if (!f || fwrite(h, 1, bytes, f) != bytes) { fprintf(stderr, "cannot write %s\n", path); exit(1); }
    fclose(f);
    free(h);
}

int main(int argc, char** argv) {
    if (argc != 2) return 2;
    dir = argv[1];
    cudaStream_t stream;
    CHECK_CUDA(cudaStreamCreateWithFlags(&stream, cudaStreamNonBlocking));
    static const int64_t shapes[2][2] = {{4, 1000}, {2, 50000}};
    for (int i = 0; i < 2; ++i) {
        const int64_t rows = shapes[i][0], cols = shapes[i][1];
        const size_t n = (size_t)(rows * cols);
        char name[32];
        snprintf(name, sizeof name, "x%d", i);
        float* x = (float*)input(name, 4 * n);
        snprintf(name, sizeof name, "tok%d", i);
        int32_t* tok = (int32_t*)input(name, 4 * rows);
        snprintf(name, sizeof name, "g%d", i);
        float* g = (float*)input(name, 4 * rows);
        float *logprob = (float*)output(4 * rows), *entropy = (float*)output(4 * rows), *lse = (float*)output(4 * rows);
        float *stats = (float*)output(8 * rows), *top = (float*)output(32 * rows), *loss = (float*)output(4 * rows);
        float *grad = (float*)output(4 * n), *dgrad = (float*)output(4 * n);
        int32_t* idx = (int32_t*)output(32 * rows);
        ws_logprobs_desc d = {0};
        d.rows = rows; d.cols = cols; d.row_stride = cols; d.dtype = WS_DTYPE_F32; d.index_type = WS_INDEX_I32;
        d.k = 8; d.temperature = 1.25f;
        CHECK_WS(ws_logprobs_validate(&d));
        CHECK_WS(ws_logprobs(&d, x, tok, logprob, entropy, lse, stats, top, idx, stream));
        CHECK_WS(ws_logprobs_backward(&d, x, tok, stats, entropy, g, g, grad, cols, stream));
        ws_distill_desc e = {0};
        e.rows = rows; e.cols = cols; e.row_stride = cols; e.grad_stride = cols; e.dtype = WS_DTYPE_F32;
        e.index_type = WS_INDEX_I32; e.k = 8; e.mode = WS_DISTILL_TAIL; e.temperature = 1.25f;
        CHECK_WS(ws_distill_validate(&e));
        CHECK_WS(ws_distill(&e, x, idx, top, g, loss, dgrad, stream));
        if (ws_logprobs_backward(&d, x, tok, stats, entropy, g, g, x + 1, cols, stream) != WS_ERR_INVALID_ARGUMENT) return 3;
        CHECK_CUDA(cudaStreamSynchronize(stream));
        dump("logprob", i, logprob, 4 * rows); dump("entropy", i, entropy, 4 * rows); dump("lse", i, lse, 4 * rows);
        dump("top", i, top, 32 * rows); dump("idx", i, idx, 32 * rows); dump("loss", i, loss, 4 * rows);
        dump("grad", i, grad, 4 * n); dump("dgrad", i, dgrad, 4 * n);
    }
    uint32_t flags = 1;
    CHECK_WS(ws_device_error(&flags, 1));
    if (flags) { fprintf(stderr, "device error %u\n", flags); return 1; }
    printf("ok\n");
    return 0;
}
"""


def test_c_client_against_the_definitions(tmp_path):
    import __graft_entry__
    __graft_entry__.build()
    from post_processing_gb300 import binding
    lib_dir, cuda = os.path.dirname(binding.LIBRARY_PATH), "/usr/local/cuda"
    src, exe = tmp_path / "client.c", tmp_path / "client"
    src.write_text(CLIENT)
    subprocess.run(["gcc", "-std=c11", "-O1", "-I" + os.path.join(ROOT, "include"), "-I" + cuda + "/include", str(src), "-o",
                    str(exe), "-L" + lib_dir, "-l:libws.so", "-L" + cuda + "/lib64", "-lcudart",
                    "-Wl,-rpath," + lib_dir + ":" + cuda + "/lib64"], check=True)
    data = []
    for i, (rows, cols) in enumerate(SHAPES):
        x = synth.logits_with_ties(77 + i, rows, cols).astype(np.float32)
        tok, g = (np.arange(rows) * 13).astype(np.int32), np.linspace(0.5, 2.0, rows).astype(np.float32)
        for name, a in (("x", x), ("tok", tok), ("g", g)):
            a.tofile(tmp_path / f"{name}{i}")
        data.append((x, tok, g))
    run = subprocess.run([str(exe), str(tmp_path)], capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stderr
    for i, (x, tok, g) in enumerate(data):
        rows, cols = x.shape
        read = lambda name, t=np.float32: np.fromfile(tmp_path / f"{name}{i}", t)  # noqa: E731
        f = ref.logprobs(x.astype(np.float64), tok, K, T)
        d = ref.delta(cols, cols // 256 + 32)
        # ln S is off by d; a difference with z, and the products, by a few roundings of operands below 100
        bound = d + 600 * ref.U
        assert np.abs(read("logprob") - f["logprob"]).max() < bound and np.abs(read("lse") - f["lse"]).max() < bound
        assert np.abs(read("entropy") - f["entropy"]).max() < bound + 2 * d * np.log(cols)
        idx, top = read("idx", np.int32).reshape(rows, K), read("top").reshape(rows, K)
        assert np.array_equal(idx, f["top_idx"]) and np.abs(top - f["top_logprob"]).max() < bound
        grad, size = ref.backward(x.astype(np.float64), tok, g, g, T)
        assert (np.abs(read("grad").reshape(rows, cols) - grad) <= 20 * ref.U * size + 2 * d * size + ref.TINY["f32"]).all()
        loss, dgrad, loss_tol, grad_tol = ref.distill(x.astype(np.float64), idx, top, g, True, T, cols // 256 + 32)
        assert (np.abs(read("loss") - loss) <= loss_tol + ref.U * np.abs(loss)).all()
        assert (np.abs(read("dgrad").reshape(rows, cols) - dgrad) <= grad_tol + 2 * ref.U * np.abs(dgrad) + ref.TINY["f32"]).all()
